"""A mixture-of-experts layer for a few tokens on torch CUDA tensors (tail_moe_create, tail_moe_run).

It forms the hidden state that the tail reads (``out_hidden``, for ``Tail.run``), or the slots and weights
that ``Tail.run_moe`` combines inside its first kernel.  ``include/tail.h`` states the formulas.
"""
from __future__ import annotations

import ctypes

from . import TAIL_BF16, TAIL_MXFP4, TAIL_OK, TailError, lib, tail_moe_config
from ._args import allocating_on, fail, need, need_opt, raw_stream

WEIGHTS = {"bf16": TAIL_BF16, "mxfp4": TAIL_MXFP4}
ACTS = {"glu": 0, "relu2": 1}
SCORES = {"softmax": 0, "sigmoid": 1}


class Moe:
    """A layer handle bound to one device; the weights stay the caller's tensors.

    ``w1`` is [n, N1, H] and ``w2`` [n, H, I] bfloat16 with n = E + n_shared and N1 = 2 I ("glu") or I ("relu2");
    with ``weight_dtype="mxfp4"`` they are uint8 [n, N1, H / 2] and [n, H, I / 2] and ``w1_scale`` [n, N1, H / 32],
    ``w2_scale`` [n, H, I / 32] uint8 hold the block exponents.  Runs of one handle share its scratch: one at a time.
    """

    def __init__(self, H: int, I: int, E: int, topk: int, t_max: int = 64, *, n_shared: int = 0, eps: float = 1e-5,
                 weight_dtype: str = "bf16", act: str = "glu", act_alpha: float = 1.0, act_beta: float = 0.0,
                 act_limit: float = 0.0, interleaved: bool = False, score: str = "softmax", route_scale: float = 1.0,
                 device: int = 0):
        self.h = None
        self.cfg = tail_moe_config(H, I, E, topk, n_shared, t_max, eps, WEIGHTS[weight_dtype], ACTS[act], act_alpha,
                                   act_beta, act_limit, int(interleaved), SCORES[score], route_scale)
        self.device = device
        h = ctypes.c_void_p()
        rc = lib().tail_moe_create(ctypes.byref(self.cfg), device, ctypes.byref(h))
        if rc != TAIL_OK:
            fail(rc, "tail_moe_create")
        self.h = h.value

    def close(self):
        if self.h:
            lib().tail_moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def run(self, x, gamma, router_w, w1, w2, *, router_bias=None, w1_scale=None, w2_scale=None, b1=None, b2=None,
            out_hidden=None, out_slots=None, out_slot_w=None, out_ids=None, stream=None):
        """One run over x [T, H] bfloat16 (tail_moe_run).  gamma [H] float32 or None (x is already normalised),
        router_w [E, H] bfloat16, router_bias [E], b1 [n, N1], b2 [n, H] float32 or None.  Outputs: out_hidden
        [T, H] bfloat16 (may be x), out_slots [T, S, H] and out_slot_w [T, S] float32, out_ids [T, S] int32 with
        S = topk + n_shared; out_hidden is allocated when neither it nor out_slots is given.  Returns out_hidden."""
        import torch
        if not self.h:
            raise ValueError("the handle is closed")
        c, d = self.cfg, self.device
        if x.dim() != 2 or x.shape[0] > c.t_max:
            raise ValueError(f"x must be [T, {c.H}] with T <= {c.t_max}; got {tuple(x.shape)}")
        T, H, I, E, n, S = x.shape[0], c.H, c.I, c.E, c.E + c.n_shared, c.topk + c.n_shared
        N1 = 2 * I if c.act == 0 else I
        bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
        if c.weight_dtype == TAIL_MXFP4:
            if w1_scale is None or w2_scale is None:
                raise ValueError("mxfp4 weights need w1_scale and w2_scale")
            p1, p2 = need(w1, "w1", u8, (n, N1, H // 2), d), need(w2, "w2", u8, (n, H, I // 2), d)
            s1 = need(w1_scale, "w1_scale", u8, (n, N1, H // 32), d)
            s2 = need(w2_scale, "w2_scale", u8, (n, H, I // 32), d)
        else:
            if w1_scale is not None or w2_scale is not None:
                raise ValueError("bf16 weights take no scales")
            p1, p2, s1, s2 = need(w1, "w1", bf16, (n, N1, H), d), need(w2, "w2", bf16, (n, H, I), d), None, None
        if out_hidden is None and out_slots is None:
            with allocating_on(stream, d):
                out_hidden = torch.empty((T, H), dtype=bf16, device=d)
        rc = lib().tail_moe_run(
            self.h, need(x, "x", bf16, (T, H), d), need_opt(gamma, "gamma", f32, (H,), d),
            need(router_w, "router_w", bf16, (E, H), d), need_opt(router_bias, "router_bias", f32, (E,), d), p1, s1,
            need_opt(b1, "b1", f32, (n, N1), d), p2, s2, need_opt(b2, "b2", f32, (n, H), d), T,
            need_opt(out_hidden, "out_hidden", bf16, (T, H), d),
            need_opt(out_slots, "out_slots", f32, (T, S, H), d),
            need_opt(out_slot_w, "out_slot_w", f32, (T, S), d), need_opt(out_ids, "out_ids", torch.int32, (T, S), d),
            raw_stream(stream, d))
        if rc != TAIL_OK:
            raise TailError(rc, "tail_moe_run")
        return out_hidden

    def check(self):
        """Synchronises and raises when a bounded device wait of a run ran out (tail_moe_check)."""
        rc = lib().tail_moe_check(self.h)
        if rc != TAIL_OK:
            raise TailError(rc, "tail_moe_check")

    def set_wait_limit(self, ns: int):
        """Bounds every device wait of later runs to ``ns`` nanoseconds (tail_moe_set_wait_limit; 1e9 at first)."""
        rc = lib().tail_moe_set_wait_limit(self.h, ns)
        if rc != TAIL_OK:
            raise TailError(rc, "tail_moe_set_wait_limit")
