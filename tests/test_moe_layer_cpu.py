"""Refusals of the mixture-of-experts layer's entry points (host side, no GPU), and its struct against the header."""
import ctypes

import pytest

import decode_sampling_tail_gb300 as dst
from decode_sampling_tail_gb300 import build as dbuild
from tests.test_abi_cpu import header_struct_fields


@pytest.fixture(scope="module")
def L():
    dbuild.build()
    return dst.lib()


BASE = dict(H=64, I=32, E=4, topk=2, n_shared=0, t_max=4, eps=1e-5, weight_dtype=dst.TAIL_BF16, act=0, act_alpha=1.0,
            act_beta=0.0, act_limit=0.0, interleaved=0, score=0, route_scale=1.0)


def create(L, **kw):
    v = {**BASE, **kw}
    cfg = dst.tail_moe_config(*[v[f[0]] for f in dst.tail_moe_config._fields_])
    h = ctypes.c_void_p()
    rc = L.tail_moe_create(ctypes.byref(cfg), 0, ctypes.byref(h))
    if h.value:
        L.tail_moe_destroy(h)
    return rc


NAN = float("nan")


@pytest.mark.parametrize("kw", [
    dict(H=0), dict(I=0), dict(E=0), dict(topk=0), dict(topk=5), dict(n_shared=-1), dict(t_max=0), dict(eps=-1.0),
    dict(eps=NAN), dict(weight_dtype=dst.TAIL_F32), dict(weight_dtype=9), dict(act=2), dict(score=2),
    dict(act_limit=-1.0), dict(act_limit=NAN), dict(act_alpha=NAN), dict(act_beta=NAN), dict(route_scale=NAN)])
def test_create_refuses(L, kw):
    assert create(L, **kw) == dst.TAIL_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(H=40), dict(I=24), dict(H=48, weight_dtype=dst.TAIL_MXFP4), dict(I=48, weight_dtype=dst.TAIL_MXFP4),
    dict(H=16400), dict(I=16416), dict(E=513), dict(E=510, n_shared=3), dict(E=64, topk=17), dict(n_shared=9),
    dict(t_max=65)])
def test_create_limits(L, kw):
    assert create(L, **kw) == dst.TAIL_ERR_UNSUPPORTED
    assert L.tail_last_error()


def test_null_handles(L):
    assert L.tail_moe_create(None, 0, ctypes.byref(ctypes.c_void_p())) == dst.TAIL_ERR_INVALID_ARG
    cfg = dst.tail_moe_config(*[BASE[f[0]] for f in dst.tail_moe_config._fields_])
    assert L.tail_moe_create(ctypes.byref(cfg), 0, None) == dst.TAIL_ERR_INVALID_ARG
    assert L.tail_moe_run(*[None] * 11, 1, *[None] * 5) == dst.TAIL_ERR_INVALID_ARG
    n = ctypes.c_int64()
    assert L.tail_moe_get_info(None, ctypes.byref(n)) == dst.TAIL_ERR_INVALID_ARG
    L.tail_moe_destroy(None)


def test_struct_and_constants_mirror_the_header():
    assert [f[0] for f in dst.tail_moe_config._fields_] == header_struct_fields("tail_moe_config")
    from decode_sampling_tail_gb300 import moe_layer
    from tests.test_abi_cpu import HEADER
    text = open(HEADER).read()
    for name, value in (("TAIL_MOE_GLU", moe_layer.ACTS["glu"]), ("TAIL_MOE_RELU2", moe_layer.ACTS["relu2"]),
                        ("TAIL_MOE_SOFTMAX", moe_layer.SCORES["softmax"]),
                        ("TAIL_MOE_SIGMOID", moe_layer.SCORES["sigmoid"]), ("TAIL_MXFP4", dst.TAIL_MXFP4)):
        assert f"{name} = {value}" in text


def test_wait_limit_needs_a_handle(L):
    assert L.tail_moe_set_wait_limit(None, 1) == dst.TAIL_ERR_INVALID_ARG
