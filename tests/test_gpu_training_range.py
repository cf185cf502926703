"""The training operators over the whole range that they document, on the GPU against the 64-bit formulas of
tests/traincheck.py: rests and lists far apart, NaN in a list, temperatures whose inverse is large or small, sums of very
unlike terms."""
import math

import numpy as np
import pytest

from tests import traincheck as tc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import decode_sampling_tail_gb300 as dst  # noqa: E402
from tests.test_gpu_training import DEV, DT, INF, _dev, _lists, _logits, _np, f32  # noqa: E402


# ------------------------------------------------------------------ a rest that outweighs its list, or is nothing beside it

ABOVE = [-120.0, -30.0, 0.5, 5.0, 10.0, 17.0, 18.0, 20.0, 25.0, 40.0, 60.0, 69.0, 75.0, 85.0, 100.0, 130.0]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 60000])  # a CTA a row, and a cluster
@pytest.mark.parametrize("T", [1.0, f32(0.7)])
def test_distill_with_a_rest_far_from_its_list(V, dt, T):
    rng = np.random.default_rng(V)
    k, kinds = 12, 6
    rows = kinds * len(ABOVE)
    z = rng.standard_normal((rows, V)).astype(np.float32)
    idx = np.stack([rng.permutation(V)[:k] for _ in range(rows)]).astype(np.int32)
    vals = rng.standard_normal((rows, k)).astype(np.float32)
    for r in range(rows):
        kind = r % kinds
        if kind == 0:
            z[r, np.setdiff1d(np.arange(40), idx[r])[0]] = 24.0  # a student sure of a token outside the list
        if kind == 1:
            z[r, idx[r, 3]] = 24.0                               # of one in it
        if kind == 2:
            z[r] = 0.25                                          # of none
        if kind == 3:
            idx[r, :3], vals[r, :3] = -1, 30.0                   # the teacher's likely tokens are none of the student's
        if kind == 4:
            z[r, idx[r]] -= 20.0                                 # the student knows as little of the list
    z = _np(_dev(z, DT[dt])).astype(np.float32)
    top = np.where(idx >= 0, vals, -INF).max(1).astype(np.float64) / T
    rest = (top + np.repeat(ABOVE, kinds)).astype(np.float32)
    w = rng.uniform(0.5, 2.0, rows).astype(np.float32)
    loss, g = (_np(x) for x in dst.distill_topk(_dev(z, DT[dt]), _dev(vals), _dev(idx), teacher_rest=_dev(rest),
                                                temperature=T, weight=_dev(w)))
    alone = _np(dst.distill_topk(_dev(z, DT[dt]), _dev(vals), _dev(idx), teacher_rest=_dev(rest), temperature=T,
                                 weight=_dev(w), grad=False)[0])
    for r in range(rows):
        v, tol = tc.distill(z[r], vals[r], idx[r], float(rest[r]), T, float(w[r]), dt)
        what = f"row {r} (student {r % kinds}, rest {ABOVE[r // kinds]} above the list)"
        tc.near(loss[r], v[0], tol[0], "loss of " + what)
        tc.near(alone[r], v[0], tol[0], "loss alone of " + what)
        tc.near(g[r], v[1], tol[1], "gradient of " + what)


