"""GPU tests of the serving operators at the ends of their ranges: rows of very large and very small
magnitude.  Tolerances as in test_gpu_serving: half a code step, and fp32 roundings of the sum and of
the factors of x_scale.
"""

import numpy as np
import pytest
import torch

from post_weight_quantization_14_b200 import gptq as G

from . import gpu_util as U_
from .test_gpu_serving import _activations, _check_rows, _rows_reference, _tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_cuda(cuda_dev):
    yield


# ---------------------------------------------------------------------------------------- rows

def _far_rows(rng, d):
    """Rows whose squares leave the range of fp32, or whose sum of squares does, beside ordinary ones."""
    a = rng.standard_normal((9, d))
    a[1] *= 2.0 ** 59 / np.abs(a[1]).max()          # below 2^60
    a[2] = np.sign(a[2]) * 2.0 ** 59                # d 2^118
    a[3] *= 2.0 ** 118 / np.abs(a[3]).max()
    a[4] *= 2.0 ** -80 / np.abs(a[4]).max()         # squares below fp32
    a[5] *= 2.0 ** -62 / np.abs(a[5]).max()         # squares among the subnormals
    a[6, d - 1] = 2.0 ** 70                         # one large value among ordinary ones
    a[7] *= 2.0 ** -90
    a[7, d // 2] = 0.5                              # one ordinary value among small ones
    a[8, : d // 2] *= 2.0 ** -70                    # half a row each
    return a


@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("xt,wt,res", [("f32", "f32", False), ("bf16", "f32", False), ("bf16", "bf16", True),
                                       ("f32", "bf16", True)])
@pytest.mark.parametrize("M,d", [(9, 64), (900, 64), (9, 8192), (450, 8192), (9, 65536)])
def test_rms_norm_of_rows_of_any_magnitude(M, d, xt, wt, res, eps):
    rng = np.random.default_rng(M + d)
    X, Xv = _tensor(np.tile(_far_rows(rng, d), (M // 9, 1)), xt)
    w, wv = _tensor(1 + 0.2 * rng.standard_normal(d), wt)
    R, Rv = (torch.zeros_like(X), 0.0) if res else (None, 0.0)
    if res:   # X + R is then exact: half of X (a power of two), on both sides
        X, Xv, Rv = X * 0.5, Xv * 0.5, Xv * 0.5
        R = X.clone()
    X8, xs = torch.empty((M, d), dtype=torch.float8_e4m3fn, device=U_.dev()), torch.empty(M, device=U_.dev())
    G.gptq_rms_norm_e4m3(X, w, X8, xs, R, R, eps)
    G.gptq_sync_status()
    y, scale = _rows_reference(Xv + Rv, wv, eps)
    _check_rows(X8, xs, y, scale, d)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 8192, 65536])
def test_rms_norm_rows_that_are_not_finite_stay_marked(d, xt):
    rng = np.random.default_rng(d + 1)
    a = _far_rows(rng, d)
    a[1, 3] = np.nan
    a[3, d - 1] = -np.inf
    a[4, 0] = np.inf
    a[5, d // 2] = np.nan
    X, Xv = _tensor(a, xt)
    w = torch.ones(d, device=U_.dev())
    X8, xs = torch.empty((9, d), dtype=torch.float8_e4m3fn, device=U_.dev()), torch.empty(9, device=U_.dev())
    G.gptq_rms_norm_e4m3(X, w, X8, xs, eps=0.0)
    assert not torch.isfinite(xs[[1, 3, 4, 5]]).any()
    fine = [0, 2, 6, 7, 8]
    y, scale = _rows_reference(Xv[fine], np.ones(d), 0.0)
    _check_rows(X8[fine], xs[fine], y, scale, d)


@pytest.mark.parametrize("exp", [-100, -60, 60, 101, 112])
@pytest.mark.parametrize("M,d", [(3, 64), (400, 4096), (400, 8200), (5, 40000)])
def test_quantize_boundaries_between_codes_at_any_magnitude(M, d, exp):
    # as test_quantize_e4m3_boundaries_between_codes: 448 v / a lies on a boundary exactly or far from it
    rng = np.random.default_rng(M + d + exp + 1000)
    X, Xv = _tensor(_activations(rng, M, d) * 2.0 ** exp, "bf16")
    assert np.all(np.isfinite(Xv))
    X8, xs = torch.empty((M, d), dtype=torch.float8_e4m3fn, device=U_.dev()), torch.empty(M, device=U_.dev())
    G.gptq_quantize_e4m3(X, X8, xs)
    a = np.max(np.abs(Xv), axis=1)
    want = torch.from_numpy((448.0 * Xv / a[:, None]).astype(np.float32)).to(torch.float8_e4m3fn)
    assert torch.equal(X8.cpu().float(), want.float())
    assert np.all(np.abs(xs.double().cpu().numpy() - a / 448.0) <= 2.0 ** -24 * a / 448.0)
