"""GPU tests of the serving operators at the ends of their ranges: rows of very large and very small
magnitude.  Tolerances as in test_gpu_serving: half a code step, and fp32 roundings of the sum and of
the factors of x_scale.
"""

import numpy as np
import pytest
import torch

from oracle import gptq_oracle as O
from post_weight_quantization_14_b200 import gptq as G

from . import gpu_util as U_
from .test_gpu_serving import Packed, _activations, _bf16, _check_rows, _e4m3, _rows_reference, _tensor, _x

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


# ------------------------------------------------------------------------------------ e4m3 product

def _near_zero_point(rng, d_out, d_in, bits, g, sym):
    """A layer whose codes lie at the zero point but for one in twenty, a step away; every third row and
    every second group of the rows after it lie at it altogether.  Zero points at both ends of the codes."""
    L = Packed(rng, d_out, d_in, bits, g, sym)
    top = (1 << bits) - 1
    gi = np.arange(d_in) // (d_in if g == -1 else g)
    z = np.full((L.ng, d_out), 1 << (bits - 1)) if sym else rng.choice([0, top, top - 1, top // 2], size=(L.ng, d_out))
    step = rng.choice([-1, 1], size=(d_out, d_in)) * (rng.random((d_out, d_in)) < 0.05)
    step[::3] = 0
    step[1::3, gi % 2 == 0] = 0
    codes = np.clip(z.T[:, gi] + step, 0, top)
    sc = rng.uniform(0.5, 1.5, size=(L.ng, d_out)).astype(np.float16)
    qw, qz = O.pack_qweight(codes, bits), None if sym else O.pack_qzeros(z, bits)
    L.qw, L.qz, L.sc = U_.t(qw), None if sym else U_.t(qz), U_.t(sc)
    L.What = O.dequant_packed(qw, sc, qz, d_out, d_in, bits, g, sym, None)
    return L


@pytest.mark.parametrize("M,d_out,d_in,bits,g,sym", [
    (3, 264, 128, 4, 128, False), (70, 264, 128, 4, -1, False), (130, 136, 128, 4, 32, False), (40, 136, 128, 3, 64, False),
    (200, 264, 128, 2, 128, False), (65, 136, 128, 4, 64, True), (2000, 1288, 128, 4, 128, False), (33, 136, 512, 4, -1, False),
    (300, 264, 1024, 4, 128, False), (20, 136, 1024, 3, 32, True), (64, 264, 4096, 4, 128, False)])
def test_gemm_e4m3_with_codes_at_the_zero_point(M, d_out, d_in, bits, g, sym):
    # q - z and its products are exact, so a row with q = z is 0 exactly, and the others are off by at most
    # one rounding, 2^-23 of S_g = sum |x| s |q - z|, for every 8 columns of a group or of a segment of 512
    # (one group per row), and 2^-23 of S for every group or segment and each of up to 8 joins, the scale
    # and the token's factor.
    rng = np.random.default_rng(M + d_in + bits + g)
    L = _near_zero_point(rng, d_out, d_in, bits, g, sym)
    X, Xv, xs, xsv = _x(rng, M, d_in, "e4m3")
    X = X.float().abs().to(torch.float8_e4m3fn)          # behind a gate: one sign
    Xv = np.abs(Xv)
    Y = torch.empty((M, d_out), device=U_.dev())
    L.gemm(X, xs, Y)
    G.gptq_sync_status()
    got = Y.double().cpu().numpy()
    dead = np.all(L.What == 0, axis=1)
    assert dead.sum() >= d_out // 3
    assert np.all(got[:, dead] == 0)
    run = min(d_in, 512 if g == -1 else g)
    S = (Xv @ np.abs(L.What).T) * xsv[:, None]
    tol = (run / 8 + d_in / run + 10) * 2.0 ** -23 * S
    err = np.abs(got - Xv @ L.What.T * xsv[:, None])
    assert np.all(err <= tol), float(np.max(err / np.maximum(tol, 1e-300)))


@pytest.mark.parametrize("bits,g,sym", [(4, 128, False), (4, 32, False), (3, 64, False), (2, -1, False), (4, 64, True)])
def test_gemm_e4m3_extreme_codes_and_scales(bits, g, sym):
    rng = np.random.default_rng(bits + g)
    M, d_out, d_in = 37, 136, 256
    L = Packed(rng, d_out, d_in, bits, g, sym)
    top = (1 << bits) - 1
    qw = O.pack_qweight(rng.choice([0, top], size=(d_out, d_in)), bits)
    qz = None if sym else O.pack_qzeros(rng.choice([0, top], size=(L.ng, d_out)), bits)
    sc = rng.choice([0.0, 2.0 ** -24, 6e-8, 65504.0, 1.0], size=(L.ng, d_out)).astype(np.float16)
    L.qw, L.qz, L.sc = U_.t(qw), None if sym else U_.t(qz), U_.t(sc)
    L.What = O.dequant_packed(qw, sc, qz, d_out, d_in, bits, g, sym, None)
    X, Xv, xs, xsv = _x(rng, M, d_in, "e4m3")
    Y = torch.empty((M, d_out), device=U_.dev())
    L.gemm(X, xs, Y)
    G.gptq_sync_status()
    L.check(Y, Xv, xsv)


# ------------------------------------------------------------------------------------ long rows of one sign

def _tiled(rng, d_out, d_in, bits, g, act):
    """A layer of 32 different rows, over and over (enough blocks of rows that K is not split), with
    positive weights: every rounding of a sum in one direction would add up."""
    L = Packed(rng, 32, d_in, bits, g, False, act)
    top = (1 << bits) - 1
    qw = O.pack_qweight(rng.integers(1, top + 1, size=(32, d_in)), bits)
    qz = O.pack_qzeros(np.zeros((L.ng, 32), dtype=np.int64), bits)
    sc = rng.uniform(0.5, 1.5, size=(L.ng, 32)).astype(np.float16)
    L.What = O.dequant_packed(qw, sc, qz, 32, d_in, bits, g, False, None if L.gi is None else L.gi.cpu().numpy())
    rep = d_out // 32
    L.qw, L.sc = U_.t(qw).repeat(1, rep).contiguous(), U_.t(sc).repeat(1, rep).contiguous()
    L.qz = U_.t(qz).repeat(1, rep).contiguous()          # 32 codes fill whole words
    L.args = (d_out, d_in, bits, g, False)
    return L


@pytest.mark.parametrize("M,d_out,bits,g,act,x", [
    (3, 56832, 2, -1, 0, "bf16"), (3, 56832, 2, -1, 0, "e4m3"), (3, 9472, 4, 128, 1, "bf16"), (3, 9472, 2, 64, 1, "e4m3"),
    (3, 9472, 3, 16, 1, "bf16"), (12, 9472, 4, 128, 1, "bf16"), (50, 9472, 4, 64, 1, "bf16"), (33, 9472, 2, 64, 1, "e4m3")])
def test_gemv_of_long_rows_has_no_bias(M, d_out, bits, g, act, x):
    # A tensor instruction may cut its sums off: at most 2^-23 of a partial sum each time, always in the same
    # direction.  As a partial sum takes 8 of them at most before it is added to the total in fp32 (rounded
    # to nearest), that is 8 2^-23 of the sum.  A warp adds some 256 partial sums, whose roundings to nearest
    # are independent: 2^-24 of the sum each, taken as if at its end throughout; five standard deviations
    # (each 2^-24 / sqrt 3) are allowed, and four roundings for joins, scales and the token's factor.
    rng = np.random.default_rng(bits + g + d_out)
    d_in = 65536
    L = _tiled(rng, d_out, d_in, bits, g, act)
    a = np.abs(_activations(rng, M, d_in))   # of many magnitudes, so that sums have bits to lose
    xs = xsv = None
    if x == "bf16":
        X, Xv = _bf16(a)
    else:
        X, Xv = _e4m3(a * 20)
        xsv = np.full(M, 0.5)
        xs = U_.t(xsv.astype(np.float32))
    Y = torch.empty((M, d_out), device=U_.dev())
    L.gemv(X, Y, xs)
    G.gptq_sync_status()
    ref = Xv @ L.What.T * (1.0 if xsv is None else xsv[:, None])
    rel = Y.double().cpu().numpy().reshape(M, d_out // 32, 32) / ref[:, None, :] - 1
    tol = 8 * 2.0 ** -23 + (5 * np.sqrt(256 / 3) + 4) * 2.0 ** -24
    assert np.all(np.abs(rel) <= tol), (float(np.abs(rel).max() / tol), float(rel.mean() / tol))
