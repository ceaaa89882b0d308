"""GPU parity of the operators that serve a quantized layer (gptq_dequant_gemv,
gptq_dequant_gemm_e4m3, gptq_rms_norm_e4m3, gptq_quantize_e4m3) against the fp64 oracle.

Tolerances, from the arithmetic:

* Products.  x (q - z) is exact, and sums are fp32: at most one rounding or truncation, 2^-23
  of the running sum, for every 8 terms (the tensor instructions add 16 or 32 terms, a lane adds
  an eighth of d_in), one for each group and a few where partial sums are joined.  The running
  sums are at most S = sum_k |x_k| |w_hat_k|, so |Y - ref| <= (d_in / 8 + n_groups + 32) 2^-23 S.
  A bf16 Y is rounded once more: 2^-8 |ref|.
* Rows.  x_scale: a sum of d_in squares (a relative error of at most (d_in / 8 + 32) 2^-24,
  halved by the root) and a few fp32 roundings, 8 2^-24 in all.  X8: half an e4m3 step of the
  value v = y / x_scale, which is 2^-4 |v| or, below 2^-6, 2^-10, and fp32 roundings of v
  itself, 8 2^-24 |v|.  residual_out: half a bf16 step 2^-8 |h|, and an fp32 addition's 2^-24 |h|.
"""

import threading

import numpy as np
import pytest
import torch

from oracle import gptq_oracle as O
from post_weight_quantization_14_b200 import gptq as G
from post_weight_quantization_14_b200.inputs import bf16_bits_from_f32, f32_from_bf16_bits

from . import gpu_util as U_

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_cuda(cuda_dev):
    yield


# ------------------------------------------------------------------------------------- helpers

def _bf16(a):
    """fp32 array -> (bf16 tensor on the device, its values in fp64)."""
    bits = bf16_bits_from_f32(np.ascontiguousarray(a, dtype=np.float32))
    return U_.t(bits.view(np.int16)).view(torch.bfloat16), f32_from_bf16_bits(bits).astype(np.float64)


def _e4m3(a):
    """fp32 array -> (e4m3 tensor on the device, its values in fp64)."""
    x = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x.to(U_.dev()), x.double().numpy()


class Packed:
    """A layer with random codes, scales and zero points in the quantizer's layouts."""

    def __init__(self, rng, d_out, d_in, bits, g, sym, act=0):
        ng = O.n_groups(d_in, g)
        self.args = (d_out, d_in, bits, g, sym)
        self.ng = ng
        qw = O.pack_qweight(rng.integers(0, 1 << bits, size=(d_out, d_in)), bits)
        sc = (rng.uniform(1e-3, 5e-2, size=(ng, d_out)) * rng.choice([-1, 1], size=(ng, d_out))).astype(np.float16)
        qz = None if sym else O.pack_qzeros(rng.integers(0, 1 << bits, size=(ng, d_out)), bits)
        gi = (rng.permutation(d_in) // (d_in if g == -1 else g)).astype(np.int32) if act else None
        self.What = O.dequant_packed(qw, sc, qz, d_out, d_in, bits, g, sym, gi)
        self.qw, self.sc = U_.t(qw), U_.t(sc)
        self.qz = None if sym else U_.t(qz)
        self.gi = None if gi is None else U_.t(gi)
        self.cfg = G.make_config(bits, g, sym, desc_act=act)

    def gemv(self, X, Y, xs=None, stream=None):
        return G.gptq_dequant_gemv(X, self.qw, self.sc, self.qz, *self.args[:2], self.cfg, Y, xs, self.gi, stream)

    def gemm(self, X8, xs, Y, stream=None):
        return G.gptq_dequant_gemm_e4m3(X8, xs, self.qw, self.sc, self.qz, *self.args[:2], self.cfg, Y, stream)

    def check(self, Y, X, xs=None):
        ref, S = X @ self.What.T, np.abs(X) @ np.abs(self.What).T
        if xs is not None:
            ref, S = ref * xs[:, None], S * np.abs(xs)[:, None]
        tol = (self.args[1] / 8 + self.ng + 32) * 2.0 ** -23 * S
        if Y.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(ref)
        got = Y.double().cpu().numpy()
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)))


def _guarded(M, N, dtype):
    """[M, N] inside a larger array whose rest must stay as it is."""
    pad = 64
    buf = torch.full((M * N + pad,), 7.0, dtype=dtype, device=U_.dev())
    buf[:M * N] = float("nan")
    return buf, buf[:M * N].view(M, N)


def _activations(rng, M, d):
    return rng.standard_normal((M, d)) * np.exp(rng.standard_normal(d))[None, :]


def _x(rng, M, d, kind):
    a = _activations(rng, M, d)
    if kind == "bf16":
        t, v = _bf16(a)
        return t, v, None, None
    t, v = _e4m3(a * 20)
    xs = rng.uniform(0.01, 0.1, size=M).astype(np.float32)
    return t, v, U_.t(xs), xs.astype(np.float64)


# ------------------------------------------------------------------------------------ products

GEMV = [
    # M, d_out, d_in, bits, g, sym, act, x, y
    (1, 1, 8, 4, -1, False, 0, "bf16", "f32"),         # the smallest layer
    (1, 3, 16, 2, 16, False, 0, "e4m3", "bf16"),
    (2, 5, 24, 3, 16, True, 0, "bf16", "bf16"),        # a last group of 8 columns, words cut short
    (5, 33, 40, 8, 32, False, 0, "e4m3", "f32"),
    (8, 64, 72, 3, 64, False, 0, "bf16", "f32"),
    (9, 65, 136, 4, 128, False, 0, "bf16", "bf16"),    # one token and one row past a tile
    (1, 4096, 4096, 4, 128, False, 0, "bf16", "f32"),
    (16, 256, 1000, 4, 64, True, 0, "e4m3", "f32"),    # d_in no multiple of the group
    (17, 100, 520, 2, 32, False, 0, "bf16", "f32"),
    (31, 130, 264, 8, -1, False, 0, "bf16", "bf16"),
    (33, 127, 2048, 4, 16, False, 0, "bf16", "f32"),
    (64, 96, 512, 3, 32, False, 0, "e4m3", "bf16"),
    (64, 1028, 768, 4, 128, True, 0, "e4m3", "f32"),
    (3, 72, 65536, 2, 128, False, 0, "bf16", "f32"),   # the longest rows
    (2, 20000, 256, 4, 32, False, 0, "bf16", "bf16"),
    (4, 516, 1536, 8, 16, False, 0, "e4m3", "f32"),
    (4, 516, 1536, 3, 16, False, 0, "e4m3", "f32"),
    (4, 516, 1536, 2, 16, True, 0, "bf16", "f32"),
    (3, 40, 384, 4, -1, False, 0, "bf16", "f32"),      # one group per row; the last columns fill half a stage
    (20, 132, 4224, 3, -1, True, 0, "e4m3", "f32"),
    # activation order
    (1, 1, 8, 4, -1, False, 1, "bf16", "f32"),
    (1, 37, 64, 3, 16, False, 1, "bf16", "f32"),
    (2, 512, 1000, 4, 128, False, 2, "bf16", "bf16"),
    (7, 130, 2056, 8, 32, True, 1, "e4m3", "f32"),
    (8, 1024, 4096, 4, 128, False, 1, "bf16", "f32"),
    (33, 44, 520, 2, 64, False, 1, "e4m3", "f32"),
    (64, 70, 16384, 4, 16, False, 1, "bf16", "f32"),   # 1024 groups
    (3, 36, 32768, 4, 16, False, 1, "e4m3", "f32"),    # 2048 groups: no table
    (17, 133, 65536, 3, 32, False, 1, "bf16", "f32"),  # the same, odd rows, several token tiles
    (9, 24, 24576, 8, 16, True, 1, "e4m3", "bf16"),
    (2, 129, 16392, 3, 16, False, 2, "e4m3", "bf16"),
    (9, 300, 1032, 3, 32, False, 1, "bf16", "f32"),
]


@pytest.mark.parametrize("M,d_out,d_in,bits,g,sym,act,x,y", GEMV)
def test_gemv_matches_fp64(M, d_out, d_in, bits, g, sym, act, x, y):
    rng = np.random.default_rng(1000 * M + d_out + d_in + bits + g)
    L = Packed(rng, d_out, d_in, bits, g, sym, act)
    X, Xv, xs, xsv = _x(rng, M, d_in, x)
    buf, Y = _guarded(M, d_out, torch.float32 if y == "f32" else torch.bfloat16)
    assert L.gemv(X, Y, xs) is Y
    G.gptq_sync_status()
    L.check(Y, Xv, xsv)
    assert torch.all(buf[M * d_out:] == 7.0)
    first = Y.clone()
    L.gemv(X, Y, xs)
    assert torch.equal(first, Y)     # the same bits on every run


GEMM = [
    # M, d_out, d_in, bits, g, sym, y
    (1, 8, 32, 4, -1, False, "f32"),
    (1, 8, 32, 2, 32, True, "bf16"),
    (2, 136, 96, 3, 32, False, "f32"),
    (7, 256, 160, 4, 32, False, "bf16"),
    (33, 120, 128, 4, 64, False, "f32"),
    (64, 128, 256, 2, 128, False, "f32"),
    (65, 264, 1024, 4, 128, False, "bf16"),
    (129, 392, 640, 3, 64, True, "f32"),
    (255, 128, 4096, 4, -1, False, "f32"),
    (257, 1032, 512, 4, 128, True, "bf16"),
    (300, 520, 672, 2, 32, False, "f32"),
    (513, 2056, 2048, 4, 128, False, "f32"),
    (1000, 144, 8192, 3, 128, False, "bf16"),
    (40, 4096, 1056, 4, 32, False, "bf16"),
    (96, 64, 65536, 4, 64, False, "f32"),
    (2000, 8, 64, 4, 64, False, "f32"),
]


@pytest.mark.parametrize("M,d_out,d_in,bits,g,sym,y", GEMM)
def test_gemm_e4m3_matches_fp64(M, d_out, d_in, bits, g, sym, y):
    rng = np.random.default_rng(1000 * M + d_out + d_in + bits + g)
    L = Packed(rng, d_out, d_in, bits, g, sym)
    X, Xv, xs, xsv = _x(rng, M, d_in, "e4m3")
    buf, Y = _guarded(M, d_out, torch.float32 if y == "f32" else torch.bfloat16)
    assert L.gemm(X, xs, Y) is Y
    G.gptq_sync_status()
    L.check(Y, Xv, xsv)
    assert torch.all(buf[M * d_out:] == 7.0)
    first = Y.clone()
    L.gemm(X, xs, Y)
    assert torch.equal(first, Y)


# More tiles than SMs: blocks go from tile to tile, with odd and even counts of K tiles, groups that end
# inside one, and zero points that change with the group, with the tile or never.
GEMM_MANY = [
    (2100, 1288, 96, 3, -1, False, "f32"),
    (2100, 1288, 160, 4, 32, False, "bf16"),
    (2100, 1288, 384, 4, 128, False, "f32"),
    (2100, 1288, 640, 4, -1, False, "f32"),
    (2100, 1288, 896, 2, 64, True, "bf16"),
    (2100, 1288, 2176, 4, 128, False, "f32"),
    (2100, 1288, 1152, 4, -1, True, "f32"),
    (40, 20488, 640, 4, 128, False, "f32"),
]


@pytest.mark.parametrize("M,d_out,d_in,bits,g,sym,y", GEMM_MANY)
def test_gemm_e4m3_many_tiles(M, d_out, d_in, bits, g, sym, y):
    test_gemm_e4m3_matches_fp64(M, d_out, d_in, bits, g, sym, y)


@pytest.mark.parametrize("bits,act", [(4, 0), (3, 0), (8, 0), (4, 1)])
def test_gemv_extreme_codes_scales_and_nonfinite_rows(bits, act):
    rng = np.random.default_rng(bits + act)
    M, d_out, d_in, g = 5, 72, 256, 64
    L = Packed(rng, d_out, d_in, bits, g, False, act)
    zeros = rng.choice([0, (1 << bits) - 1], size=(L.ng, d_out))       # |q - z| up to 2^bits - 1
    codes = rng.choice([0, (1 << bits) - 1], size=(d_out, d_in))
    sc = rng.choice([0.0, 2.0 ** -24, 6e-8, 65504.0, 1.0], size=(L.ng, d_out)).astype(np.float16)
    qw, qz = O.pack_qweight(codes, bits), O.pack_qzeros(zeros, bits)
    L.qw, L.qz, L.sc = U_.t(qw), U_.t(qz), U_.t(sc)
    L.What = O.dequant_packed(qw, sc, qz, d_out, d_in, bits, g, False, None if L.gi is None else L.gi.cpu().numpy())
    X, Xv, _, _ = _x(rng, M, d_in, "bf16")
    X[1, 17], X[3, 255] = float("nan"), float("inf")
    Y = torch.empty((M, d_out), device=U_.dev())
    L.gemv(X, Y)
    fine = [0, 2, 4]
    L.check(Y[fine], Xv[fine])
    assert torch.isnan(Y[1]).all()
    weighted = torch.from_numpy(L.What[:, 255] != 0)
    assert not torch.isfinite(Y[3].cpu()[weighted]).any()


def test_gemm_e4m3_nonfinite_rows_stay_apart():
    rng = np.random.default_rng(5)
    M, d_out, d_in = 150, 136, 320
    L = Packed(rng, d_out, d_in, 4, 64, False)
    X, Xv, xs, xsv = _x(rng, M, d_in, "e4m3")
    X[7, 3] = float("nan")
    xs[149] = float("inf")
    xs[20] = 0.0
    xsv[20] = 0.0
    Y = torch.empty((M, d_out), device=U_.dev())
    L.gemm(X, xs, Y)
    fine = [m for m in range(M) if m not in (7, 149)]
    L.check(Y[fine], Xv[fine], xsv[fine])
    assert torch.isnan(Y[7]).all()
    assert not torch.isfinite(Y[149]).any()
    assert torch.all(Y[20] == 0)


def test_gemv_reports_a_group_index_out_of_range():
    rng = np.random.default_rng(6)
    L = Packed(rng, 16, 64, 4, 16, False, 1)
    X, _, _, _ = _x(rng, 1, 64, "bf16")
    Y = torch.empty((1, 16), device=U_.dev())
    for bad in (4, -1):
        good = int(L.gi[9])
        L.gi[9] = bad
        L.gemv(X, Y)
        with pytest.raises(G.GPTQError) as e:
            G.gptq_sync_status()
        assert e.value.status == G.GPTQ_ERR_INVALID_ARG
        L.gi[9] = good
    L.gemv(X, Y)
    G.gptq_sync_status()


def test_products_agree_with_each_other():
    # the few-token and the many-token forms on the same e4m3 rows
    rng = np.random.default_rng(8)
    L = Packed(rng, 264, 512, 4, 128, False)
    X, Xv, xs, xsv = _x(rng, 64, 512, "e4m3")
    A, B = torch.empty((64, 264), device=U_.dev()), torch.empty((64, 264), device=U_.dev())
    L.gemv(X, A, xs)
    L.gemm(X, xs, B)
    L.check(A, Xv, xsv)
    L.check(B, Xv, xsv)


# ---------------------------------------------------------------------------------------- rows

def _rows_reference(h, w, eps):
    d = h.shape[1]
    y = h if w is None else h * w / np.sqrt(np.sum(h * h, axis=1, keepdims=True) / d + eps)
    return y, np.max(np.abs(y), axis=1) / 448.0


def _check_rows(X8, xs, y, scale, d):
    got = xs.double().cpu().numpy()
    rel = ((d / 8 + 32) / 2 + 8) * 2.0 ** -24
    assert np.all(np.abs(got - scale) <= rel * scale), float(np.max(np.abs(got - scale) / np.maximum(scale, 1e-300)))
    v = y / np.where(scale == 0, 1.0, scale)[:, None]
    tol = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 8 * 2.0 ** -24 * np.abs(v)
    assert np.all(np.abs(X8.double().cpu().numpy() - v) <= tol)


ROWS = [(1, 8), (3, 24), (2, 1000), (7, 2048), (5, 4096), (150, 136), (3, 11008), (2, 32768), (2, 65536), (1000, 64)]


def _tensor(a, dtype):
    if dtype == "bf16":
        return _bf16(a)
    a = np.ascontiguousarray(a, dtype=np.float32)
    return U_.t(a), a.astype(np.float64)


@pytest.mark.parametrize("xt,wt,res", [("bf16", "bf16", True), ("bf16", "f32", False), ("f32", "bf16", True),
                                       ("f32", "f32", False), ("bf16", "f32", True)])
@pytest.mark.parametrize("M,d", ROWS)
def test_rms_norm_e4m3_matches_fp64(M, d, xt, wt, res):
    rng = np.random.default_rng(M + d)
    X, Xv = _tensor(_activations(rng, M, d), xt)
    w, wv = _tensor(1 + 0.2 * rng.standard_normal(d), wt)
    R, Rv = _tensor(4 * rng.standard_normal((M, d)), xt) if res else (None, 0.0)
    X8 = torch.zeros((M * d + 64,), dtype=torch.uint8, device=U_.dev()).fill_(0x55)
    xs = torch.full((M + 8,), 7.0, device=U_.dev())
    out = X8[:M * d].view(M, d).view(torch.float8_e4m3fn)
    R2 = torch.empty_like(X) if res else None
    keep = (X.clone(), None if R is None else R.clone())
    G.gptq_rms_norm_e4m3(X, w, out, xs[:M], R, R2, 1e-5)
    G.gptq_sync_status()
    h = Xv + Rv
    y, scale = _rows_reference(h, wv, 1e-5)
    _check_rows(out, xs[:M], y, scale, d)
    assert torch.all(X8[M * d:] == 0x55) and torch.all(xs[M:] == 7.0)
    assert torch.equal(X, keep[0])
    if res:
        assert torch.equal(R, keep[1])
        got = R2.double().cpu().numpy()
        assert np.all(np.abs(got - h) <= (2.0 ** -8 if xt == "bf16" else 0) * np.abs(h) + 2.0 ** -24 * np.abs(h))
        # in place over the residual, and over X: the same bits
        for into in (R, X):
            A, B = torch.empty_like(out), torch.empty_like(xs[:M])
            x, r = X.clone(), R.clone()
            G.gptq_rms_norm_e4m3(x, w, A, B, r, r if into is R else x, 1e-5)
            assert torch.equal(A.view(torch.uint8), out.view(torch.uint8)) and torch.equal(B, xs[:M])
            assert torch.equal(r if into is R else x, R2)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("M,d", ROWS)
def test_quantize_e4m3_matches_fp64(M, d, xt):
    rng = np.random.default_rng(M + d + 1)
    X, Xv = _tensor(_activations(rng, M, d), xt)
    X8, xs = torch.empty((M, d), dtype=torch.float8_e4m3fn, device=U_.dev()), torch.empty(M, device=U_.dev())
    G.gptq_quantize_e4m3(X, X8, xs)
    y, scale = _rows_reference(Xv, None, 0.0)
    _check_rows(X8, xs, y, scale, d)


@pytest.mark.parametrize("M,d", [(3, 64), (40, 1024), (500, 4096), (400, 8200), (5, 40000)])
def test_quantize_e4m3_boundaries_between_codes(M, d):
    # A bf16 v has 8 significant bits, and so has the row's maximum a; the boundary m between two codes
    # has 5.  So 448 v - m a is a multiple of 2^-16 of its terms or 0: the fp64 quotient lies on the
    # boundary exactly or far from it in units of fp32, and the codes are the same, ties to even.
    rng = np.random.default_rng(M + d + 3)
    X, Xv = _tensor(_activations(rng, M, d), "bf16")
    X8, xs = torch.empty((M, d), dtype=torch.float8_e4m3fn, device=U_.dev()), torch.empty(M, device=U_.dev())
    G.gptq_quantize_e4m3(X, X8, xs)
    q = 448.0 * Xv / np.max(np.abs(Xv), axis=1, keepdims=True)
    want = torch.from_numpy(q.astype(np.float32)).to(torch.float8_e4m3fn)
    assert torch.equal(X8.cpu().float(), want.float())


@pytest.mark.parametrize("d", [64, 8192, 65536])
def test_rows_special_values(d):
    rng = np.random.default_rng(d)
    a = rng.standard_normal((8, d)).astype(np.float32)
    a[0] = 0.0                                   # an empty row
    a[1] *= 1e-37                                # 448 / max overflows fp32 without care
    a[2] = 0.0
    a[2, d - 1] = -3.0                           # one value
    a[3, 5] = np.nan
    a[4, d // 2] = np.inf
    a[5] *= 1e15
    a[6, :] = 0.25                               # all equal: every code is 448
    X = U_.t(a)
    w = torch.ones(d, device=U_.dev())
    for norm in (True, False):
        X8, xs = torch.empty((8, d), dtype=torch.float8_e4m3fn, device=U_.dev()), torch.empty(8, device=U_.dev())
        if norm:
            G.gptq_rms_norm_e4m3(X, w, X8, xs, eps=1e-6)
        else:
            G.gptq_quantize_e4m3(X, X8, xs)
        fine = [0, 2, 5, 6, 7] + ([] if norm else [1])
        y, scale = _rows_reference(a[fine].astype(np.float64), np.ones(d) if norm else None, 1e-6)
        _check_rows(X8[fine], xs[fine], y, scale, d)
        assert float(xs[0]) == 0.0 and torch.all(X8[0].float() == 0)
        assert torch.all(X8[6].float() == 448.0)
        assert not torch.isfinite(xs[3]) and not torch.isfinite(xs[4])
        if norm:   # the codes do not depend on the norm's factor: those of the row 1e-37 times smaller
            v = a[1].astype(np.float64) / np.abs(a[1].astype(np.float64)).max() * 448
            tol = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 8 * 2.0 ** -24 * np.abs(v)
            assert np.all(np.abs(X8[1].double().cpu().numpy() - v) <= tol)


# ------------------------------------------------------------------------------------ together

def _block(rng, d, f, act=0):
    return dict(w=_bf16(1 + 0.2 * rng.standard_normal(d))[0], up=Packed(rng, f, d, 4, 128, False),
                down=Packed(rng, d, f, 3, 64, True), head=Packed(rng, 77, d, 4, 128, False, act))


def _forward(b, X, R, out, stream=None):
    """norm + residual -> up product -> e4m3 -> down product -> head on bf16 rows, all into out's buffers."""
    few = X.shape[0] <= 16
    G.gptq_rms_norm_e4m3(X, b["w"], out["X8"], out["xs"], R, out["R2"], 1e-6, stream)
    if few:
        b["up"].gemv(out["X8"], out["up"], out["xs"], stream)
    else:
        b["up"].gemm(out["X8"], out["xs"], out["up"], stream)
    G.gptq_quantize_e4m3(out["up"], out["U8"], out["us"], stream)
    b["down"].gemm(out["U8"], out["us"], out["down"], stream)
    b["head"].gemv(out["down"][:64], out["head"], None, stream)


def _buffers(M, d, f):
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device=U_.dev())
    return dict(X8=e(M, d, t=torch.float8_e4m3fn), xs=e(M, t=torch.float32), R2=e(M, d), up=e(M, f),
                U8=e(M, f, t=torch.float8_e4m3fn), us=e(M, t=torch.float32), down=e(M, d),
                head=e(min(M, 64), 77, t=torch.float32))


def _check_forward(b, X, R, out):
    """Each stage against fp64 on the stage's own stored inputs."""
    f64 = lambda t: t.double().cpu().numpy()
    y, scale = _rows_reference(f64(X) + f64(R), f64(b["w"]), 1e-6)
    _check_rows(out["X8"], out["xs"], y, scale, X.shape[1])
    b["up"].check(out["up"], f64(out["X8"]), f64(out["xs"]))
    y, scale = _rows_reference(f64(out["up"]), None, 0.0)
    _check_rows(out["U8"], out["us"], y, scale, out["up"].shape[1])
    b["down"].check(out["down"], f64(out["U8"]), f64(out["us"]))
    b["head"].check(out["head"], f64(out["down"][:64]))


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_a_block_of_layers_runs_together(M):
    rng = np.random.default_rng(M)
    d, f = 256, 640
    b = _block(rng, d, f, act=1)
    X, R = _bf16(_activations(rng, M, d))[0], _bf16(rng.standard_normal((M, d)))[0]
    out = _buffers(M, d, f)
    _forward(b, X, R, out)
    G.gptq_sync_status()
    _check_forward(b, X, R, out)


@pytest.mark.parametrize("M", [3, 200])
def test_captured_and_replayed_with_new_inputs(M):
    rng = np.random.default_rng(70 + M)
    d, f = 256, 384
    b = _block(rng, d, f)
    X, R = _bf16(_activations(rng, M, d))[0], _bf16(rng.standard_normal((M, d)))[0]
    out = _buffers(M, d, f)
    _forward(b, X, R, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _forward(b, X, R, out)
    for k in range(3):
        X.copy_(_bf16(_activations(rng, M, d))[0])
        for t in out.values():
            t.view(torch.uint8).fill_(0x7F)
        graph.replay()
        torch.cuda.synchronize()
        _check_forward(b, X, R, out)


def test_two_graphs_and_two_streams_do_not_share_anything():
    rng = np.random.default_rng(12)
    d, f, M = 256, 384, 24
    b = _block(rng, d, f)
    jobs = []
    for k in range(2):
        X, R = _bf16(_activations(rng, M, d))[0], _bf16(rng.standard_normal((M, d)))[0]
        out = _buffers(M, d, f)
        _forward(b, X, R, out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _forward(b, X, R, out)
        jobs.append((g, torch.cuda.Stream(), X, R, out))
    for _, _, _, _, out in jobs:
        for t in out.values():
            t.view(torch.uint8).fill_(0x7F)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st, *_ in jobs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, _, X, R, out in jobs:
        _check_forward(b, X, R, out)


def test_side_stream_argument_orders_the_calls():
    rng = np.random.default_rng(13)
    d, f, M = 256, 384, 8
    b = _block(rng, d, f)
    X, R = _bf16(_activations(rng, M, d))[0], _bf16(rng.standard_normal((M, d)))[0]
    out = _buffers(M, d, f)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    _forward(b, X, R, out, st)
    st.synchronize()
    _check_forward(b, X, R, out)


def test_calls_from_two_threads():
    rng = np.random.default_rng(14)
    d, f, M = 256, 384, 70
    b = _block(rng, d, f)
    jobs = []
    for k in range(2):
        X, R = _bf16(_activations(rng, M, d))[0], _bf16(rng.standard_normal((M, d)))[0]
        jobs.append((X, R, _buffers(M, d, f), torch.cuda.Stream()))
    torch.cuda.synchronize()
    errors = []

    def work(X, R, out, st):
        try:
            with torch.cuda.stream(st):
                for _ in range(50):
                    _forward(b, X, R, out)
            st.synchronize()
        except Exception as e:   # reported by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for X, R, out, _ in jobs:
        _check_forward(b, X, R, out)


@pytest.mark.parametrize("act", [0, 1])
def test_a_layer_quantized_here_serves_its_tokens(act):
    # quantizer's own output (natural and activation order) through the decoding product
    rng = np.random.default_rng(15 + act)
    d_out, d_in, n = 192, 384, 256
    X, Xv = _bf16(_activations(rng, n, d_in))
    q = G.quantize_layer(U_.t((0.02 * rng.standard_normal((d_out, d_in))).astype(np.float32)), X, 4, 64, False,
                         desc_act=act)
    cfg = G.make_config(4, 64, False, desc_act=act)
    Y = torch.empty((5, d_out), device=U_.dev())
    G.gptq_dequant_gemv(X[:5], q.qweight, q.scales, q.qzeros, d_out, d_in, cfg, Y, g_idx=q.g_idx)
    G.gptq_sync_status()
    np32 = lambda t: t.cpu().numpy()
    What = O.dequant_packed(np32(q.qweight), np32(q.scales), np32(q.qzeros), d_out, d_in, 4, 64, False,
                            None if q.g_idx is None else np32(q.g_idx))
    S = np.abs(Xv[:5]) @ np.abs(What).T
    assert np.all(np.abs(Y.double().cpu().numpy() - Xv[:5] @ What.T) <= (d_in / 8 + 6 + 32) * 2.0 ** -23 * S)
