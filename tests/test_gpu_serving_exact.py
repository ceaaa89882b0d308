"""The products where every sum is exact: x is 1 or -1, the scales and the tokens' factors are powers of two,
and sum |q - z| s stays below 2^24, so each partial sum, in whatever order and however a tensor instruction
rounds, is a whole number that fp32 holds.  Y has to equal the fp64 product bit for bit: one column left out
or taken twice, one group's scale or zero point looked up wrongly, at the end of a row, of a group or of a
part of a split row, changes it by one at least, however long the row is."""

import numpy as np
import pytest
import torch

from oracle import gptq_oracle as O
from post_weight_quantization_14_b200 import gptq as G

from . import gpu_util as U_
from .test_gpu_serving import Packed, _bf16, _e4m3, _guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_cuda(cuda_dev):
    yield


def _layer(rng, d_out, d_in, bits, g, sym, act=0):
    L = Packed(rng, d_out, d_in, bits, g, sym, act)
    top = (1 << bits) - 1
    exponents = int(np.log2((1 << 24) / (d_in * top)))        # scales 1 .. 2^exponents keep the sums below 2^24
    assert exponents >= 0 and top * d_in < 1 << 24
    sc = np.exp2(rng.integers(0, min(exponents, 8) + 1, size=(L.ng, d_out))).astype(np.float16)
    codes = rng.integers(0, top + 1, size=(d_out, d_in))
    zeros = np.full((L.ng, d_out), 1 << (bits - 1)) if sym else rng.integers(0, top + 1, size=(L.ng, d_out))
    gi = np.arange(d_in) // (d_in if g == -1 else g) if L.gi is None else L.gi.cpu().numpy()
    # no weight is 0, so that every column counts
    codes = np.where(codes == zeros.T[:, gi], np.where(codes == 0, 1, codes - 1), codes)
    qw, qz = O.pack_qweight(codes, bits), None if sym else O.pack_qzeros(zeros, bits)
    L.qw, L.qz, L.sc = U_.t(qw), None if sym else U_.t(qz), U_.t(sc)
    L.What = O.dequant_packed(qw, sc, qz, d_out, d_in, bits, g, sym, None if L.gi is None else gi)
    assert np.all(L.What != 0)
    return L


def _tokens(rng, M, d_in, x):
    a = rng.choice([-1.0, 1.0], size=(M, d_in))
    if x == "bf16":
        return _bf16(a)[0], a, None, 1.0
    xs = np.exp2(rng.integers(-3, 4, size=M))
    return _e4m3(a)[0], a, U_.t(xs.astype(np.float32)), xs[:, None]


GEMV = [
    # M, d_out, d_in, bits, g, sym, act, x
    (3, 72, 65536, 2, 128, False, 0, "bf16"),
    (1, 1028, 65528, 4, -1, False, 0, "bf16"),
    (9, 40, 65512, 3, 64, False, 0, "e4m3"),      # the last group has 40 columns
    (20, 37, 32760, 8, 32, False, 0, "bf16"),     # odd rows: no TMA
    (33, 45, 65528, 4, 128, True, 0, "e4m3"),     # nor with 8 bytes past a multiple of 16
    (2, 260, 40008, 4, 16, False, 0, "e4m3"),
    (64, 132, 16392, 2, 16, True, 0, "bf16"),
    (8, 9600, 2056, 4, 128, False, 0, "bf16"),    # K not split
    (8, 20000, 1032, 3, -1, False, 0, "e4m3"),
    # activation order, the table in shared memory
    (64, 70, 16384, 4, 16, False, 1, "bf16"),
    (12, 45, 65536, 4, 128, False, 1, "e4m3"),
    (64, 33, 20480, 4, 16, False, 1, "e4m3"),     # 1280 groups: the largest table, beside the sums of 32 tokens
    (33, 45, 20488, 2, 128, False, 1, "bf16"),
    (1, 36, 65536, 3, 64, False, 2, "bf16"),
    (5, 39, 32760, 8, 32, False, 1, "e4m3"),
    (7, 4800, 2056, 4, 32, False, 1, "bf16"),     # K not split
    # more than 1280 groups: no table
    (3, 36, 32768, 4, 16, False, 1, "bf16"),
    (5, 131, 40008, 4, 16, False, 2, "e4m3"),
    (17, 133, 65536, 3, 32, False, 1, "bf16"),
    (8, 34, 40008, 3, 16, True, 1, "e4m3"),
    (9, 35, 65528, 2, 32, False, 1, "bf16"),
    (4, 64, 20488, 2, 16, False, 1, "e4m3"),
    (1, 33, 24584, 8, 16, False, 1, "bf16"),
    (2, 37, 24584, 8, 16, True, 1, "e4m3"),
]


@pytest.mark.parametrize("M,d_out,d_in,bits,g,sym,act,x", GEMV)
def test_gemv_exact_sums(M, d_out, d_in, bits, g, sym, act, x):
    rng = np.random.default_rng(M + d_out + d_in + bits)
    L = _layer(rng, d_out, d_in, bits, g, sym, act)
    X, Xv, xs, factor = _tokens(rng, M, d_in, x)
    buf, Y = _guarded(M, d_out, torch.float32)
    L.gemv(X, Y, xs)
    G.gptq_sync_status()
    assert np.array_equal(Y.double().cpu().numpy(), Xv @ L.What.T * factor)
    assert torch.all(buf[M * d_out:] == 7.0)


GEMM = [
    (96, 64, 65536, 4, 64, False),
    (70, 136, 65536, 4, -1, False),
    (130, 72, 32672, 3, 32, False),      # a last K tile of 32 columns
    (3, 24, 65504, 2, 32, True),
    (64, 264, 24576, 4, 128, False),
    (300, 264, 8192, 4, 128, False),
    (2100, 1288, 672, 4, 32, False),     # more tiles than SMs
    (2100, 1288, 1152, 4, -1, False),
    (200, 520, 4160, 2, 64, False),
]


@pytest.mark.parametrize("M,d_out,d_in,bits,g,sym", GEMM)
def test_gemm_e4m3_exact_sums(M, d_out, d_in, bits, g, sym):
    rng = np.random.default_rng(M + d_out + d_in + bits)
    L = _layer(rng, d_out, d_in, bits, g, sym)
    X, Xv, xs, factor = _tokens(rng, M, d_in, "e4m3")
    buf, Y = _guarded(M, d_out, torch.float32)
    L.gemm(X, xs, Y)
    G.gptq_sync_status()
    assert np.array_equal(Y.double().cpu().numpy(), Xv @ L.What.T * factor)
    assert torch.all(buf[M * d_out:] == 7.0)
