"""Host-side checks, without a GPU, of the entry points that serve a quantized layer: every
argument that they refuse is refused before anything is enqueued, by the library for raw
addresses and by the binding for tensors."""

import ctypes

import pytest
import torch

from post_weight_quantization_14_b200 import gptq as G


def _fake(n=1, off=0):
    # host addresses are never dereferenced: validation fails before any CUDA call
    return ctypes.c_void_p(0x10000 * n + off)


def _gemv(cfg, M=4, d_out=64, d_in=128, X=_fake(1), xt=G.GPTQ_BF16, xs=None, qw=_fake(2), sc=_fake(3), qz=_fake(4),
          gi=None, Y=_fake(5), yt=G.GPTQ_F32):
    return G.lib().gptq_dequant_gemv(X, xt, xs, M, qw, sc, qz, gi, d_out, d_in, ctypes.byref(cfg), Y, yt, None)


def _gemm(cfg, M=4, d_out=64, d_in=128, X=_fake(1), xs=_fake(6), qw=_fake(2), sc=_fake(3), qz=_fake(4), Y=_fake(5),
          yt=G.GPTQ_F32):
    return G.lib().gptq_dequant_gemm_e4m3(X, xs, M, qw, sc, qz, d_out, d_in, ctypes.byref(cfg), Y, yt, None)


SHARED = [dict(M=0), dict(M=-1), dict(d_out=0), dict(d_in=0), dict(d_in=60), dict(d_in=65544), dict(X=None),
          dict(qw=None), dict(sc=None), dict(qz=None), dict(Y=None), dict(yt=G.GPTQ_E4M3), dict(yt=7),
          dict(qw=_fake(2, 4)), dict(sc=_fake(3, 2)), dict(qz=_fake(4, 8))]


@pytest.mark.parametrize("kw", SHARED + [
    dict(M=G.GPTQ_GEMV_MAX_M + 1), dict(xt=G.GPTQ_F32), dict(xt=9), dict(xs=_fake(6)), dict(xt=G.GPTQ_E4M3),
    dict(gi=_fake(7)), dict(X=_fake(1, 8)), dict(X=_fake(1, 4), xt=G.GPTQ_E4M3, xs=_fake(6)), dict(Y=_fake(5, 2)),
    dict(Y=_fake(5, 1), yt=G.GPTQ_BF16), dict(xt=G.GPTQ_E4M3, xs=_fake(6, 2))])
def test_gemv_refuses(kw):
    assert _gemv(G.make_config(4, 128, False), **kw) == G.GPTQ_ERR_INVALID_ARG
    assert G.lib().gptq_last_error()


def test_gemv_refuses_configurations():
    assert _gemv(G.make_config(5, 128, False)) == G.GPTQ_ERR_INVALID_ARG
    assert _gemv(G.make_config(4, 256, False)) == G.GPTQ_ERR_INVALID_ARG
    assert _gemv(G.make_config(4, 128, True)) == G.GPTQ_ERR_INVALID_ARG              # symmetric has no qzeros
    assert _gemv(G.make_config(4, 128, False, desc_act=1)) == G.GPTQ_ERR_INVALID_ARG  # needs g_idx
    assert _gemv(G.make_config(4, 128, False, desc_act=1), gi=_fake(7, 2)) == G.GPTQ_ERR_INVALID_ARG
    assert G.lib().gptq_dequant_gemv(_fake(), 0, None, 1, _fake(), _fake(), _fake(), None, 8, 64, None, _fake(), 1,
                                     None) == G.GPTQ_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SHARED + [dict(xs=None), dict(xs=_fake(6, 2)), dict(d_in=104), dict(d_out=60),
                                         dict(X=_fake(1, 8)), dict(Y=_fake(5, 4)), dict(M=(1 << 30) + 1)])
def test_gemm_e4m3_refuses(kw):
    assert _gemm(G.make_config(4, -1, False), **kw) == G.GPTQ_ERR_INVALID_ARG
    assert G.lib().gptq_last_error()


def test_gemm_e4m3_unsupported_configurations():
    assert _gemm(G.make_config(8, 128, False)) == G.GPTQ_ERR_UNSUPPORTED     # 8-bit q - z is not an e4m3 value
    assert _gemm(G.make_config(4, 16, False)) == G.GPTQ_ERR_UNSUPPORTED
    assert _gemm(G.make_config(4, 128, False), d_in=160) == G.GPTQ_ERR_UNSUPPORTED
    assert _gemm(G.make_config(4, 128, False, desc_act=2)) == G.GPTQ_ERR_UNSUPPORTED
    assert _gemm(G.make_config(6, 128, False)) == G.GPTQ_ERR_INVALID_ARG


def test_rows_refuse():
    norm = lambda X=_fake(1), R=None, xt=0, w=_fake(2), wt=0, M=4, d=64, eps=1e-6, X8=_fake(3), xs=_fake(4), R2=None: \
        G.lib().gptq_rms_norm_e4m3(X, R, xt, w, wt, M, d, eps, X8, xs, R2, None)
    quant = lambda X=_fake(1), xt=0, M=4, d=64, X8=_fake(3), xs=_fake(4): \
        G.lib().gptq_quantize_e4m3(X, xt, M, d, X8, xs, None)
    for kw in (dict(X=None), dict(X8=None), dict(xs=None), dict(xt=2), dict(M=0), dict(M=(1 << 30) + 1), dict(d=0),
               dict(d=60), dict(d=65544), dict(X=_fake(1, 8)), dict(X8=_fake(3, 4)), dict(xs=_fake(4, 2))):
        assert norm(**kw) == G.GPTQ_ERR_INVALID_ARG, kw
        assert quant(**kw) == G.GPTQ_ERR_INVALID_ARG, kw
    for kw in (dict(w=None), dict(wt=2), dict(R=_fake(5)), dict(R2=_fake(5)), dict(R=_fake(5, 8), R2=_fake(6)),
               dict(R=_fake(5), R2=_fake(6, 4)), dict(w=_fake(2, 8)), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf"))):
        assert norm(**kw) == G.GPTQ_ERR_INVALID_ARG, kw


def test_binding_refuses_tensors_before_any_call():
    M, d_out, d_in = 4, 64, 128
    cfg = G.make_config(4, 128, False)
    X = torch.zeros((M, d_in), dtype=torch.bfloat16)
    X8, xs = torch.zeros((M, d_in), dtype=torch.float8_e4m3fn), torch.zeros(M)
    qw, sc = torch.zeros((16, d_out), dtype=torch.int32), torch.zeros((1, d_out), dtype=torch.float16)
    qz, Y = torch.zeros((1, 8), dtype=torch.int32), torch.zeros((M, d_out))
    gi = torch.zeros(d_in, dtype=torch.int32)
    act = G.make_config(4, 128, False, desc_act=1)

    def gemv(X=X, qw=qw, sc=sc, qz=qz, cfg=cfg, Y=Y, xs=None, gi=None):
        G.gptq_dequant_gemv(X, qw, sc, qz, d_out, d_in, cfg, Y, xs, gi)

    for kw in (dict(X=X.float()), dict(X=X[:, :64]), dict(X=X[0]), dict(Y=Y.half()), dict(Y=Y[:2]), dict(Y=Y.t()),
               dict(X=X8), dict(xs=xs), dict(X=X8, xs=xs[:2]), dict(X=X8, xs=xs.double()), dict(gi=gi), dict(cfg=act),
               dict(cfg=act, gi=gi.long()), dict(cfg=act, gi=gi[:8]), dict(qw=qw[:8]), dict(sc=sc.float()),
               dict(qz=None), dict()):   # the last: tensors of the host
        with pytest.raises(ValueError):
            gemv(**kw)

    def gemm(X8=X8, xs=xs, qw=qw, Y=Y):
        G.gptq_dequant_gemm_e4m3(X8, xs, qw, sc, qz, d_out, d_in, cfg, Y)

    for kw in (dict(X8=X), dict(X8=X8[:, :64]), dict(X8=X8[0]), dict(xs=xs[:1]), dict(xs=xs.half()), dict(qw=qw.long()),
               dict(Y=Y.double()), dict(Y=Y[:, :8]), dict()):
        with pytest.raises(ValueError):
            gemm(**kw)

    w = torch.ones(d_in)

    def norm(X=X, w=w, X8=X8, xs=xs, R=None, R2=None):
        G.gptq_rms_norm_e4m3(X, w, X8, xs, R, R2)

    for kw in (dict(X=X.half()), dict(X=X[0]), dict(w=w[:8]), dict(w=w.half()), dict(X8=X8[:2]), dict(X8=X),
               dict(xs=xs[:2]), dict(R=X), dict(R2=X), dict(R=X.float(), R2=X.float()), dict(R=X, R2=X.float()),
               dict(R=X[:2], R2=X[:2]), dict()):
        with pytest.raises(ValueError):
            norm(**kw)
    for a in ((X.half(), X8, xs), (X[0], X8, xs), (X, X8[:, :8], xs), (X, X8, xs[:1]), (X, X8, xs)):
        with pytest.raises(ValueError):
            G.gptq_quantize_e4m3(*a)
