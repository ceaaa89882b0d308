"""The serving operators take their place in stream order whatever precedes them: a wait for a slow
producer in another stream, right behind a kernel of their own stream, eagerly and in a captured fork
and join.  Before each call the inputs hold other values, so a call that starts early is seen."""

import shutil

import numpy as np
import pytest
import torch

from post_weight_quantization_14_b200 import gptq as G

from . import gpu_util as U_
from .test_gpu_serving import Packed, _activations, _bf16, _e4m3, _x

pytestmark = pytest.mark.gpu

M, D, N = 24, 1024, 264
SLOW = 2_000_000   # clocks, about a millisecond


@pytest.fixture(autouse=True)
def _need_cuda(cuda_dev):
    yield


def _call(op, L, w, b):
    if op == "quant":
        G.gptq_quantize_e4m3(b["X"], b["X8"], b["xs"])
    elif op == "norm":
        G.gptq_rms_norm_e4m3(b["X"], w, b["X8"], b["xs"], b["R"], b["R2"])
    elif op == "gemv":
        L.gemv(b["X"], b["Y"])
    else:
        L.gemm(b["I8"], b["Is"], b["Y"])


def _buffers():
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device=U_.dev())
    return dict(X=e(M, D), R=e(M, D), I8=e(M, D, t=torch.float8_e4m3fn), Is=e(M, t=torch.float32),
                X8=e(M, D, t=torch.float8_e4m3fn), xs=e(M, t=torch.float32), R2=e(M, D), Y=e(M, N))


INPUTS, OUTPUTS = ("X", "R", "I8", "Is"), dict(quant=("X8", "xs"), norm=("X8", "xs", "R2"), gemv=("Y",), gemm=("Y",))


def _setup(op):
    rng = np.random.default_rng(len(op))
    L = Packed(rng, N, D, 4, 128, False)
    w = _bf16(1 + 0.2 * rng.standard_normal(D))[0]
    sets = [dict(X=_bf16(_activations(rng, M, D))[0], R=_bf16(rng.standard_normal((M, D)))[0],
                 I8=_e4m3(20 * rng.standard_normal((M, D)))[0], Is=U_.t(rng.uniform(0.01, 0.1, M).astype(np.float32)))
            for _ in range(4)]
    want = []
    for s in sets:
        b = _buffers()
        for k in INPUTS:
            b[k].copy_(s[k])
        torch.cuda.synchronize()
        _call(op, L, w, b)
        torch.cuda.synchronize()
        want.append({k: b[k].clone() for k in OUTPUTS[op]})
    return L, w, sets, want


def _same(b, want):
    for k, t in want.items():
        assert torch.equal(b[k].view(torch.uint8), t.view(torch.uint8)), k


def _produce(b, s):
    torch.cuda._sleep(SLOW)
    for k in INPUTS:
        b[k].copy_(s[k])


@pytest.mark.parametrize("op", list(OUTPUTS))
def test_behind_a_wait_for_another_stream(op):
    L, w, sets, want = _setup(op)
    b, side = _buffers(), torch.cuda.Stream()
    for k in INPUTS:
        b[k].copy_(sets[-1][k])
    for s, y in zip(sets, want):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _produce(b, s)
        b["X8"].view(torch.uint8).zero_()             # a kernel of the call's own stream, before the wait
        torch.cuda.current_stream().wait_stream(side)
        _call(op, L, w, b)
        torch.cuda.synchronize()
        _same(b, y)


@pytest.mark.parametrize("op", list(OUTPUTS))
def test_behind_a_join_of_captured_streams(op):
    L, w, sets, want = _setup(op)
    b, src, side = _buffers(), {k: t.clone() for k, t in sets[0].items()}, torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            _produce(b, src)
        b["X8"].view(torch.uint8).zero_()
        main.wait_stream(side)
        _call(op, L, w, b)
    for s, y in zip(sets, want):
        for k in INPUTS:
            b[k].copy_(sets[-1][k] if s is not sets[-1] else sets[0][k])
            src[k].copy_(s[k])
        graph.replay()
        torch.cuda.synchronize()
        _same(b, y)


def test_two_copies_of_the_library_in_one_process(tmp_path):
    # what one copy has set up for its kernels says nothing about the other's
    rng = np.random.default_rng(16)
    L = Packed(rng, 136, 512, 4, 128, False)
    A = Packed(rng, 136, 512, 4, 128, False, 1)
    X, Xv, xs, xsv = _x(rng, 70, 512, "e4m3")
    first = G.lib()
    try:
        for k in range(2):
            Y, Z, V = (torch.empty((m, 136), device=U_.dev()) for m in (70, 9, 9))
            L.gemm(X, xs, Y)
            L.gemv(X[:9], Z, xs[:9])
            A.gemv(X[:9], V, xs[:9])
            G.gptq_sync_status()
            L.check(Y, Xv, xsv)
            L.check(Z, Xv[:9], xsv[:9])
            A.check(V, Xv[:9], xsv[:9])
            if k == 0:
                copy = tmp_path / "libgptq_b200_copy.so"
                shutil.copy(G.LIB_PATH, copy)
                G._lib, path, G.LIB_PATH = None, G.LIB_PATH, str(copy)
                try:
                    assert G.lib() is not first
                finally:
                    G.LIB_PATH = path
    finally:
        G._lib = first
