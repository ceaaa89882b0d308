"""The first call of an operator in a process may be a captured one: whatever a kernel needs set up, and
whatever the driver loads late, is done without disturbing the capture."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
import numpy as np
import torch
from tests import gpu_util as U_
from tests.test_gpu_serving import Packed, _bf16, _e4m3
from post_weight_quantization_14_b200 import gptq as G

op = sys.argv[1]
rng = np.random.default_rng(3)
M, d, n = 40, 512, 136
L = Packed(rng, n, d, 4, 128, False, 1 if op == "act" else 0)
X, Xv = _bf16(rng.standard_normal((M, d)))
I8, Iv = _e4m3(20 * rng.standard_normal((M, d)))
s = np.full(M, 0.5)
Is, w = U_.t(s.astype(np.float32)), _bf16(np.ones(d))[0]
R, R2 = X.clone(), torch.empty_like(X)
X8, xs = torch.empty((M, d), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(M, device="cuda")
Y = torch.empty((M, n), device="cuda")

def call():
    if op in ("gemv", "act"):
        L.gemv(X, Y)
    elif op == "gemm":
        L.gemm(I8, Is, Y)
    elif op == "norm":
        G.gptq_rms_norm_e4m3(X, w, X8, xs, R, R2)
    else:
        G.gptq_quantize_e4m3(X, X8, xs)

graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    call()
outputs = [Y] if op in ("gemv", "act", "gemm") else [X8, xs, R2]
for t in outputs:
    t.view(torch.uint8).fill_(0x7F)
graph.replay()
torch.cuda.synchronize()
G.gptq_sync_status()
if op in ("gemv", "act"):
    L.check(Y, Xv)
elif op == "gemm":
    L.check(Y, Iv, s)
got = [t.clone() for t in outputs]
call()
torch.cuda.synchronize()
for a, t in zip(got, outputs):
    assert torch.equal(a.view(torch.uint8), t.view(torch.uint8))
print("same")
"""


@pytest.mark.parametrize("op", ["gemv", "act", "gemm", "norm", "quant"])
def test_first_call_is_captured(cuda_dev, op):
    r = subprocess.run([sys.executable, "-c", PROGRAM, op], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout[-2000:] + r.stderr[-3000:]
