"""Calls under a context that the caller made with the driver's own interface, as a C
program may: they run in it and leave it current.  In a process of its own, in which
nothing else uses the GPU."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = r"""
import ctypes, math, sys
import torch  # for host arithmetic alone
from io_aware_exact_12_gb300 import build
build.build()
import io_aware_exact_12_gb300 as p
cu = ctypes.CDLL("libcuda.so.1")

def ok(rc):
    assert rc == 0, rc

ok(cu.cuInit(0))
dev, own, now = ctypes.c_int(), ctypes.c_void_p(), ctypes.c_void_p()
ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
ok(cu.cuCtxCreate_v2(ctypes.byref(own), 0, dev))

def up(t):
    at = ctypes.c_uint64()
    n = t.numel() * t.element_size()
    ok(cu.cuMemAlloc_v2(ctypes.byref(at), ctypes.c_size_t(n)))
    ok(cu.cuMemcpyHtoD_v2(at, ctypes.c_void_p(t.data_ptr()), ctypes.c_size_t(n)))
    return at.value

def down(at, t):
    ok(cu.cuMemcpyDtoH_v2(ctypes.c_void_p(t.data_ptr()), ctypes.c_uint64(at), ctypes.c_size_t(t.numel() * t.element_size())))
    return t

g = torch.Generator().manual_seed(1)
B, H, N, d = 1, 2, 200, 64
q, k, v = (torch.randn((B, H, N, d), generator=g).to(torch.bfloat16) for _ in range(3))
o, lse = torch.zeros_like(q), torch.zeros((B, H, N))
pq, pk, pv, po, pl = (up(t) for t in (q, k, v, o, lse))
bhnd = lambda x: ctypes.byref(p._BhndStruct(x, H * N * d, N * d, d))
L = p.lib()
ok(L.attn_sync_status(None))
ok(cu.cuCtxGetCurrent(ctypes.byref(now)))
assert now.value == own.value
i, j = torch.arange(N)[:, None], torch.arange(N)
for window in (N, 30):
    if window == N:
        ok(L.attn_fwd(pq, pk, pv, po, pl, B, H, N, d, 0.125, 1, None))
    else:
        ok(L.attn_fwd_window(bhnd(pq), bhnd(pk), bhnd(pv), bhnd(po), pl, B, H, H, N, N, d, window, 0, 0.125, 0, None))
    ok(L.attn_sync_status(None))
    ok(cu.cuCtxGetCurrent(ctypes.byref(now)))
    assert now.value == own.value
    s = (0.125 * (q.double() @ k.double().mT)).masked_fill((j > i) | (j <= i - window), -math.inf)
    w = torch.softmax(s, -1)
    # weights and results rounded to bf16, 2^-8 each way; fp32 parts below a tenth of that
    tol = 2.0 ** -8 * (w @ v.double()).abs() + 2.2 * 2.0 ** -8 * (w @ v.double().abs())
    assert ((down(po, o).double() - w @ v.double()).abs() <= tol).all()
print("in its own context")
"""


def test_a_context_of_the_callers_own():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "in its own context" in r.stdout, r.stdout + r.stderr
