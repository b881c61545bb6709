"""Calls from several host threads: a thread whose first call of all it is, and first calls at once."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import DT, gen, rand

pytestmark = pytest.mark.gpu


def calls():
    """One call of each kind that encodes tensor maps, with its output."""
    g = gen(111)
    for dtype, M, K, O in (("bf16", 40, 128, 72), ("bf16", 5000, 128, 72), ("bf16", 5000, 1800, 72), ("f32", 40, 128, 72)):
        x, w = rand(g, 1, M, K, dtype=dtype), rand(g, O, K, dtype=dtype)
        y = torch.zeros(1, M, O, dtype=DT[dtype], device="cuda")
        desc = mcs.linear_desc(1, M, K, O, DT[dtype])
        yield y, lambda s, d=desc, x=x, w=w, y=y: mcs.mcs_linear(d, x, w, None, None, None, y, stream=s)
    q, k, v = (rand(g, 1, 2, 300, 64, dtype="bf16") for _ in range(3))
    o, desc = torch.zeros_like(q), mcs.make_desc(1, 2, 300, 64, 64, torch.bfloat16)
    yield o, lambda s: mcs.mcs_dense_attn(desc, q, k, v, o, None, stream=s)


def test_first_call_of_a_thread():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    stream = torch.cuda.Stream()
    for out, call in calls():
        call(stream)
        stream.synchronize()
        want = out.clone()
        out.zero_()
        torch.cuda.synchronize()
        failed = []

        def work():
            try:
                call(stream)
            except Exception as e:
                failed.append(e)

        t = threading.Thread(target=work)
        t.start()
        t.join()
        assert not failed, failed
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    mcs.mcs_check_status()


CONTEXT = """
import ctypes, threading, torch
from sparse_attention_diffusion_gb300 import mcs
mcs.load()
cu = ctypes.CDLL("libcuda.so.1")
x, w = torch.randn(1, 40, 128).bfloat16().cuda(), torch.randn(72, 128).bfloat16().cuda()
y = torch.zeros(1, 40, 72, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
before, after = ctypes.c_void_p(), ctypes.c_void_p()
cu.cuCtxGetCurrent(ctypes.byref(before))
mcs.mcs_linear(mcs.linear_desc(1, 40, 128, 72, torch.bfloat16), x, w, None, None, None, y)
cu.cuCtxGetCurrent(ctypes.byref(after))
assert before.value and before.value == after.value
failed = []
def work():
    # a thread with no context of its own gets the device's, and keeps it
    now = ctypes.c_void_p()
    cu.cuCtxGetCurrent(ctypes.byref(now))
    if now.value:
        failed.append("a new thread has a context")
    mcs.mcs_linear(mcs.linear_desc(1, 40, 128, 72, torch.bfloat16), x, w, None, None, None, y, stream=torch.cuda.default_stream())
    cu.cuCtxGetCurrent(ctypes.byref(now))
    if now.value != before.value:
        failed.append("another context")
t = threading.Thread(target=work)
t.start()
t.join()
assert not failed, failed
torch.cuda.synchronize()
mcs.mcs_check_status()
"""


def test_a_context_that_is_there_stays():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    mcs.load(build_if_missing=True)
    r = subprocess.run([sys.executable, "-c", CONTEXT], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


THREADS = """
import threading, torch
from sparse_attention_diffusion_gb300 import mcs
mcs.load()
torch.cuda.init()
n = 8
jobs = []
for i in range(n):
    g = torch.Generator().manual_seed(i)
    x, w = torch.randn(1, 100 + 900 * i, 256, generator=g).bfloat16().cuda(), torch.randn(200, 256, generator=g).bfloat16().cuda()
    jobs.append((x, w, torch.empty(1, x.shape[1], 200, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream()))
torch.cuda.synchronize()
start, failed = threading.Barrier(n), []
def work(x, w, y, s):
    start.wait()
    try:
        for _ in range(20):
            mcs.mcs_linear(mcs.linear_desc(1, x.shape[1], 256, 200, torch.bfloat16), x, w, None, None, None, y, stream=s)
    except Exception as e:
        failed.append(e)
threads = [threading.Thread(target=work, args=j) for j in jobs]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
mcs.mcs_check_status()
assert not failed, failed
for x, w, y, _ in jobs:
    assert float((y.double() - x.double() @ w.double().t()).abs().max()) < 1.0
"""


def test_first_calls_of_several_threads():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    mcs.load(build_if_missing=True)
    r = subprocess.run([sys.executable, "-c", THREADS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
