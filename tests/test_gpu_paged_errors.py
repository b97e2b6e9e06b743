"""A launch that fails is reported by its own call and by no other."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A stream whose capture has been invalidated refuses every launch: a failure on the host alone.
_SCRIPT = r"""
import ctypes, sys
sys.path[:0] = [%(root)r, %(root)r + "/tests"]
import torch
from test_gpu_paged import Cache, _append
from test_gpu_prep import _freq
c = Cache([100, 90, 140], 4, 2, 64, 16, "bf16", 20, seed=1, prefix=64)
dma = c.dma
B, N, d = 1, 40, 64
p = dma.make_params(B, 4, 2, N, d, 1)
g = lambda *s: torch.randn(*s, device="cuda").bfloat16()
q, k, Q, K = g(B, N, 4, d), g(B, N, 2, d), g(B, 4, N, d), g(B, 2, N, d)
w, f32 = g(d), lambda: torch.empty(d, device="cuda")
r = dma.make_prep(_freq(torch, 64), w, w)
ws = dma.alloc_prep_workspace(p, r)
a = _append(c, None, 64, False, True)
O, L = torch.empty_like(c.normal(3, 4, 64).to(c.t)), torch.empty(3, 4, device="cuda")
Qd = c.normal(3, 4, 64).to(c.t)
calls = {
    "prep": lambda s: dma.prep(p, r, q, k, None, Q, K, None, stream=s),
    "prep_bwd": lambda s: dma.prep_bwd(p, r, q, k, Q, K, None, None, g0, k0, None, w0, w1, ws, stream=s),
    "append": lambda s: dma.paged_append(c.p, c.c, a["r"], a["q"], a["k"], a["v"], a["Delta"], a["A"], a["Q"], c.ws, stream=s),
    "topk": lambda s: dma.paged_topk(c.p, c.c, c.ws, stream=s),
    "attn": lambda s: dma.paged_attn(c.p, c.c, Qd, c.ws, O, L, stream=s),
    "status": lambda s: dma.check("dma_check_device_status", dma.load().dma_check_device_status(
        c.p, c.ws.data_ptr(), dma._stream(s), ctypes.c_int32(0))),
    "clear": lambda s: dma.clear_device_status(c.p, c.ws, stream=s),
}
g0, k0, w0, w1 = torch.empty_like(q), torch.empty_like(k), f32(), f32()
for f in calls.values():
    f(None)
torch.cuda.synchronize()
rt = ctypes.CDLL("libcudart.so.12")
for bad in calls:
    s = torch.cuda.Stream()
    h = ctypes.c_void_p(s.cuda_stream)
    assert rt.cudaStreamBeginCapture(h, 1) == 0
    assert rt.cudaStreamSynchronize(h) != 0      # not allowed while capturing: the capture is void from here on
    try:
        calls[bad](s)
    except dma.DmaError as e:
        assert e.code == 4, e
    else:
        raise AssertionError(bad + " launched into a void capture")
    graph = ctypes.c_void_p()
    assert rt.cudaStreamEndCapture(h, ctypes.byref(graph)) != 0
    rt.cudaGetLastError()
    try:
        calls["prep"](None)
    except dma.DmaError as e:
        raise AssertionError("prep after a failed " + bad + ": " + str(e))
torch.cuda.synchronize()
print("ok")
"""


def test_a_failed_launch_is_not_reported_by_the_next_call():
    r = subprocess.run([sys.executable, "-c", _SCRIPT % {"root": ROOT}], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
