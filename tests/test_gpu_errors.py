"""A launch that the CUDA runtime refuses is that call's error alone.

In a process of its own: a launch into the legacy stream is refused while
another stream is captured, before anything reaches the GPU. The next call,
after the capture has been given up, must run."""
import os
import subprocess
import sys

import pytest

from rank_delta_gb300 import build as rdbuild

pytestmark = pytest.mark.gpu

CHILD = """
import ctypes
import torch
import rank_delta_gb300 as rd

torch.zeros(1, device="cuda")
cudart = ctypes.CDLL("libcudart.so.13")
x = torch.randn(4, 100, device="cuda")
entropy = torch.zeros(4, device="cuda")
w = torch.randn(4, 64, device="cuda")
codes, scales = torch.zeros(128, dtype=torch.uint8, device="cuda"), torch.zeros(8, dtype=torch.uint8, device="cuda")
ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()

def score():
    rd.lora_logprobs(x, rd.LORA_DTYPE_F32, 100, 4, 100, None, 1.0, 0, None, entropy, None, None, None, ws, 256)

def quantise():
    rd.lora_mx4_quantize(w, rd.LORA_DTYPE_F32, 64, 4, 64, codes, scales)

def pool():
    from rank_delta_gb300 import torch_helpers as th
    r = th.DeviceRoute(2, 8, 64, 32)
    a, b = torch.ones(4, 64, device="cuda").bfloat16(), torch.ones(32, 4, device="cuda").bfloat16()
    rd.lora_pool_pack(r.rt, 0, a, b, 4, 0.0, False, 1.0)

stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
for call in (score, quantise):
    for after in (pool, score, quantise):
        assert cudart.cudaStreamCreateWithFlags(ctypes.byref(stream), 0) == 0
        assert cudart.cudaStreamBeginCapture(stream, 0) == 0
        try:
            call()
        except rd.LoraError as e:
            assert e.code == rd.LORA_ERR_CUDA, e
        else:
            raise AssertionError("the launch was not refused")
        cudart.cudaStreamEndCapture(stream, ctypes.byref(graph))
        cudart.cudaGetLastError()
        after()
        torch.cuda.synchronize()
        assert cudart.cudaStreamDestroy(stream) == 0
print("the next calls ran")
"""


def test_a_refused_launch_is_not_reported_by_the_next_call():
    rdbuild.build()
    root = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "the next calls ran" in r.stdout, r.stderr[-2000:]
