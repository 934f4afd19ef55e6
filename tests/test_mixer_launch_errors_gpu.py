"""A launch that CUDA refuses is reported with CUDA's reason.

While a blocking stream is captured, the host refuses a launch on the legacy stream (it would depend on the captured work);
nothing reaches the GPU.  The calls have valid inputs and run in a process of their own, each in a capture of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import ctypes, torch
import gated_delta_rule_123_b200 as kda
driver = ctypes.CDLL("libcuda.so.1")
x, w = torch.ones((2, 40, 64), device="cuda"), torch.ones((64, 4), device="cuda")
A, bc, h0 = -torch.ones((64, 16), device="cuda"), torch.ones((2, 40, 1, 16), device="cuda"), torch.zeros((2, 64, 16), device="cuda")
h, many, dh = (torch.ones(s, device="cuda", dtype=torch.bfloat16) for s in ((40, 64), (120, 64), (40, 40)))
x1, bc1, cache, mean = (torch.ones(s, device="cuda") for s in ((2, 64), (2, 1, 16), (2, 3, 64), (2, 40)))
calls = dict(
    layer_norm_fwd=lambda: kda.layer_norm_fwd(x), layer_norm_bwd=lambda: kda.layer_norm_bwd(x, x, None, mean, mean),
    linear_act=lambda: kda.linear_act(h, h), linear_act_many_rows=lambda: kda.linear_act(many, h),
    linear_act_bwd=lambda: kda.linear_act_bwd(dh, h, h),
    short_conv_fwd=lambda: kda.short_conv_fwd(x, w), short_conv_bwd=lambda: kda.short_conv_bwd(x, x, w),
    short_conv_step=lambda: kda.short_conv_step(x1, w, cache),
    selective_scan_fwd=lambda: kda.selective_scan_fwd(x, x, A, bc, bc),
    selective_scan_bwd=lambda: kda.selective_scan_bwd(x, x, x, A, bc, bc),
    selective_scan_step=lambda: kda.selective_scan_step(x1, x1, A, bc1, bc1, h0))
for f in calls.values():
    f()  # memory for the outputs is at hand afterwards
for name, f in calls.items():
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert driver.cuStreamCreate(ctypes.byref(stream), 0) == 0
    assert driver.cuStreamBeginCapture_v2(stream, 2) == 0
    try:
        f()
        print(name, "|", "not refused")
    except kda.KDAError as e:
        print(name, "|", e)
    driver.cuStreamEndCapture(stream, ctypes.byref(graph))
    assert driver.cuStreamDestroy_v2(stream) == 0
    f()
torch.cuda.synchronize()
"""


def test_reason_of_a_refused_launch():
    run = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    lines = [line for line in run.stdout.splitlines() if "|" in line]
    assert len(lines) == 11
    for line in lines:
        assert "KDA_ERR_CUDA" in line and "legacy stream" in line, run.stdout
