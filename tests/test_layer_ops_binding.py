"""The binding of the 8-bit steps and the gated linear recurrence where torch lacks the direct
entries that it prefers."""
import os
import subprocess
import sys

import pytest
import torch

import linear_attention_state_zero_b200 as tr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_direct_entries():
    """A torch without CUDA has none of them: the package imports, and its calls refuse host tensors."""
    code = """
import sys, torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
sys.modules["torch._C._dynamo.guards"] = None
import linear_attention_state_zero_b200 as tr
try:
    tr.quantize_fp8(torch.zeros(4, 128))
except ValueError as e:
    assert "CUDA" in str(e)
    print("refused")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr


@pytest.mark.gpu
def test_calls_without_direct_entries(cuda_device, monkeypatch):
    x = torch.randn(70, 256, device=cuda_device)
    side = torch.cuda.Stream()

    def calls():
        q, s, r = tr.rmsnorm_fp8(x, residual=x)
        w, ws = tr.quantize_fp8(x, block_rows=128)
        y = tr.projection_fp8(q, s, w, ws)
        h = tr.linear_recurrence(x, -x.abs(), [0, 30, 70])
        return [q.float(), s, r, y, *h, *tr.linear_recurrence_backward(x, -x.abs(), h[0], [0, 30, 70])[:2]]
    want = calls()
    monkeypatch.setattr(tr, "_raw_stream", tr._handle_of_current_stream)
    monkeypatch.setattr(tr, "_device_index", torch.cuda.current_device)
    monkeypatch.setattr(tr, "_empty_strided_cuda", tr._empty_strided)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
