"""The binding of the router, row movement and 4-bit product calls: what it
needs of torch, and buffers it refuses."""

import os
import subprocess
import sys

import pytest
import torch

from combine_ep_layout_04_amd import ep

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_imports_without_torchs_private_name():
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "from combine_ep_layout_04_amd import ep\n"
            "assert ep._raw_stream is ep._stream_handle\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=600)


@pytest.mark.gpu
def test_stream_handles():
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            assert ep._raw_stream(0) == ep._stream_handle(0) == stream.cuda_stream


def test_a_weights_gradient_needs_weights_and_rows():
    # refused before anything is looked at on a device
    rows, w = torch.zeros(4, 8), torch.zeros(4, 2)
    slot = torch.zeros(4, 2, dtype=torch.int32)
    grad = torch.zeros(4, 2)
    for kw in (dict(), dict(topk_weights=w), dict(x=rows)):
        with pytest.raises(ValueError, match="grad_weights needs topk_weights and x"):
            ep.ep_permute_backward(rows, slot, grad_weights=grad, **kw)
    for kw in (dict(), dict(topk_weights=w), dict(y=rows)):
        with pytest.raises(ValueError, match="grad_weights needs topk_weights and y"):
            ep.ep_unpermute_backward(rows, slot, grad_weights=grad, **kw)
    # with both the tensors are looked at
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_permute_backward(rows, slot, w, rows, grad_weights=grad)
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_unpermute_backward(rows, slot, w, rows, grad_weights=grad)
