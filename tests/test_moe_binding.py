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
