"""The stream that calls go to, with and without torch's private accessor."""
import subprocess
import sys
from types import SimpleNamespace
from pathlib import Path

import pytest
import torch

ROOT = Path(__file__).resolve().parents[1]


def test_public_accessor_where_the_private_one_is_missing(monkeypatch):
    import nvfp4_block_scaled_04_gb300 as m
    monkeypatch.setattr(m, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(cuda_stream=0x1234))
    assert m._stream() == 0x1234


def test_private_accessor_is_asked_for_the_current_device(monkeypatch):
    import nvfp4_block_scaled_04_gb300 as m
    monkeypatch.setattr(m, "_raw_stream", lambda device: 0x100 + device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert m._stream() == 0x103


def test_package_imports_without_the_private_accessor():
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import nvfp4_block_scaled_04_gb300 as m\n"
            "from types import SimpleNamespace\n"
            "torch.cuda.current_stream = lambda *a: SimpleNamespace(cuda_stream=77)\n"
            "assert m._stream() == 77\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


@pytest.mark.gpu
def test_both_accessors_agree_on_a_side_stream():
    import nvfp4_block_scaled_04_gb300 as m
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert m._stream() == side.cuda_stream == torch.cuda.current_stream().cuda_stream
