"""Kernels that start beside the grid ahead of them read what it may write by ordinary loads: the read-only path is for what
is constant as long as the kernel lives (here a norm's gain)."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "nvfp4_block_scaled_04_gb300" / "csrc"


def read_only_loads(name):
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    assert "pdl_wait()" in text
    return [line.strip() for line in text.splitlines() if re.search(r"__ldg|\.nc\b|ld_stream", line)]


def test_the_draw_reads_logits_by_ordinary_loads():
    assert read_only_loads("sample.cu") == []


def test_the_norm_reads_only_its_gain_through_the_read_only_path():
    loads = read_only_loads("norm.cu")
    assert loads and all("(weight + k)" in line for line in loads), loads


def test_activation_rows_are_read_by_ordinary_loads():
    """(The loads of a decode linear's activations: its first kernel starts beside a norm, an attention or a linear.)"""
    text = (CSRC / "gemv_core.cuh").read_text()
    for name in ("xprep_row(", "xprep_row_regs("):
        at = text.index("NVFP4_DEV void " + name)
        body = text[at:text.index("\n}\n", at)]
        assert "src)" in body and "__ldg" not in body, name
