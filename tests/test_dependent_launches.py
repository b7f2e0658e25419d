"""Kernels that start while the one before them still writes (programmatic dependent launches) read global memory
through coherent loads: a non-coherent load promises that nobody writes while the kernel lives, and may be moved
ahead of the wait for the kernel before."""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parents[1] / "log_mel_spectrogram_gb300" / "csrc"


def test_no_non_coherent_loads():
    dependents = [f for f in CSRC.glob("*.cu") if "pdl_wait()" in f.read_text()]
    assert {f.name for f in dependents} >= {"linear.cu", "kv_attend.cu", "kv_cache.cu", "beam.cu"}
    for f in dependents:
        code = re.sub(r"//.*", "", f.read_text())
        assert not re.search(r"__ldg\b|\.nc\b|__restrict__", code), f.name
