"""The measured memory traffic that bench.py reports is that of the kernel's present sources (no GPU)."""
import bench


def test_the_record_holds():
    rec = bench._traffic_record()
    assert rec is not None and rec["dram_bytes_per_launch"] == rec["dram_read_bytes_per_launch"] + rec["dram_write_bytes_per_launch"]
