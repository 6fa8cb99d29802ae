"""bench.py's records of measured traffic go with the sources they were taken on."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_traffic_records_are_of_the_present_sources(monkeypatch):
    monkeypatch.syspath_prepend(ROOT)
    monkeypatch.setattr(sys, "argv", ["bench.py"])
    import bench
    for kernel in bench.KERNEL_SOURCES:
        assert bench._traffic(kernel) is not None, kernel
