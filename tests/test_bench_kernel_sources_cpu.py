"""The sources that bench.py ties its recorded DRAM counters to: the attention
kernel's and the planner's files, with every header of this library that they
include."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "mla_latent_kv_05_gb300", "csrc")


def included(name, seen):
    """`name` and the csrc headers that it includes, directly or not."""
    if name not in seen and os.path.exists(os.path.join(CSRC, name)):
        seen.add(name)
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            for header in re.findall(r'^\s*#include\s+"([^"]+)"', f.read(), re.M):
                included(header, seen)
    return seen


def test_the_recorded_counters_depend_on_every_file_of_the_kernel_and_the_planner():
    want = included("decode.cu", set()) | included("plan.cu", set())
    assert {"decode.cu", "decode.cuh", "plan.cu", "common.cuh"} <= want
    assert set(bench.KERNEL_SOURCES) == want


def test_a_change_of_any_of_them_makes_the_records_stale(tmp_path, monkeypatch):
    h0 = bench.kernel_source_hash()
    dst = tmp_path / "mla_latent_kv_05_gb300" / "csrc"
    dst.mkdir(parents=True)
    for name in bench.KERNEL_SOURCES:
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            (dst / name).write_text(f.read())
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() == h0
    for name in bench.KERNEL_SOURCES:
        text = (dst / name).read_text()
        (dst / name).write_text(text + "\nint changed;\n")
        assert bench.kernel_source_hash() != h0, name
        (dst / name).write_text(text)
