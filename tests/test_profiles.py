"""The committed profiles count for the kernels as they are: a summary names the hash of its kernel's sources (comments
left out), and the bench reports HBM traffic only from one that matches.  After a change to those sources a profile is
taken again, or, where the kernels compile to the same instructions, stamped again with a line that says so.  CPU only."""
import glob
import os
import re

import pytest

import bench

FILES = [p for p in sorted(glob.glob(os.path.join(bench.ROOT, "profiles", "*.txt"))) if "\nkernel_source_hash = " in open(p).read()]


def kind(name):
    if "producer" in name:
        return "producer"
    return ("step" if "decode" in name else "prefill") + ("_mimo" if "mimo" in name else "")


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(p) for p in FILES])
def test_profile_is_of_the_current_kernel(path):
    stamps = re.findall(r"^kernel_source_hash = (\w+)$", open(path).read(), re.M)
    assert stamps == [bench.kernel_source_hash(kind(os.path.basename(path)))]


def test_the_bench_finds_its_traffic():
    assert len(FILES) > 10
    for workload, launches in (("prefill_64k", 1), ("decode_256x28", 28)):
        assert bench.read_traffic(workload, launches) > 0
