"""Arrivals on another CTA's mbarrier, by the kernels' sources: without a scope an arrival has the CTA's own,
which orders nothing with the CTA that waits; and a relaxed one orders earlier writes only behind a fence."""
import glob
import os
import re

import pytest

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "smem_swizzle_layouts_gb300", "csrc", "*.cu*")))
ARRIVE = re.compile(r"mbarrier\.arrive[.\w:]*shared::cluster[.\w:]*")


def code(path):
    return re.sub(r"//.*$", "", open(path).read(), flags=re.M)


def functions(text):
    """(name, body) of the device functions that hold an assembler statement."""
    for m in re.finditer(r"__device__ __forceinline__ void (\w+)\([^)]*\)\n\{\n(.*?)\n\}", text, re.S):
        if "asm volatile" in m.group(2):
            yield m.group(1), m.group(2)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_remote_arrivals_name_the_cluster_scope(path):
    for form in ARRIVE.findall(code(path)):
        assert ".release.cluster." in form or ".relaxed.cluster." in form, form


def test_the_pattern_finds_them():
    assert sum(len(ARRIVE.findall(code(p))) for p in SOURCES) >= 3


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_relaxed_arrivals_follow_a_fence_or_reads_alone(path):
    """A relaxed arrival stands behind a release fence in its function, or in one that is named for reads."""
    for name, body in functions(code(path)):
        if ".relaxed.cluster.shared::cluster" in body:
            assert "fence.release" in body or name.endswith("_read"), name
    text = code(path)
    for call in re.finditer(r"mbar_arrive_peer_read\((?!uint32_t)", text):
        before = text[:call.start()].rsplit("asm volatile", 1)[-1][-900:]
        assert "tc_fence_before_sync();" in before  # TMEM reads are complete and ordered
    for call in re.finditer(r"mbar_arrive_peer_written\((?!uint32_t)", text):
        before = text[:call.start()][-400:]
        assert all(f in before for f in ("fence_proxy_async_smem();", "tmem_st_wait();", "tc_fence_before_sync();", "__syncwarp();"))
