"""Another CTA's shared memory, by the kernels' sources: it may be written, and its barriers signalled, only once that CTA is
known to have started, which a barrier of the cluster says. Each kernel that takes another CTA's address has one before."""
import glob
import os
import re

import pytest

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "smem_swizzle_layouts_gb300", "csrc", "*.cu*")))
REMOTE = re.compile(r"mapa_shared\(|st\.(?:async|shared::cluster)|\bmma_commit_pair_multicast\(|_peer_\w+\(")
STARTED = re.compile(r"cluster_sync_all\(\)|cluster_wait\(\)")


def kernels(path):
    """(name, body) of the kernels, without comments."""
    text = re.sub(r"//.*$", "", open(path).read(), flags=re.M)
    for m in re.finditer(r"__global__[^;{]*?(\w+)\(", re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", lambda b: " " * len(b.group()), text)):
        at = text.index("{", m.end())
        depth, end = 0, at
        for end in range(at, len(text)):
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            if depth == 0:
                break
        yield m.group(1), text[at:end]


FOUND = [(os.path.basename(p), name, body) for p in SOURCES for name, body in kernels(p) if REMOTE.search(body)]


@pytest.mark.parametrize("body", [f[2] for f in FOUND], ids=[f"{f[0]}-{f[1]}" for f in FOUND])
def test_a_cluster_has_started_before_its_memory_is_written(body):
    before = body[:REMOTE.search(body).start()]
    assert STARTED.search(before)


def test_the_kernels_of_clusters_are_found():
    assert {f[1] for f in FOUND} >= {"balance_join_kernel", "head_kernel"}
    assert len(FOUND) >= 3
