"""Ranks of a multi-GPU bench run use no TMA multicast load: the library's own planner, on every workload, no GPU."""
import json

import pytest

import bench

KINDS = {"nvfp4": 3, "mxfp4": 4}


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    from smem_swizzle_layouts_gb300 import _lib
    return _lib


def planned(g, wl, options):
    kind = KINDS[wl["fp4"]] if wl.get("fp4") else 2 if wl.get("mx") else 1 if wl.get("in_fmt") in ("e4m3", "e5m2") else 0
    opts = {k: v for k, v in (options or {}).items() if k != "workspace"}
    grouped = wl.get("kind") == "grouped"
    return g.gemm_debug_plan(4096 if grouped else wl["M"], wl["N"], wl["K"], kind, int(wl["a_major"] == "MN"), int(wl["b_major"] == "MN"),
                             grouped=grouped, options=opts or None, sms=152)


@pytest.mark.parametrize("name", sorted(bench.WORKLOADS))
@pytest.mark.parametrize("extra", ["", '{"cta_group": 1}', '{"cta_group": 1, "tile_n": 256, "tile_m": 128}',
                                   '{"cta_group": 1, "tile_n": 256, "tile_m": 256}'])
def test_ranks_plan_no_multicast(g, name, extra):
    wl = bench.WORKLOADS[name]
    options = dict(wl["options"] or {}, **json.loads(extra)) if extra else wl["options"]
    try:
        alone = planned(g, wl, bench.rank_options(options, 1))
    except g.GemmError:
        pytest.skip("tiles this kind does not have")
    ranks = planned(g, wl, bench.rank_options(options, 2))
    assert ranks["multicast_b"] == 0
    if not alone["multicast_b"] and alone["tile_n"] != 224:
        assert ranks == alone  # only what shares an operand changes


def test_one_gpu_keeps_its_options():
    assert bench.rank_options(None, 1) is None
    options = dict(cta_group=1, multicast_b=1)
    assert bench.rank_options(options, 1) is options
    assert bench.rank_options(dict(cta_group=1), 2) == dict(cta_group=1, multicast_b=-1)
    with pytest.raises(ValueError):
        bench.rank_options(options, 2)


def test_some_single_gpu_plan_multicasts(g):
    """What the ranks' options turn off is there to be turned off."""
    wl = bench.WORKLOADS["square8192_pair_f32_beta1"]
    assert planned(g, wl, dict(cta_group=1))["multicast_b"] == 1
