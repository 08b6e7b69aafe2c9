"""The cases that the GPU tests run reach every kernel variant of the router's
backward pass that a call within the library's limits can reach."""
import shutil

import pytest

import router_plans as R


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_the_cases_reach_every_variant(tmp_path):
    T = [1, 3, 33, 100, 300, 777, 1001, 2050, 4099, 8207, 16400, 32771, 65541, 131077, 270001, 1100001]
    d = [128, 384, 640, 1024, 2048, 4096, 7168, 16384, 65536]
    E = [1, 3, 4, 8, 13, 16, 20, 30, 32, 33, 50, 64, 65, 100, 128, 129, 150, 192, 200, 250, 256, 257, 300, 320, 333,
         384, 400, 448, 500, 511, 512]
    sweep = [(t, c, e, 1, act, mask, want) for t in T for c in d for e in E for act in ("bf16", "f32")
             for mask in (None, "random") for want in (R.ALL, R.DW, R.DX, ("dlogits",)) if t * c < 2 ** 31]
    reach = set().union(*R.variants(sweep, tmp_path))
    tested = set().union(*R.variants(R.CASES, tmp_path))
    assert len(reach) > 100
    assert not reach - tested, sorted(reach - tested)
