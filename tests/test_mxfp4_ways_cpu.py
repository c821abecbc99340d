"""That the sizes the GPU tests run reach every way of the MXFP4 products and of
the experts (on the host: the rules that choose are refitted now and then, and
sizes chosen for one set of rules would quietly go another way)."""
import os

import pytest

import latency_skinny_gemm_amd as skg
from latency_skinny_gemm_amd import build as lib_build
from tests import mxfp4_sizes as sizes


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(skg.library_path()):
        lib_build.build()
    return skg.lib()


TILES = {"e4m3": (0, 1, 2, 3, 4), "e2m1": (0, 5, 6, 7)}


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_sizes_reach_every_way_of_a_product(lib, fmt, codes):
    want = {f"tile {t}{end}" for t in TILES[fmt] for end in ("", ", K inside a step", ", K past 8192")}
    for way in (("codes", "codes over 16") if codes else ("rows", "first", "first over 16")):
        want |= {way, way + ", ragged", way + ", rounds"}
    reached = set()
    for M, N, K in sizes.PRODUCTS:
        reached |= sizes.product_way(lib, M, N, K, fmt, codes)
    assert want <= reached, want - reached
    assert {w for w in reached if w.startswith("tile")} <= want  # no other tile
    if fmt == "e4m3":  # as many rows as LDS holds
        assert any(w.endswith("all that fit") for w in reached)


def test_no_way_but_those_tested(lib):
    """Over the whole domain: no product takes a tile that the tests leave out,
    and every block fits its kernel."""
    for fmt in ("e4m3", "e2m1"):
        for codes in (False, True):
            for M in (*range(1, 40), *range(40, 513, 13), 512):
                for N in (1, 16, 100, 576, 1111, 2112, 4096, 6300, 16384, 65536, (1 << 20) - 1):
                    for K in (32, 96, 1056, 2048, 4224, 7168, 9440, 30016, 130000):
                        for w in sizes.product_way(lib, M, N, K, fmt, codes):
                            if w.startswith("tile"):
                                assert int(w.split()[1].rstrip(",")) in TILES[fmt]
                            else:
                                assert not w.startswith("rows over 16")  # bf16 rows: at most 16 a block


def test_sizes_reach_every_way_of_the_experts(lib):
    assert {sizes.experts_way(lib, *s, "e4m3") for s in sizes.EXPERTS} == {0, 16, 32, 64}
    assert {sizes.experts_way(lib, *s, "e2m1") for s in sizes.EXPERTS} == {0, 16, 32, 64, 96}
