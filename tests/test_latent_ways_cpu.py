"""That the sizes the GPU tests run reach every form of latent attention and of the
products per head (on the host: the rules that choose are refitted now and then, and
sizes chosen for one set of rules would quietly go another way)."""
import ctypes
import os

import pytest

import latency_skinny_gemm_amd as skg
from latency_skinny_gemm_amd import build as lib_build
from tests import latent_sizes as sizes


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(skg.library_path()):
        lib_build.build()
    L = skg.lib()
    L.skg_latent_rows.argtypes = [ctypes.c_int] * 3 + [ctypes.c_long, ctypes.c_int]
    L.skg_heads_ring.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_long]
    return L


@pytest.mark.parametrize("e4m3", [False, True])
def test_sizes_take_the_rows_they_name(lib, e4m3):
    for counts, lens, H, page, width, rows in sizes.UNSEEN + sizes.SHORT + sizes.LONG:
        assert sizes.rows_of(lib, counts, lens, H, page, width, e4m3) == rows, (counts, H)


def test_unseen_rows_are_tried_in_every_form(lib):
    """Both tiles, tables entered by steps (pages of 32 rows and more) and by eight rows, both ways to plan."""
    forms = {(rows, page >= 32) for _, _, _, page, _, rows in sizes.UNSEEN}
    assert forms == {(32, False), (32, True), (64, False), (64, True)}
    assert {len(counts) > 64 for counts, *_ in sizes.UNSEEN} == {False, True}
    for counts, lens, H, *_, rows in sizes.UNSEEN:
        assert rows // H > 1  # a tile has tokens that see different rows
    assert {sizes.parts_of(lib, counts, keys, H) > 1 for counts, keys, H, _ in sizes.UNSEEN_KEYS} == {False, True}
    for counts, keys, H, shared in sizes.UNSEEN_KEYS:
        assert (sizes.parts_of(lib, counts, keys, H) > 1) == shared, (counts, keys)


@pytest.mark.parametrize("e4m3", [0, 1])
def test_rows_of_a_workgroup(lib, e4m3):
    """The rule's clauses, one by one: as many tiles of either, tiles enough, rows wasted, long tables, many tiles."""
    rows = lib.skg_latent_rows
    assert rows(1, 1, 32, 1 << 20, e4m3) == 32          # one tile either way
    assert rows(1, 1, 128, 4000, e4m3) == 32            # one sequence's token
    assert rows(128, 128, 128, 6016, e4m3) == 64        # 256 tiles of 64 rows
    assert rows(12, 150, 20, 9024, e4m3) == 64          # three tokens of 20 heads fill 60 of 64 rows, one 20 of 32
    assert rows(2, 512, 128, 8192, e4m3) == 64
    assert rows(16, 16, 128, 24000, e4m3) == 64         # 32 tiles of long sequences
    assert rows(16, 16, 128, 4000, e4m3) == 32
    assert rows(4, 4, 128, 100000, e4m3) == 32          # fewer than 32 tiles
    assert rows(1, 100, 128, 200, e4m3) == (32 if e4m3 else 64)  # 400 tiles of 32 rows


def test_products_per_head(lib):
    for T, K, ring in ((1, 128, 0), (127, 128, 0), (128, 128, 1), (31, 512, 0), (32, 512, 1), (64, 256, 1), (43, 384, 1),
                       (42, 384, 0), (2048, 96, 0), (2048, 480, 0), (1 << 20, 128, 1)):
        assert lib.skg_heads_ring(T, K, 128 * K) == ring, (T, K)
    assert lib.skg_heads_ring(2048, 512, (1 << 26) - 8) == 1 and lib.skg_heads_ring(2048, 512, 1 << 26) == 0
