"""Sizes of MXFP4 products and of the experts that reach every way they are done,
and what names a way (test infrastructure)."""
import ctypes

FORMATS = {"e4m3": 0, "e2m1": 4}

# (M, N, K): one row; blocks of rows, whole and ragged, in one round of loads and in
# several, as many as fit in LDS, more than 16; every tile, with K that ends inside a
# step of 128 and K past the 8192 whose scales a tile holds at once
PRODUCTS = [(1, 40, 7168), (1, 1000, 96), (7, 500, 2880), (16, 576, 4096), (37, 1111, 2880), (102, 539, 5472),
            (173, 470, 4768), (43, 1173, 5088), (208, 147, 8768), (446, 21, 9440), (276, 162, 4288), (21, 2294, 4832),
            (33, 2948, 1792), (100, 548, 4032), (22, 2351, 4224), (329, 129, 5152), (280, 146, 5376), (61, 1119, 4192),
            (24, 4096, 1056), (128, 2112, 544), (512, 272, 288), (500, 1100, 160), (512, 600, 96), (512, 2100, 544),
            (222, 1942, 160), (512, 6300, 96), (486, 3998, 96), (64, 2112, 8480), (130, 2112, 8736), (300, 2112, 8224),
            (490, 2180, 8736), (512, 4100, 8224), (482, 6400, 8480)]

# (T, k, E, H, I): pair by pair; sorted into tiles of 16, 32 and 64 rows, and 96
EXPERTS = [(1, 1, 1, 96, 64), (5, 2, 6, 1056, 992), (72, 4, 72, 480, 480), (200, 4, 40, 288, 288), (600, 8, 12, 96, 96),
           (2500, 2, 20, 128, 96), (2000, 4, 6, 96, 64), (2500, 2, 100, 32, 1024)]


def steps(K):
    return (K + 127) // 128


def product_way(lib, M, N, K, fmt, codes):
    """Names of the way of skinny_gemm_mxfp4 and of what is particular about it."""
    rows, first, tile = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    blocks = lib.skg_mxfp4_way(M, N, K, FORMATS[fmt], 1 if codes else 0, ctypes.byref(rows), ctypes.byref(first),
                               ctypes.byref(tile))
    if blocks == 0:
        way = f"tile {tile.value}"
        return {way} | ({way + ", K inside a step"} if K % 128 else set()) | ({way + ", K past 8192"} if K > 8192 else set())
    r = rows.value
    assert (blocks - 1) * r < M <= blocks * r
    way = ("first" if first.value else "codes" if codes else "rows") + (" over 16" if r > 16 else "")
    names = {way}
    if M % r:
        names.add(way + ", ragged")
    waves = 4 if steps(K) <= 16 else 8 if steps(K) <= 32 else 16
    bf16 = not codes and not first.value
    pieces = steps(K) * (16 if bf16 else 8 if fmt == "e4m3" else 4)
    if r * ((pieces + 63) // 64) > 4 * waves:
        names.add(way + ", rounds")
    if r == 124 * 1024 // (steps(K) * ((128 if fmt == "e4m3" else 64) + 4) + 64):
        names.add(way + ", all that fit")
    return names


def experts_way(lib, T, k, E, H, I, fmt):
    return lib.skg_moe_way(T, k, H, I, E, FORMATS[fmt])
