"""The entry points of skinny_moe.h on the CPU: exported, and every refusal
made before any device call (addresses here are fake and never read); and the
plain implementations that the GPU tests compare with, against torch."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import latency_skinny_gemm_amd as skg
from latency_skinny_gemm_amd import build as lib_build
from latency_skinny_gemm_amd import moe
from tests import mx_reference as ref
from workloads import inputs as gen

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ARG, ALIGN, UNSUP = skg.OK, skg.ERR_INVALID_ARG, skg.ERR_ALIGNMENT, skg.ERR_UNSUPPORTED
A, B, C, D, E, F = (0x10000000 * (i + 1) for i in range(6))  # far apart


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(skg.library_path()):
        lib_build.build()
    return skg.lib()


def test_every_declared_symbol_is_exported(lib):
    txt = open(os.path.join(ROOT, "include", "skinny_moe.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    names = set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(skinny_\w+)\s*\(", txt, flags=re.M))
    assert len(names) == 9
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("args,status", [
    ((A, B, C, 1, 4, 64), ARG),            # no such format
    ((A, B, C, 0, -1, 64), ARG),
    ((A, B, C, 0, 0, 64), OK),             # no rows
    ((0, 0, 0, 0, 0, 64), OK),
    ((A, B, C, 0, 4, 0), UNSUP),
    ((A, B, C, 0, 4, 48), UNSUP),          # not whole blocks
    ((A, B, C, 4, 1 << 20, 1 << 11), UNSUP),  # 2^31 values
    ((0, B, C, 0, 4, 64), ARG),
    ((A, 0, C, 0, 4, 64), ARG),
    ((A, B, 0, 0, 4, 64), ARG),
    ((A + 2, B, C, 0, 4, 64), ALIGN),
    ((A, B + 8, C, 0, 4, 64), ALIGN),
    ((A, A, C, 0, 4, 64), ARG),            # codes over x
    ((A, B, A + 500, 0, 4, 64), ARG),      # scales over x
    ((A, B, B + 255, 0, 4, 64), ARG),      # scales over codes
])
def test_quant_mx_refusals(lib, args, status):
    assert lib.skinny_quant_mx(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((A, B, 2, C, 4, 64), ARG),            # no such format
    ((A, B, 0, C, -1, 64), ARG),
    ((0, 0, 0, 0, 0, 64), OK),
    ((A, B, 0, C, 4, 48), UNSUP),
    ((0, B, 0, C, 4, 64), ARG),
    ((A, 0, 0, C, 4, 64), ARG),
    ((A, B, 0, 0, 4, 64), ARG),
    ((A + 4, B, 0, C, 4, 64), ALIGN),
    ((A, B, 0, C + 2, 4, 64), ALIGN),
    ((A, B, 0, A - 496, 4, 64), ARG),      # values over codes
    ((A, B, 4, B - 500, 4, 64), ALIGN),
    ((A, B, 4, B - 496, 4, 64), ARG),      # values over scales
])
def test_dequant_mx_refusals(lib, args, status):
    assert lib.skinny_dequant_mx(*args, None) == status


def _norm(lib, x=A, r=0, w=B, eps=1e-6, fmt=0, scale=0, y=C, e=0, ro=0, M=4, K=64):
    return lib.skinny_rmsnorm(x, r, w, eps, fmt, scale, y, e, ro, M, K, None)


@pytest.mark.parametrize("change,status", [
    (dict(M=0), OK), (dict(M=-1), ARG), (dict(K=4), UNSUP), (dict(K=68), UNSUP),
    (dict(K=65544), UNSUP), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(fmt=3), ARG), (dict(fmt=-1), ARG), (dict(x=0), ARG), (dict(w=0), ARG), (dict(y=0), ARG),
    (dict(r=D), ARG), (dict(ro=D), ARG),                      # one without the other
    (dict(fmt=1), ARG), (dict(scale=D), ARG),                 # a scale goes with e4m3 only
    (dict(fmt=2), ARG), (dict(e=D), ARG),                     # e8m0 goes with MX only
    (dict(fmt=2, e=D, K=72), UNSUP),
    (dict(x=A + 8), ALIGN), (dict(w=B + 2), ALIGN), (dict(y=C + 8), ALIGN),
    (dict(r=D + 2, ro=E), ALIGN), (dict(fmt=1, scale=D + 2), ALIGN),
    (dict(y=A), ARG), (dict(y=A + 496), ARG), (dict(y=B), ARG),
    (dict(r=D, ro=A + 256), ARG), (dict(r=D, ro=C), ARG), (dict(r=D, ro=D + 16), ARG),
    (dict(r=D, ro=E, y=D), ARG), (dict(r=D, ro=D, y=D), ARG), (dict(r=D, ro=A, y=A), ARG),
    (dict(M=1 << 30, K=1024), UNSUP),
])
def test_rmsnorm_refusals(lib, change, status):
    assert _norm(lib, **change) == status


def _route(lib, l=A, dtype=2, bias=0, scores=0, k=2, groups=1, top=1, renorm=1, w=B, ids=C, T=3, E_=16,
           o=True):
    opt = moe.RouteOptions(scores, k, groups, top, renorm, 1.0)
    return lib.skinny_route(l, dtype, bias, ctypes.byref(opt) if o else None, w, ids, T, E_, None)


@pytest.mark.parametrize("change,status", [
    (dict(T=0), OK), (dict(T=-1), ARG), (dict(E_=0), ARG), (dict(k=0), ARG), (dict(o=False), ARG),
    (dict(dtype=1), ARG), (dict(scores=2), ARG), (dict(groups=0), ARG), (dict(top=0), ARG),
    (dict(k=17), UNSUP), (dict(k=65, E_=128), UNSUP), (dict(E_=1025), UNSUP),
    (dict(groups=3), UNSUP), (dict(groups=4, top=5), UNSUP), (dict(groups=4, top=1, k=5), UNSUP),
    (dict(groups=128, E_=128, top=128), UNSUP),
    (dict(l=0), ARG), (dict(w=0), ARG), (dict(ids=0), ARG),
    (dict(l=A + 2), ALIGN), (dict(l=A + 1, dtype=0), ALIGN), (dict(bias=D + 1), ALIGN),
    (dict(w=B + 2), ALIGN), (dict(ids=C + 1), ALIGN),
    (dict(ids=B), ARG), (dict(w=A), ARG), (dict(ids=D, bias=D), ARG),
])
def test_route_refusals(lib, change, status):
    assert _route(lib, **change) == status


def test_pack_sizes_and_refusals(lib):
    size = lib.skinny_mxfp4_packed_bytes
    # 16-column groups: 1 KB for each 128 K, 256 bytes for each 512
    assert size(1, 16, 128) == 1024 + 256
    assert size(3, 17, 544) == 3 * 2 * (5 * 1024 + 2 * 256)
    for bad in ((0, 16, 128), (1, 0, 128), (1, 16, 0), (1, 16, 40), (65536, 16, 128),
                (1, 1 << 20, 128), (1, 16, 1 << 20)):
        assert size(*bad) == 0
    pack = lib.skinny_mxfp4_pack
    assert pack(A, B, C, 0, 16, 128, None) == ARG
    assert pack(A, B, C, 1, 16, 40, None) == UNSUP
    assert pack(0, B, C, 1, 16, 128, None) == ARG
    assert pack(A, B, 0, 1, 16, 128, None) == ARG
    assert pack(A + 8, B, C, 1, 16, 128, None) == ALIGN
    assert pack(A, B, C + 8, 1, 16, 128, None) == ALIGN
    assert pack(A, B, A, 1, 16, 128, None) == ARG
    assert pack(A, B, B - 1024, 1, 16, 128, None) == ARG


def _gemm(lib, x=A, xe=0, fmt=0, w=B, bias=0, out=C, dtype=0, M=4, N=32, K=64):
    return lib.skinny_gemm_mxfp4(x, xe, fmt, w, bias, out, dtype, M, N, K, None)


@pytest.mark.parametrize("change,status", [
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=-1), ARG), (dict(N=-1), ARG), (dict(K=-32), ARG),
    (dict(M=513), UNSUP), (dict(K=0), UNSUP), (dict(K=48), UNSUP), (dict(K=1 << 20), UNSUP),
    (dict(N=1 << 20), UNSUP), (dict(fmt=2), ARG), (dict(dtype=1), ARG),
    (dict(x=0), ARG), (dict(w=0), ARG), (dict(out=0), ARG),
    (dict(x=A + 8), ALIGN), (dict(w=B + 4), ALIGN), (dict(out=C + 1), ALIGN),
    (dict(out=C + 2, dtype=2), ALIGN), (dict(bias=D + 1), ALIGN),
    (dict(out=A), ARG), (dict(out=B), ARG), (dict(out=D, bias=D), ARG), (dict(out=D, xe=D), ARG),
])
def test_gemm_mxfp4_refusals(lib, change, status):
    assert _gemm(lib, **change) == status


def _moe(lib, x=A, ids=B, w=C, w13=D, w2=E, out=F, fmt=0, T=2, k=2, H=64, I=32, E_=4):
    return lib.skinny_moe_mxfp4(x, ids, w, w13, w2, out, fmt, T, k, H, I, E_, None)


@pytest.mark.parametrize("change,status", [
    (dict(T=0), OK), (dict(T=-1), ARG), (dict(k=0), ARG), (dict(H=0), ARG), (dict(I=0), ARG),
    (dict(E_=0), ARG), (dict(fmt=1), ARG), (dict(H=48), UNSUP), (dict(I=40), UNSUP),
    (dict(E_=1025), UNSUP), (dict(k=65), UNSUP), (dict(T=1 << 26), UNSUP),
    (dict(x=0), ARG), (dict(ids=0), ARG), (dict(w=0), ARG), (dict(w13=0), ARG), (dict(w2=0), ARG),
    (dict(out=0), ARG), (dict(x=A + 2), ALIGN), (dict(ids=B + 2), ALIGN), (dict(w=C + 1), ALIGN),
    (dict(w13=D + 8), ALIGN), (dict(w2=E + 8), ALIGN), (dict(out=F + 8), ALIGN),
    (dict(out=A), ARG), (dict(out=B), ARG), (dict(out=D), ARG), (dict(out=E), ARG),
])
def test_moe_refusals(lib, change, status):
    assert _moe(lib, **change) == status


def test_reserve_refusals(lib):
    r = lib.skinny_moe_reserve
    assert r(0, 0, 0, 1, 32, 32, 1, None) == OK      # nothing asked for
    assert r(513, 64, 0, 1, 32, 32, 1, None) == UNSUP
    assert r(1, 40, 0, 1, 32, 32, 1, None) == UNSUP
    assert r(-1, 64, 0, 1, 32, 32, 1, None) == ARG
    assert r(0, 0, -1, 1, 32, 32, 1, None) == ARG
    assert r(0, 0, 1, 0, 32, 32, 1, None) == ARG
    assert r(0, 0, 1, 1, 40, 32, 1, None) == UNSUP


def test_binding_refusals_need_no_device():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: skg.quant_mx(x), lambda: skg.rmsnorm(x, x[0]),
                 lambda: skg.route(x, 2), lambda: skg.mxfp4_pack(x, x),
                 lambda: skg.moe_mxfp4(x, x, x, None, None)):
        with pytest.raises((ValueError, TypeError)):  # host tensors
            call()
    with pytest.raises(ValueError):
        skg.quant_mx(x, "e5m2")
    with pytest.raises(TypeError):
        skg.gemm_mxfp4(x, x)


# ------------------------------------------------------------ the references

def test_reference_e4m3_matches_the_generator():
    g = torch.Generator().manual_seed(3)
    v = torch.randn(64, 320, generator=g) * torch.exp2(torch.randint(-20, 20, (64, 320), generator=g).float())
    v[3, 32:64] = 0
    q, e = gen.quantise_mx(v)
    codes, er = ref.quantise(v.double().numpy(), "e4m3")
    assert np.array_equal(er, e.numpy())
    assert np.array_equal(ref.pack_bytes(codes, "e4m3"), gen.bits8(q))
    assert np.array_equal(ref.dequantise(codes, er, "e4m3"),
                          (q.double().reshape(64, 10, 32) * torch.exp2(e.double() - 127)[..., None])
                          .reshape(64, 320).numpy())


def test_reference_e2m1_rounds_ties_to_even():
    v = np.zeros((1, 32))
    v[0, :16] = [6, 0.25, 0.2500001, 0.75, 0.7499999, 1.25, 1.75, 2.5, 3.5, 5, 5.0000001, -0.75, -5,
                 0.5, -6, -0.1]
    codes, e = ref.quantise(v, "e2m1")
    assert e[0, 0] == 127
    assert list(codes[0, :16]) == [7, 0, 1, 2, 1, 2, 4, 4, 6, 6, 7, 10, 14, 1, 15, 8]
    assert np.array_equal(ref.unpack_bytes(ref.pack_bytes(codes, "e2m1"), "e2m1"), codes)


def test_reference_route_by_hand():
    l = np.array([[0.0, 3.0, 1.0, 2.0], [1.0, 1.0, 1.0, 1.0]])
    _, _, ids, w = ref.route(l, 2, "softmax", None, 1, 1, True, 2.0)
    assert ids.tolist() == [[1, 3], [0, 1]]
    assert np.allclose(w, [[2 / (1 + np.exp(-1.0)), 2 / (1 + np.exp(1.0))], [1, 1]])
    _, _, ids, _ = ref.route(l, 2, "sigmoid", np.array([9.0, 0, 0, 0]), 2, 1, True, 1.0)
    assert ids.tolist() == [[0, 1], [0, 1]]
