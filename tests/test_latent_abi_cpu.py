"""The entry points of skinny_latent.h on the CPU: exported, and every refusal made
before any device call (addresses here are fake and never read); the binding's
checks; and the plain implementations that the GPU tests compare with, against
torch."""
import ctypes
import math
import os
import re

import pytest
import torch

import latency_skinny_gemm_amd as skg
from latency_skinny_gemm_amd import build as lib_build
from latency_skinny_gemm_amd.latent import LatentBatch
from tests import latent_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ARG, ALIGN, UNSUP = skg.OK, skg.ERR_INVALID_ARG, skg.ERR_ALIGNMENT, skg.ERR_UNSUPPORTED
A, B, C, D, E, F, G, H_, I_ = (0x100000000 * (i + 1) for i in range(9))  # far apart


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(skg.library_path()):
        lib_build.build()
    return skg.lib()


def test_every_declared_symbol_is_exported(lib):
    txt = open(os.path.join(ROOT, "include", "skinny_latent.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    names = set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(skinny_\w+)\s*\(", txt, flags=re.M))
    assert names == {"skinny_latent_append", "skinny_latent_attention", "skinny_latent_attention_expanded",
                     "skinny_heads_gemm", "skinny_latent_reserve"}
    for n in names:
        assert hasattr(lib, n), n


def _batch(table=G, kv_lens=H_, q_starts=I_, B=2, T=5, table_width=4, page_size=16, pages=9):
    return LatentBatch(table, kv_lens, q_starts, B, T, table_width, page_size, pages)


BATCHES = [
    (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(table_width=-1), ARG), (dict(page_size=0), ARG), (dict(pages=-1), ARG),
    (dict(B=8193), UNSUP), (dict(page_size=4), UNSUP), (dict(page_size=48), UNSUP), (dict(page_size=1 << 17), UNSUP),
    (dict(table_width=1 << 16, page_size=1 << 15), UNSUP),
    (dict(q_starts=0), ARG),                 # five tokens of two sequences
    (dict(T=0), OK), (dict(B=0), OK), (dict(B=0, T=0, q_starts=0), OK),
    (dict(table=0), ARG), (dict(kv_lens=0), ARG),
    (dict(table=G + 2), ALIGN), (dict(kv_lens=H_ + 1), ALIGN), (dict(q_starts=I_ + 2), ALIGN),
]


def _append(lib, batch=None, kv=A, kv_stride=576, weight=B, eps=1e-6, rot=C, rows=64, style=0, cache=D, dtype=0, scale=0,
            latent=0, q=E, qt=192, qh=64, qo=F, ot=192, oh=64, heads=3):
    b = _batch(**(batch or {}))
    return lib.skinny_latent_append(b, kv, kv_stride, weight, eps, rot, rows, style, cache, dtype, scale, latent, q, qt, qh,
                                    qo, ot, oh, heads, None)


@pytest.mark.parametrize("batch,status", BATCHES)
def test_append_batch_refusals(lib, batch, status):
    b = dict(batch)
    if "table_width" in b:
        assert _append(lib, batch=b, rows=2147483647) == status
    else:
        assert _append(lib, batch=b) == status


@pytest.mark.parametrize("kw,status", [
    (dict(style=2), ARG), (dict(rows=-1), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG),
    (dict(dtype=2), ARG), (dict(dtype=1), ARG), (dict(scale=B), ARG),
    (dict(q=0), ARG), (dict(qo=0), ARG), (dict(heads=0), ARG), (dict(heads=-1), ARG),
    (dict(heads=1025), UNSUP),
    (dict(kv_stride=568), ARG), (dict(kv_stride=580), ARG), (dict(qt=190), ARG), (dict(oh=-8), ARG),
    (dict(kv_stride=1 << 41), UNSUP),
    (dict(oh=56), ARG),                              # heads over each other
    (dict(ot=128), ARG),                             # tokens over each other
    (dict(rows=63), UNSUP),                          # the table may name row 63
    (dict(kv=0), ARG), (dict(rot=0), ARG), (dict(cache=0), ARG),
    (dict(kv=A + 8), ALIGN), (dict(weight=B + 2), ALIGN), (dict(rot=C + 4), ALIGN), (dict(cache=D + 8), ALIGN),
    (dict(dtype=1, scale=B + 0x1002), ALIGN), (dict(latent=F + 0x100008), ALIGN), (dict(q=E + 2), ALIGN),
    (dict(cache=A), ARG), (dict(latent=A + 1152 * 4), ARG), (dict(qo=D + 16), ARG), (dict(qo=E + 16), ARG),
    (dict(qo=E, ot=200), ARG),                       # in place, but with other strides
    (dict(kv_stride=1280, q=A + 1152, qt=1280, qo=A + 1136, ot=1280), ARG),      # queries beside the latents, one piece into them
    (dict(kv_stride=1280, qo=A + 2192, ot=1280), ARG),                           # or into the next row's
    (dict(kv_stride=1280, qo=A + 1152, ot=1288), ARG),                           # or at another stride
    (dict(kv_stride=0x7000, q=E, qt=320, qh=64, qo=E + 368, ot=320, oh=64), ARG),
    (dict(latent=E), ARG), (dict(cache=G - 1152 * 9 * 16 + 16), ARG), (dict(qo=C), ARG),
])
def test_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status


def test_append_without_rotations(lib):
    """No page and no rotation: new tokens, which then have no row, would still be turned by the first."""
    assert _append(lib, batch=dict(table_width=0), rows=0) == UNSUP
    assert _append(lib, batch=dict(table_width=0, T=0), rows=0) == OK


def _attend(lib, batch=None, q=A, cache=B, dtype=0, scale=0, softmax=0.1, out=C, heads=3):
    return lib.skinny_latent_attention(_batch(**(batch or {})), q, cache, dtype, scale, softmax, out, heads, None)


@pytest.mark.parametrize("batch,status", BATCHES)
def test_attention_batch_refusals(lib, batch, status):
    assert _attend(lib, batch=batch) == status


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), ARG), (dict(softmax=0.0), ARG), (dict(softmax=-1.0), ARG), (dict(softmax=math.nan), ARG),
    (dict(softmax=math.inf), ARG), (dict(softmax=2.9e38), ARG), (dict(dtype=3), ARG), (dict(dtype=1), ARG), (dict(scale=D), ARG),
    (dict(heads=1025), UNSUP), (dict(batch=dict(T=1 << 22), heads=1024), UNSUP),
    (dict(q=0), ARG), (dict(cache=0), ARG), (dict(out=0), ARG),
    (dict(q=A + 8), ALIGN), (dict(cache=B + 1), ALIGN), (dict(out=C + 2), ALIGN), (dict(dtype=1, scale=D + 2), ALIGN),
    (dict(out=A), ARG), (dict(out=B + 16), ARG), (dict(out=G), ARG), (dict(out=H_ - 16), ARG), (dict(out=I_), ARG),
    (dict(dtype=1, scale=C + 16), ARG),
])
def test_attention_refusals(lib, kw, status):
    assert _attend(lib, **kw) == status


def _expanded(lib, q=A, kv=B, rope=C, stride=64, qs=D, ks=E, out=F, softmax=0.1, causal=1, n=2, T=5, S=9, heads=3):
    return lib.skinny_latent_attention_expanded(q, kv, rope, stride, qs, ks, out, softmax, causal, n, T, S, heads, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), ARG), (dict(T=-1), ARG), (dict(S=-1), ARG), (dict(heads=0), ARG), (dict(softmax=0.0), ARG),
    (dict(softmax=math.inf), ARG), (dict(softmax=2.9e38), ARG), (dict(causal=2), ARG), (dict(stride=56), ARG), (dict(stride=65), ARG),
    (dict(n=8193), UNSUP), (dict(heads=1025), UNSUP), (dict(stride=1 << 25), UNSUP), (dict(T=1 << 22, heads=1024), UNSUP),
    (dict(n=8192, heads=1024), UNSUP),
    (dict(T=0), OK), (dict(n=0), OK), (dict(T=0, q=0, kv=0, qs=0), OK),
    (dict(q=0), ARG), (dict(kv=0), ARG), (dict(rope=0), ARG), (dict(qs=0), ARG), (dict(ks=0), ARG), (dict(out=0), ARG),
    (dict(q=A + 8), ALIGN), (dict(kv=B + 2), ALIGN), (dict(rope=C + 8), ALIGN), (dict(out=F + 4), ALIGN), (dict(qs=D + 1), ALIGN),
    (dict(out=A), ARG), (dict(out=B), ARG), (dict(out=C), ARG), (dict(out=D), ARG), (dict(out=E - 16), ARG),
])
def test_expanded_refusals(lib, kw, status):
    assert _expanded(lib, **kw) == status


def _heads(lib, x=A, xt=96, xh=32, W=B, out=C, ot=48, oh=16, T=5, heads=3, N=16, K=32):
    return lib.skinny_heads_gemm(x, xt, xh, W, out, ot, oh, T, heads, N, K, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(heads=0), ARG), (dict(N=-8), ARG), (dict(K=-32), ARG), (dict(xt=100), ARG), (dict(oh=-16), ARG),
    (dict(heads=1025), UNSUP), (dict(K=0), UNSUP), (dict(K=48), UNSUP), (dict(K=544), UNSUP), (dict(N=12), UNSUP),
    (dict(N=1 << 20), UNSUP), (dict(xt=1 << 41), UNSUP), (dict(T=1 << 30, N=1024, ot=3 * 1024, oh=1024), UNSUP),
    (dict(T=0), OK), (dict(N=0), OK), (dict(T=0, x=0, W=0, out=0), OK),
    (dict(x=0), ARG), (dict(W=0), ARG), (dict(out=0), ARG), (dict(oh=8), ARG), (dict(ot=40), ARG),
    (dict(x=A + 8), ALIGN), (dict(W=B + 4), ALIGN), (dict(out=C + 2), ALIGN),
    (dict(out=A), ARG), (dict(out=B + 16), ARG),
    (dict(xt=144, xh=48, out=A + 48, ot=144, oh=48), ARG), (dict(xt=144, xh=48, out=A + 80, ot=144, oh=48), ARG),  # columns into others
    (dict(xt=152, xh=48, out=A + 64, ot=152, oh=48, N=40), ARG),
])
def test_heads_refusals(lib, kw, status):
    assert _heads(lib, **kw) == status


def test_reserve_refusals(lib):
    assert lib.skinny_latent_reserve(0, None) == ARG
    assert lib.skinny_latent_reserve(1025, None) == UNSUP


def test_binding_takes_no_host_tensors():
    """Tensors that are not on a device, before anything else is looked at."""
    z = torch.zeros
    b = torch.bfloat16
    with pytest.raises(ValueError, match="device"):
        skg.latent_append(z(1, 576, dtype=b), z(1, 8, 576, dtype=b), z(1, 1, dtype=torch.int32), z(1, dtype=torch.int32), z(8, 64))
    with pytest.raises(ValueError, match="device"):
        skg.latent_attention(z(1, 2, 576, dtype=b), z(1, 8, 576, dtype=b), z(1, 1, dtype=torch.int32), z(1, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="device"):
        skg.latent_attention_expanded(z(1, 2, 192, dtype=b), z(1, 2, 256, dtype=b), z(1, 64, dtype=b), z(2, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="device"):
        skg.heads_gemm(z(1, 2, 32, dtype=b), z(2, 8, 32, dtype=b))


# ------------------------------------------------------------ the plain implementations

def test_rounding_against_torch():
    x = torch.randn(20000, generator=torch.Generator().manual_seed(0)) * torch.exp2(torch.randint(-12, 9, (20000,), generator=torch.Generator().manual_seed(1)).float())
    assert torch.equal(ref.to_bf16(x.double()), x.bfloat16())
    assert torch.equal(ref.to_e4m3(x.double()).view(torch.uint8), x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    # a tie of bf16 that fp32 cannot tell from its neighbour
    t = torch.tensor([1 + 2.0 ** -8 + 2.0 ** -40, 1 + 2.0 ** -8, 1 - 2.0 ** -9 - 2.0 ** -45], dtype=torch.float64)
    assert ref.to_bf16(t).double().tolist() == [1 + 2.0 ** -7, 1.0, 1 - 2.0 ** -8]


def test_attention_forms_agree():
    """The absorbed form over a paged cache is the expanded one with the keys and values that the latents stand for."""
    g = torch.Generator().manual_seed(3)
    H, n, m = 2, 3, 40
    wk, wv = torch.randn(H, 512, 128, generator=g).double() / 20, torch.randn(H, 128, 512, generator=g).double() / 20
    rows = torch.randn(m, 576, generator=g).bfloat16()
    q = torch.randn(n, H, 192, generator=g).double()
    keys = torch.cat((torch.einsum("ml,hld->mhd", rows[:, :512].double(), wk), rows[:, None, 512:].double().expand(-1, H, -1)), -1)
    values = torch.einsum("ml,hdl->mhd", rows[:, :512].double(), wv)
    seen = torch.arange(m)[None] <= torch.arange(m - n, m)[:, None]
    want, _ = ref.softmax_rows(q, keys, values, seen, 0.07)
    ql = torch.cat((torch.einsum("nhd,hld->nhl", q[..., :128], wk), q[..., 128:]), -1)
    cache = torch.zeros(6, 8, 576, dtype=torch.bfloat16)
    table = torch.tensor([[5, 0, 3, 1, 2]], dtype=torch.int32)
    cache[table[0].long()] = rows.reshape(5, 8, 576)
    o, _ = ref.attention(ql, cache, None, table, [m], [0, n], 0.07)
    got = torch.einsum("nhl,hdl->nhd", o, wv)
    assert (got - want).abs().max() < 1e-12


def test_softmax_rows_against_torch():
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(*s, generator=g).double() for s in ((5, 3, 192), (9, 3, 192), (9, 3, 128)))
    seen = torch.arange(9)[None] <= torch.arange(4, 9)[:, None]
    got, bound = ref.softmax_rows(q, k, v, seen, 0.1)
    s = torch.einsum("nhd,mhd->hnm", q, k) * 0.1
    w = torch.softmax(s.masked_fill(~seen[None], -math.inf), -1)
    assert (got - torch.einsum("hnm,mhe->nhe", w, v)).abs().max() < 1e-13
    assert (bound > 0).all()
