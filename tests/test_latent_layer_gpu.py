"""The operators of skinny_latent.h run together, on other streams, in graphs,
over caches past 4 GiB, and what the binding refuses of device tensors."""
import importlib.util
import os

import pytest
import torch

import latency_skinny_gemm_amd as pkg
from tests import latent_reference as ref
from tests.test_latent_gpu import DEV, SCALE, _cache, _dev, _ints, _randn, _starts, skg  # noqa: F401

pytestmark = pytest.mark.gpu


def _block(**k):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_layer.py")
    spec = importlib.util.spec_from_file_location("latent_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    torch.manual_seed(5)
    return mod.LatentBlock(**k)


def _plain(block, x, lens):
    """The block's outputs for whole sequences in 64 bits, from its bf16 weights."""
    w = {k: getattr(block, k).cpu().double() for k in ("wq", "wkv", "gain", "up", "wo")}
    rot, H = block.rotations.cpu(), block.heads
    outs, at = [], 0
    for n in lens:
        xs = x[at:at + n].double()
        at += n
        q = (xs @ w["wq"].T).view(n, H, 192)
        kv = xs @ w["wkv"].T
        c = kv[:, :512]
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-6) * w["gain"]
        r = torch.stack([ref.rotate(kv[t, 512:], rot[t], "pairs") for t in range(n)])
        qr = torch.stack([ref.rotate(q[t, :, 128:], rot[t], "pairs") for t in range(n)])
        up = torch.einsum("hnk,tk->thn", w["up"], c)
        s = (torch.einsum("thd,shd->hts", q[..., :128], up[..., :128]) + torch.einsum("thd,sd->hts", qr, r)) * block.softmax_scale
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), float("-inf"))
        o = torch.einsum("hts,shd->thd", torch.softmax(s, -1), up[..., 128:])
        outs.append(o.reshape(n, H * 128) @ w["wo"].T)
    return torch.cat(outs)


# Roundings to bf16 between x and the output, each at most 2^-8 of its value: latents and
# queries, the row, keys, values, weights, the attention's output, the block's.  Scores are
# of order 1, so that a rounding of what makes them moves a weight by about as much.  In
# the norm at most their sum, 8 of them (e4m3 rows: one of 2^-4 more in keys and in values).
NORM = 8 * 2.0 ** -8
NORM_E4M3 = NORM + 2 * 2.0 ** -4


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompts_then_single_tokens(skg, e4m3):  # noqa: F811
    """Prompts in the expanded form, the same tokens again in the absorbed form, then steps of one
    token, against 64 bits; the steps as a graph, replayed with eager work between."""
    lens, more, page = [37, 1, 90], 4, 16
    block = _block(hidden=320, heads=5, pages=40, page_size=page, width=8, e4m3=e4m3)
    full = [n + more for n in lens]
    xs = [(0.7 * _randn(40 + i, n, 320)).bfloat16() for i, n in enumerate(full)]
    want = _plain(block, torch.cat(xs), full).split(full)
    table = torch.randperm(40, generator=torch.Generator().manual_seed(3))[:24].view(3, 8).to(torch.int32).to(DEV)
    first = torch.cat([x[:n] for x, n in zip(xs, lens)]).to(DEV)
    starts, kv_lens = _starts(lens).to(DEV), _ints(lens).to(DEV)
    got = block.prompt(first, starts, table, kv_lens).cpu().double()
    whole = torch.cat([w[:n] for w, n in zip(want, lens)])
    assert torch.linalg.norm(got - whole) <= NORM * torch.linalg.norm(whole)

    # the prompts' last tokens again, their queries absorbed, over the cache's rows
    T = len(first)
    q = skg.gemm_bf16(first, block.wq).view(T, 5, 192)
    qa = torch.empty(T, 5, 576, dtype=torch.bfloat16, device=DEV)
    skg.latent_append(skg.gemm_bf16(first, block.wkv), block.cache, table, kv_lens, block.rotations, q_starts=starts,
                      weight=block.gain, scale=block.scale, q_rope=q[..., 128:], q_rope_out=qa[..., 512:])
    skg.heads_gemm(q[..., :128], block.absorb, out=qa[..., :512])
    o = skg.latent_attention(qa, block.cache, table, kv_lens, block.softmax_scale, q_starts=starts, scale=block.scale)
    again = skg.gemm_bf16(skg.heads_gemm(o, block.values).view(T, 640), block.wo).cpu().double()
    assert torch.linalg.norm(again - whole) <= (NORM_E4M3 if e4m3 else NORM) * torch.linalg.norm(whole)

    # steps: eager, and as a graph whose tokens and lengths change
    x = torch.empty(3, 320, dtype=torch.bfloat16, device=DEV)
    now = kv_lens.clone()
    graph, out = block.capture(x, table, now)
    for i in range(more):
        x.copy_(torch.stack([s[n + i] for s, n in zip(xs, lens)]))
        now.add_(1)
        eager = block.step(x, table, now).clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i
        w = torch.stack([s[n + i] for s, n in zip(want, lens)])
        assert torch.linalg.norm(out.cpu().double() - w) <= (NORM_E4M3 if e4m3 else NORM) * torch.linalg.norm(w), i


def test_the_example_runs():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_layer.py")
    spec = importlib.util.spec_from_file_location("latent_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.main(["--sequences", "1", "3", "--length", "200", "--hidden", "256", "--heads", "4", "--e4m3"])


# ------------------------------------------------------------ streams and graphs

def _absorbed(seed, lens, H, page=64, e4m3=False):
    cache, scale, table = _cache(seed, lens, page, e4m3)
    q = _randn(seed + 1, len(lens), H, 576).bfloat16()
    return _dev(q, cache, table, _ints(lens)), None if scale is None else scale.to(DEV)


def _expanded(seed, n, m, H):
    q, kv, kr = _randn(seed, n, H, 192).bfloat16(), _randn(seed + 1, m, H, 256).bfloat16(), _randn(seed + 2, m, 64).bfloat16()
    return _dev(q, kv, kr, _ints([0, n]), _ints([0, m]))


def test_streams(skg):  # noqa: F811
    """As the argument and as the current one, two at once: each has its own workspace."""
    (q, c, t, n), _ = _absorbed(1, [1500, 700, 3000], 16)
    eq, ekv, ekr, qs, ks = _expanded(2, 40, 2000, 3)
    want = skg.latent_attention(q, c, t, n, SCALE)
    ewant = skg.latent_attention_expanded(eq, ekv, ekr, qs, SCALE, kv_starts=ks)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got, egot = [], []
    for i in range(6):
        s = side[i & 1]
        with torch.cuda.stream(s):
            got.append(skg.latent_attention(q, c, t, n, SCALE))
            egot.append(skg.latent_attention_expanded(eq, ekv, ekr, qs, SCALE, kv_starts=ks))
        out, eout = torch.empty_like(want), torch.empty_like(ewant)
        torch.cuda.synchronize()
        got.append(skg.latent_attention(q, c, t, n, SCALE, out=out, stream=s))
        egot.append(skg.latent_attention_expanded(eq, ekv, ekr, qs, SCALE, kv_starts=ks, out=eout, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got) and all(torch.equal(o, ewant) for o in egot)


def test_two_graphs_of_one_stream(skg):  # noqa: F811
    """Captured on one stream they share its workspace: replayed there in turn, with eager work between."""
    (q, c, t, n), _ = _absorbed(3, [900, 2500], 128)
    eq, ekv, ekr, qs, ks = _expanded(4, 100, 3000, 2)
    cap = torch.cuda.Stream()
    skg.reserve_latent(128, stream=cap)
    cap.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.stream(cap):
        with torch.cuda.graph(graphs[0], stream=cap):
            a = skg.latent_attention(q, c, t, n, SCALE)
        with torch.cuda.graph(graphs[1], stream=cap):
            b = skg.latent_attention_expanded(eq, ekv, ekr, qs, SCALE, kv_starts=ks)
    for i in range(4):
        q.copy_(_randn(20 + i, *q.shape).bfloat16())
        eq.copy_(_randn(30 + i, *eq.shape).bfloat16())
        n.copy_(_ints([900 - 300 * i, 2500 - 7 * i]))
        want = skg.latent_attention(q, c, t, n, SCALE)
        ewant = skg.latent_attention_expanded(eq, ekv, ekr, qs, SCALE, kv_starts=ks)
        torch.cuda.synchronize()
        with torch.cuda.stream(cap):
            graphs[i & 1].replay()
            graphs[1 - (i & 1)].replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, ewant), i


def test_first_call_of_a_kernel_in_a_graph(skg):  # noqa: F811
    """A depth that nothing else here takes: its kernel is loaded while the graph is captured."""
    x, w = _randn(70, 100, 2, 448).bfloat16().to(DEV)[..., :384], (_randn(71, 2, 128, 384) / 20).bfloat16().to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = skg.heads_gemm(x, w)
    for i in range(3):
        x.copy_(_randn(72 + i, 100, 2, 384).bfloat16())
        want = skg.heads_gemm(x, w)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_capture_needs_reserved_workspace(skg):  # noqa: F811
    (q, c, t, n), _ = _absorbed(5, [100], 16)
    eq, ekv, ekr, qs, ks = _expanded(6, 10, 1000, 2)
    out, eout = torch.empty(1, 16, 512, dtype=torch.bfloat16, device=DEV), torch.empty(10, 2, 128, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(skg.SkinnyGemmError) as err:
                skg.latent_attention(q, c, t, n, SCALE, out=out)
            assert err.value.status == skg.ERR_WORKSPACE
            with pytest.raises(skg.SkinnyGemmError) as err:
                skg.latent_attention_expanded(eq, ekv, ekr, qs, SCALE, kv_starts=ks, out=eout)
            assert err.value.status == skg.ERR_WORKSPACE


# ------------------------------------------------------------ large and odd layouts

@pytest.mark.parametrize("page", [8, 32, 1024, 65536])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_of_all_sizes(skg, page, e4m3):  # noqa: F811
    lens, H = [70, 33], 20
    cache, scale, table = _cache(7, lens, page, e4m3, spare=1)
    q = _randn(8, 2, H, 576).bfloat16()
    out, bound = ref.attention(q, cache, scale, table, lens, None, SCALE)
    got = skg.latent_attention(*_dev(q, cache, table, _ints(lens)), SCALE, scale=None if scale is None else scale.to(DEV))
    ref.check(got, out, bound)


@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_past_32_bits(skg, e4m3):  # noqa: F811
    """Rows more than 4 GiB behind the cache's start: the bits of a small cache."""
    page, H, lens = 64, 16, [200, 65]
    row = 576 * (1 if e4m3 else 2)
    pages = (2 ** 32 + 2 ** 28) // (page * row)
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    big = torch.empty(pages, page, 576, dtype=dtype, device=DEV)
    small = torch.zeros(6, page, 576, dtype=dtype, device=DEV)
    far = [pages - 1, 5, pages - 3, pages // 2 + 7, pages - 8, 2 ** 31 // (page * row)]
    near = list(range(6))
    kv, q = _randn(9, sum(lens), 576).bfloat16().to(DEV), _randn(10, 2, H, 576).bfloat16().to(DEV)
    scale = torch.full((1,), 0.05, device=DEV) if e4m3 else None
    rot = ref.rotation_rows(4 * page).to(DEV)
    outs = []
    for cache, at in ((big, far), (small, near)):
        table = _ints([at[:4], at[4:] + [-1, -1]]).to(DEV)
        n = _ints(lens).to(DEV)
        skg.latent_append(kv, cache, table, n, rot, q_starts=_starts(lens).to(DEV), scale=scale)
        outs.append(skg.latent_attention(q, cache, table, n, SCALE, scale=scale))
    assert torch.equal(*outs)
    for f, n in zip(far[:3] + [far[4]], near[:3] + [near[4]]):
        assert torch.equal(big[f].view(torch.uint8), small[n].view(torch.uint8))
    w, _, _ = ref.append(kv.cpu(), None, 1e-6, rot.cpu(), "pairs", torch.zeros_like(small).cpu(), None if scale is None else scale.cpu(),
                         _ints([near[:4], near[4:] + [-1, -1]]), lens, _starts(lens).tolist(), None)
    assert torch.equal(w.view(torch.uint8), small.cpu().view(torch.uint8))


def test_expanded_keys_past_32_bits(skg):  # noqa: F811
    H, S, n, m = 128, 70000, 3, 90
    kv = torch.empty(S, H, 256, dtype=torch.bfloat16, device=DEV)
    kr = torch.empty(S, 64, dtype=torch.bfloat16, device=DEV)
    tail, tr, q = _randn(11, m, H, 256).bfloat16(), _randn(12, m, 64).bfloat16(), _randn(13, n, H, 192).bfloat16()
    kv[S - m:], kr[S - m:] = tail.to(DEV), tr.to(DEV)
    got = skg.latent_attention_expanded(q.to(DEV), kv, kr, _ints([0, n]).to(DEV), SCALE, kv_starts=_ints([S - m, S]).to(DEV))
    out, bound = ref.expanded(q, tail, tr, [0, n], [0, m], SCALE, True)
    ref.check(got, out, bound)


@pytest.mark.parametrize("T", [3, 70, 200])
def test_heads_past_32_bits(skg, T):  # noqa: F811
    """Strides from token to token that leave 4 GiB behind, of x and of the output."""
    H, N, K = 2, 40, 128
    step = (2 ** 31 + 2 ** 28) // (T - 1) // 8 * 8  # values
    store = torch.empty(step * (T - 1) + H * K, dtype=torch.bfloat16, device=DEV)
    x, w = _randn(14, T, H, K).bfloat16(), (_randn(15, H, N, K) / 11).bfloat16()
    far = store.as_strided((T, H, K), (step, K, 1))
    far.copy_(x)
    want = skg.heads_gemm(x.to(DEV), w.to(DEV))
    assert torch.equal(skg.heads_gemm(far, w.to(DEV)), want)
    out = store.as_strided((T, H, N), (step, N, 1))
    skg.heads_gemm(x.to(DEV), w.to(DEV), out=out)
    assert torch.equal(out, want)


# ------------------------------------------------------------ nothing to do, and refusals

@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("H", [1, 3])
def test_columns_of_one_matrix(skg, T, H):  # noqa: F811
    """Inputs and outputs that are slices of one projection's output: the same values as apart, the rest untouched."""
    cache, _, table = _cache(60, [9] * T, 8, False)
    cd, td, lens, rot = cache.to(DEV), table.to(DEV), _ints([9] * T).to(DEV), ref.rotation_rows(16).to(DEV)
    m = _randn(61, T, H * 192 + 576).bfloat16().to(DEV)
    q, kv = m[:, :H * 192].unflatten(1, (H, 192)), m[:, H * 192:]
    apart = skg.latent_append(kv.clone(), cd.clone(), td, lens, rot, q_rope=q[..., 128:].clone(), latent=True)
    before = m.clone()
    got = skg.latent_append(kv, cd, td, lens, rot, q_rope=q[..., 128:], q_rope_out=q[..., 128:], latent=True)
    assert torch.equal(got.latent, apart.latent) and torch.equal(q[..., 128:], apart.q_rope)
    before[:, :H * 192].unflatten(1, (H, 192))[..., 128:] = apart.q_rope
    assert torch.equal(m, before)
    # a head's 128 values, and its 512 latent ones behind them
    both = _randn(62, T, H, 640).bfloat16().to(DEV)
    w = _randn(63, H, 512, 128).bfloat16().to(DEV)
    x, before = both[..., :128], both.clone()
    want = skg.heads_gemm(x.clone(), w)
    skg.heads_gemm(x, w, out=both[..., 128:])
    assert torch.equal(both[..., 128:], want) and torch.equal(x, before[..., :128])
    # all heads' inputs, then all heads' outputs
    row = _randn(64, T, H * 640).bfloat16().to(DEV)
    x, out = row[:, :H * 128].unflatten(1, (H, 128)), row[:, H * 128:].unflatten(1, (H, 512))
    want = skg.heads_gemm(x.clone(), w)
    skg.heads_gemm(x, w, out=out)
    assert torch.equal(out, want)
    with pytest.raises(skg.SkinnyGemmError):  # one piece into the inputs
        skg.heads_gemm(both[..., :128], w, out=both[..., 120:632])


def test_nothing_to_do(skg):  # noqa: F811
    cache = torch.zeros(2, 8, 576, dtype=torch.bfloat16, device=DEV)
    e = dict(dtype=torch.bfloat16, device=DEV)
    none, one = _ints([]).to(DEV), _ints([0]).to(DEV)
    rot = ref.rotation_rows(8).to(DEV)
    table = torch.empty(0, 1, dtype=torch.int32, device=DEV)
    skg.latent_append(torch.empty(0, 576, **e), cache, table, none, rot, q_rope=torch.empty(0, 4, 64, **e))
    assert skg.latent_attention(torch.empty(0, 4, 576, **e), cache, table, none, SCALE).shape == (0, 4, 512)
    assert skg.latent_attention_expanded(torch.empty(0, 4, 192, **e), torch.empty(0, 4, 256, **e), torch.empty(0, 64, **e), one, SCALE).shape == (0, 4, 128)
    assert skg.heads_gemm(torch.empty(0, 4, 64, **e), torch.empty(4, 8, 64, **e)).shape == (0, 4, 8)
    # tokens of no sequence: outputs stay; no keys at all: zeros
    out = torch.full((3, 4, 128), 2.0, **e)
    skg.latent_attention_expanded(torch.ones(3, 4, 192, **e), torch.empty(0, 4, 256, **e), torch.empty(0, 64, **e), _ints([0, 2]).to(DEV), SCALE,
                                  kv_starts=_ints([0, 0]).to(DEV), out=out)
    assert (out[:2] == 0).all() and (out[2] == 2.0).all()


def test_refusals(skg):  # noqa: F811
    (q, c, t, n), _ = _absorbed(16, [20, 9], 4)
    e = dict(dtype=torch.bfloat16, device=DEV)
    rot = ref.rotation_rows(64).to(DEV)
    kv = torch.zeros(2, 576, **e)
    one = torch.ones(1, device=DEV)

    def no(error, f, *a, **k):
        with pytest.raises(error):
            f(*a, **k)

    attend, append, expanded, heads = skg.latent_attention, skg.latent_append, skg.latent_attention_expanded, skg.heads_gemm
    no(TypeError, attend, q.float(), c, t, n, SCALE)
    no(ValueError, attend, q.cpu(), c, t, n, SCALE)
    no(ValueError, attend, q[..., :512], c, t, n, SCALE)
    no(ValueError, attend, q.transpose(0, 1), c, t, n, SCALE)
    no(ValueError, attend, q, c, t, n, SCALE, scale=one)                       # a scale without codes
    no(ValueError, attend, q, c.to(torch.float8_e4m3fn), t, n, SCALE)          # and codes without one
    no(ValueError, attend, q, c[:, ::2], t, n, SCALE)
    no(ValueError, attend, q, c[..., :512], t, n, SCALE)
    no(TypeError, attend, q, c, t.long(), n, SCALE)
    no(ValueError, attend, q, c, t, n[:1], SCALE)
    no(ValueError, attend, q[:1], c, t, n, SCALE)                              # one token a sequence
    no(ValueError, attend, q, c, t, n, SCALE, q_starts=n)
    no(ValueError, attend, q, c, t, n, SCALE, out=q[..., :512])
    no(skg.SkinnyGemmError, attend, q, c, t, n, 0.0)
    no(skg.SkinnyGemmError, attend, q, c, t, n, float("nan"))
    flat = torch.zeros(4 * 2 * 576, **e)
    no(skg.SkinnyGemmError, attend, flat.view(2, 4, 576), c, t, n, SCALE, out=flat[:2 * 4 * 512].view(2, 4, 512))
    no(ValueError, append, kv, c, t, n, rot, rope="both")
    no(skg.SkinnyGemmError, append, kv, c, t, n, rot[:32])                     # fewer rotations than rows
    no(skg.SkinnyGemmError, append, kv, c, t, n, rot, eps=-1.0)
    no(ValueError, append, kv, c, t, n, rot, q_rope_out=torch.empty(2, 4, 64, **e))
    no(ValueError, append, kv, c, t, n, rot, weight=torch.ones(511, **e))
    odd = torch.zeros(2 * 580, **e).as_strided((2, 576), (580, 1))
    no(skg.SkinnyGemmError, append, odd, c, t, n, rot)
    q2, kv2, kr2, s2 = torch.zeros(3, 4, 192, **e), torch.zeros(3, 4, 256, **e), torch.zeros(3, 64, **e), _ints([0, 3]).to(DEV)
    no(ValueError, expanded, q2[..., :191], kv2, kr2, s2, SCALE)
    no(ValueError, expanded, q2, kv2[:, :3], kr2, s2, SCALE)
    no(ValueError, expanded, q2, kv2, kr2[:2], s2, SCALE)
    no(ValueError, expanded, q2, kv2, kr2, s2, SCALE, kv_starts=s2[:1])
    no(skg.SkinnyGemmError, expanded, q2, kv2, kr2, s2, -1.0)
    x, w = torch.zeros(3, 4, 64, **e), torch.zeros(4, 8, 64, **e)
    no(ValueError, heads, x, w[:3])
    no(ValueError, heads, x[..., :32], w)
    no(ValueError, heads, x.transpose(1, 2), w)
    no(skg.SkinnyGemmError, heads, torch.zeros(3, 4, 40, **e), torch.zeros(4, 8, 40, **e))
    no(skg.SkinnyGemmError, heads, x, torch.zeros(4, 12, 64, **e))
    out = torch.zeros(3, 1, 8, **e).expand(3, 4, 8)                            # heads on one another
    no(skg.SkinnyGemmError, heads, x, w, out=out)
    no(skg.SkinnyGemmError, skg.reserve_latent, 0)


def test_the_package_has_them():
    for name in ("latent_append", "latent_attention", "latent_attention_expanded", "heads_gemm", "reserve_latent"):
        assert callable(getattr(pkg, name))


# ------------------------------------------------------------ the largest batches and head counts

def test_largest_batch(skg):  # noqa: F811
    """8192 sequences: appended to and read, one token each, and a few of several."""
    B, page = 8192, 8
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 2 * page + 3, (B,), generator=g).tolist()
    cache, _, table = _cache(23, [2 * page] * B, page, False, spare=1)
    kv, q = _randn(24, B, 576).bfloat16(), _randn(25, B, 1, 576).bfloat16()
    rot = ref.rotation_rows(2 * page)
    n = _ints(lens).to(DEV)
    cd, td = _dev(cache, table)
    skg.latent_append(kv.to(DEV), cd, td, n, rot.to(DEV))
    want, _, _ = ref.append(kv, None, 1e-6, rot, "pairs", cache, None, table, lens, None, None)
    assert torch.equal(cd.cpu().view(torch.int16), want.view(torch.int16))
    out, bound = ref.attention(q, want, None, table, lens, None, SCALE)
    ref.check(skg.latent_attention(q.to(DEV), cd, td, n, SCALE), out, bound)
    # most of them without a token
    counts = [0] * B
    for b in (0, 1, 4000, 8191):
        counts[b], lens[b] = 3, 9
    starts = _starts(counts)
    few, fq = _randn(26, 12, 576).bfloat16(), _randn(27, 12, 2, 576).bfloat16()
    n = _ints(lens).to(DEV)
    skg.latent_append(few.to(DEV), cd, td, n, rot.to(DEV), q_starts=starts.to(DEV))
    want, _, _ = ref.append(few, None, 1e-6, rot, "pairs", want, None, table, lens, starts.tolist(), None)
    assert torch.equal(cd.cpu().view(torch.int16), want.view(torch.int16))
    out, bound = ref.attention(fq, want, None, table, lens, starts.tolist(), SCALE)
    ref.check(skg.latent_attention(fq.to(DEV), cd, td, n, SCALE, q_starts=starts.to(DEV)), out, bound)


@pytest.mark.parametrize("e4m3", [False, True])
def test_most_heads(skg, e4m3):  # noqa: F811
    H, lens, counts = 1024, [70, 33], [1, 2]
    cache, scale, table = _cache(28, lens, 16, e4m3)
    q = _randn(29, 3, H, 576).bfloat16()
    starts = _starts(counts)
    out, bound = ref.attention(q, cache, scale, table, lens, starts.tolist(), SCALE)
    sd = None if scale is None else scale.to(DEV)
    ref.check(skg.latent_attention(*_dev(q, cache, table, _ints(lens)), SCALE, q_starts=starts.to(DEV), scale=sd), out, bound)
    if e4m3:
        return
    eq, ekv, ekr = _randn(30, 3, H, 192).bfloat16(), _randn(31, 40, H, 256).bfloat16(), _randn(32, 40, 64).bfloat16()
    out, bound = ref.expanded(eq, ekv, ekr, [0, 3], [0, 40], SCALE, True)
    ref.check(skg.latent_attention_expanded(*_dev(eq, ekv, ekr, _ints([0, 3])), SCALE, kv_starts=_ints([0, 40]).to(DEV)), out, bound)
    x, w = _randn(33, 5, H, 64).bfloat16(), (_randn(34, H, 16, 64) / 8).bfloat16()
    out, bound = ref.heads(x, w)
    ref.check(skg.heads_gemm(*_dev(x, w)), out, bound)
    kv, qr = _randn(35, 3, 576).bfloat16(), _randn(36, 3, H, 64).bfloat16()
    rot = ref.rotation_rows(table.shape[1] * 16)
    got = skg.latent_append(kv.to(DEV), cache.to(DEV), table.to(DEV), _ints(lens).to(DEV), rot.to(DEV), q_starts=starts.to(DEV), q_rope=qr.to(DEV)).q_rope
    _, _, want = ref.append(kv, None, 1e-6, rot, "pairs", cache, None, table, lens, starts.tolist(), qr)
    ref.check(got, want, 1.01 * 2.0 ** -8 * want.abs() + 2.0 ** -22 * qr.double().abs().amax())  # two fp32 products and their sum, one rounding
