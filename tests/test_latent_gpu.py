"""The operators of skinny_latent.h on the GPU against plain implementations in
64 bits (tests/latent_reference.py, which derives the bounds), through the Python
binding.  Cache rows and codes are decided exactly on both sides: bit for bit."""
import math

import pytest
import torch

from tests import latent_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SCALE = 192 ** -0.5


@pytest.fixture(scope="module")
def skg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import latency_skinny_gemm_amd as m
    m.lib()
    return m


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32)


def _starts(counts):
    s = [0]
    for c in counts:
        s.append(s[-1] + c)
    return _ints(s)


def _cache(seed, lens, page, e4m3, spare=3, width=None):
    """A cache in pages of random order, scale, table."""
    W = max([1] + [-(-n // page) for n in lens]) if width is None else width
    B = len(lens)
    pages = B * W + spare
    g = torch.Generator().manual_seed(seed + 1)
    table = torch.randperm(pages, generator=g)[:B * W].reshape(B, W).to(torch.int32)
    v = _randn(seed, pages, page, 576)
    scale = torch.tensor([0.05]) if e4m3 else None
    cache = (v / 0.05).clamp(-448, 448).to(torch.float8_e4m3fn) if e4m3 else v.bfloat16()
    return cache, scale, table


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


# ------------------------------------------------------------ append

APPENDS = [
    # counts, lens after, heads, page, style, latent, weight
    ([1], [1], 1, 8, "pairs", True, True),
    ([1], [37], 128, 64, "pairs", False, True),
    ([1, 1, 1], [9, 64, 65], 16, 16, "halves", True, True),
    ([5, 0, 1, 17], [5, 3, 8, 40], 3, 16, "pairs", True, False),
    ([70, 3], [200, 3], 20, 64, "halves", True, True),
    ([33] * 9, [33] * 9, 0, 32, "pairs", False, True),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("counts,lens,H,page,style,latent,weighted", APPENDS)
def test_append(skg, counts, lens, H, page, style, latent, weighted, e4m3):
    T = sum(counts)
    seed = 100 * T + H
    single = all(c == 1 for c in counts)
    starts = None if single else _starts(counts)
    cache, scale, table = _cache(seed, lens, page, e4m3)
    kv = (_randn(seed + 2, T, 600) * 3).bfloat16()
    weight = (1 + 0.2 * _randn(seed + 3, 512)).bfloat16() if weighted else None
    q = _randn(seed + 4, T, H, 192).bfloat16() if H else None
    rot = ref.rotation_rows(table.shape[1] * page)
    want, lat, qo = ref.append(kv[:, 24:], weight, 1e-6, rot, style, cache, scale, table, lens,
                               None if single else starts.tolist(), None if q is None else q[..., 128:])
    kd, wd, qd, rd, cd, sd, td, ld, pd = _dev(kv, weight, q, rot, cache, scale, table, _ints(lens), starts)
    got = skg.latent_append(kd[:, 24:], cd, td, ld, rd, q_starts=pd, weight=wd, rope=style, scale=sd,
                            q_rope=None if q is None else qd[..., 128:], latent=latent)
    assert torch.equal(cd.cpu().view(torch.uint8), want.view(torch.uint8))
    assert (got.latent is not None) == latent and (got.q_rope is not None) == (q is not None)
    if latent:
        assert torch.equal(got.latent.cpu(), ref.to_bf16(lat))
    if q is not None:
        # two products and a sum in fp32, then bf16
        size = (2 * q[..., 128:].double() ** 2).sum(-1, keepdim=True).sqrt()
        ref.check(got.q_rope, qo, 1.01 * 2.0 ** -8 * qo.abs() + 2.0 ** -22 * size)
        # in place, with the strides it has
        skg.latent_append(kd[:, 24:], cd, td, ld, rd, q_starts=pd, weight=wd, rope=style, scale=sd,
                          q_rope=qd[..., 128:], q_rope_out=qd[..., 128:])
        assert torch.equal(qd[..., 128:], got.q_rope)
        assert torch.equal(qd[..., :128].cpu(), q[..., :128])


def test_append_ends_of_the_types(skg):
    """Codes past 448, zeros, infinities and NaN, a row of zeros (eps alone), and huge values."""
    T = 5
    kv = _randn(1, T, 576)
    kv[0] *= 1e4
    kv[1] = 0.0
    kv[2, 3] = math.inf
    kv[3, 520] = math.nan
    kv[4] *= 1e30
    kv = kv.bfloat16()
    cache, scale, table = _cache(2, [T], 8, True)
    rot = ref.rotation_rows(8)
    want, lat, _ = ref.append(kv, None, 0.0, rot, "pairs", cache, scale, table, [T], [0, T], None)
    cd, td, sd = _dev(cache, table, scale)
    skg.latent_append(kv.to(DEV), cd, td, _ints([T]).to(DEV), rot.to(DEV), q_starts=_ints([0, T]).to(DEV), scale=sd)
    assert torch.equal(torch.nan_to_num(cd.cpu().float(), nan=1e9), torch.nan_to_num(want.float(), nan=1e9))
    weight = torch.ones(512).bfloat16()
    for row, w in ((0, weight), (1, weight), (4, weight)):
        one = kv[row:row + 1]
        c2, s2, t2 = _cache(3, [1], 8, False)
        want, lat, _ = ref.append(one, w, 1e-6, rot, "pairs", c2, None, t2, [1], None, None)
        cd, td = _dev(c2, t2)
        skg.latent_append(one.to(DEV), cd, td, _ints([1]).to(DEV), rot.to(DEV), weight=w.to(DEV))
        assert torch.equal(cd.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("scale", [math.inf, 0.0, 2.0 ** -149, -0.05, 3.0, math.nan])
def test_append_odd_scales(skg, scale):
    kv = _randn(21, 4, 576)
    kv[1] = 0.0
    kv[2, 5] = math.inf
    kv = kv.bfloat16()
    cache, _, table = _cache(22, [4], 8, True)
    rot, s = ref.rotation_rows(8), torch.tensor([scale])
    want, _, _ = ref.append(kv, None, 0.0, rot, "halves", cache, s, table, [4], [0, 4], None)
    cd, td, sd = _dev(cache, table, s)
    skg.latent_append(kv.to(DEV), cd, td, _ints([4]).to(DEV), rot.to(DEV), q_starts=_ints([0, 4]).to(DEV), scale=sd, rope="halves")
    got, want = cd.cpu().float(), want.float()
    assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want, nan=1e9))


def test_append_where_there_is_no_row(skg):
    """Pages outside the cache, tokens before row 0, lengths past the table, tokens behind the last sequence."""
    page, H = 8, 2
    counts, lens = [3, 2, 4, 1], [2, 8, 1000, 0]
    T = sum(counts) + 5
    cache, _, table = _cache(4, [16] * 4, page, False, width=2)
    table[1, 0] = -1
    table[2, 1] = cache.shape[0]
    kv, q = _randn(5, T, 576).bfloat16(), _randn(6, T, H, 64).bfloat16()
    rot = ref.rotation_rows(2 * page)
    starts = _starts(counts)
    want, lat, qo = ref.append(kv, None, 1e-6, rot, "pairs", cache, None, table, lens, starts.tolist(), q)
    cd, td, kd, qd = _dev(cache, table, kv, q)
    before = torch.full((T, H, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    got = skg.latent_append(kd, cd, td, _ints(lens).to(DEV), rot.to(DEV), q_starts=starts.to(DEV), q_rope=qd,
                            q_rope_out=before, latent=True)
    assert torch.equal(cd.cpu().view(torch.int16), want.view(torch.int16))
    n = sum(counts)
    assert torch.equal(got.latent[:n].cpu(), ref.to_bf16(lat[:n]))
    assert (got.q_rope[n:] == 7.0).all()


# ------------------------------------------------------------ absorbed form

DECODES = [
    # lens, heads, page
    ([1], 1, 8),
    ([31], 128, 16),
    ([33, 64, 1, 200], 16, 64),
    ([0, 5, 0], 20, 32),
    ([700], 128, 64),
    ([97, 3, 512, 1000, 40], 33, 16),
    ([500, 130], 64, 256),
    ([40], 129, 64),
]


def _attention_case(skg, counts, lens, H, page, e4m3, seed, single=None, qscale=1.2, table=None):
    T = sum(counts)
    single = all(c == 1 for c in counts) if single is None else single
    starts = None if single else _starts(counts)
    cache, scale, made = _cache(seed, lens, page, e4m3)
    table = made if table is None else table
    q = (qscale * _randn(seed + 7, T, H, 576)).bfloat16()
    out, bound = ref.attention(q, cache, scale, table, lens, None if single else starts.tolist(), SCALE)
    qd, cd, sd, td, ld, pd = _dev(q, cache, scale, table, _ints(lens), starts)
    got = skg.latent_attention(qd, cd, td, ld, SCALE, q_starts=pd, scale=sd)
    ref.check(got, out, bound)
    again = skg.latent_attention(qd, cd, td, ld, SCALE, q_starts=pd, scale=sd)
    assert torch.equal(got, again)  # the same bits
    return got


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,H,page", DECODES)
def test_decode(skg, lens, H, page, e4m3):
    _attention_case(skg, [1] * len(lens), lens, H, page, e4m3, seed=sum(lens) + H)


CHUNKS = [
    # new tokens, lens, heads, page
    ([2], [2], 1, 8),
    ([40], [40], 16, 16),
    ([1, 33, 0, 7], [300, 33, 9, 100], 20, 64),
    ([70], [133], 5, 32),
    ([9, 4], [520, 4], 48, 64),
    ([3, 5], [64, 200], 128, 64),
    ([6], [4], 3, 16),          # two tokens fall before row 0
    ([150], [400], 2, 64),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("counts,lens,H,page", CHUNKS)
def test_chunk(skg, counts, lens, H, page, e4m3):
    _attention_case(skg, counts, lens, H, page, e4m3, seed=sum(lens) + H, single=False)


@pytest.mark.parametrize("T,B,H", [(300, 300, 1), (260, 260, 40), (600, 520, 2)])
def test_many_sequences(skg, T, B, H):
    """More sequences than one pass of the prefix sums takes, and enough rows for the larger tile."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 40, (B,), generator=g).tolist()
    if T == B:
        counts = [1] * B
    else:
        counts = [1] * B
        for b in range(T - B):
            counts[3 * b % B] += 1
        lens = [max(n, c) for n, c in zip(lens, counts)]
    _attention_case(skg, counts, lens, H, 16, False, seed=B)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("counts,lens,H", [([40], [300], 20), ([7, 0, 30, 1], [70, 5, 1000, 600], 20), ([9], [9], 100), ([5, 2], [400, 2], 65)])
def test_wide_tables(skg, counts, lens, H, e4m3):
    """Sequences that may be long and are not: the larger tile at few rows, and tables whose ends are never read."""
    page, width = 64, 4096
    cache, scale, made = _cache(sum(lens), lens, page, e4m3)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    table[:, :made.shape[1]] = made
    _attention_case(skg, counts, lens, H, page, e4m3, seed=sum(lens), single=False, table=table)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("counts,lens,H", [([20], [60], 100), ([11, 9], [400, 9], 65)])
def test_wide_tables_of_many_heads(skg, counts, lens, H, e4m3):
    """Sequences that may be long and are not: the larger tile at few rows, and tables whose ends are never read."""
    page, width = 64, 4096
    cache, scale, made = _cache(sum(lens), lens, page, e4m3)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    table[:, :made.shape[1]] = made
    _attention_case(skg, counts, lens, H, page, e4m3, seed=sum(lens), single=False, table=table)


@pytest.mark.parametrize("B", [63, 64, 65])
def test_batches_around_a_wave(skg, B):
    g = torch.Generator().manual_seed(B)
    counts = torch.randint(0, 4, (B,), generator=g).tolist()
    lens = [max(c, n) for c, n in zip(counts, torch.randint(0, 300, (B,), generator=g).tolist())]
    _attention_case(skg, counts, lens, 3, 32, True, seed=B, single=False)


def test_large_scores(skg):
    """Scores of hundreds: one key takes all the weight, and the running maximum climbs step after step."""
    _attention_case(skg, [1] * 3, [400, 33, 64], 16, 64, False, seed=9, qscale=60.0)
    # ascending scores
    n, H = 320, 4
    q = torch.zeros(1, H, 576)
    q[..., 0] = 8.0
    cache, _, table = _cache(10, [n], 32, False)
    order = torch.arange(n).float()
    rows = cache[table[0].long()].flatten(0, 1)
    rows[:n, 0] = order
    cache[table[0].long()] = rows.reshape(table.shape[1], 32, 576)
    q = q.bfloat16()
    out, bound = ref.attention(q, cache, None, table, [n], None, SCALE)
    got = skg.latent_attention(*_dev(q, cache, table, _ints([n])), SCALE)
    ref.check(got, out, bound)


@pytest.mark.parametrize("e4m3", [False, True])
def test_what_a_token_does_not_see_has_no_effect(skg, e4m3):
    """NaN (and infinities) behind the end, in pages of nobody, in pages outside the cache, and in later tokens' rows."""
    page, H, counts, lens = 16, 20, [9, 1], [75, 33]
    cache, scale, table = _cache(11, lens, page, e4m3)
    q = _randn(12, 10, H, 576).bfloat16()
    args = (_starts(counts), _ints(lens))
    clean = skg.latent_attention(*_dev(q, cache, table, args[1]), SCALE, q_starts=args[0].to(DEV), scale=None if scale is None else scale.to(DEV))
    dirty = cache.clone().view(torch.uint8)
    bad = torch.tensor([0x7F] * 576 if e4m3 else [0x80, 0x7F, 0xC0, 0x7F] * 288, dtype=torch.uint8)
    used = set(table[0, :5].tolist()) | set(table[1, :3].tolist())
    for p in range(cache.shape[0]):
        if p not in used:
            dirty[p] = bad
    dirty[table[0, 4], 75 % 16:] = bad
    dirty[table[1, 2], 33 % 16:] = bad
    got = skg.latent_attention(*_dev(q, dirty.view(cache.dtype), table, args[1]), SCALE, q_starts=args[0].to(DEV), scale=None if scale is None else scale.to(DEV))
    assert torch.equal(got, clean)
    # the last two tokens' rows of sequence 0: seven tokens do not see them
    dirty[table[0, 4], 73 % 16:75 % 16] = bad
    got = skg.latent_attention(*_dev(q, dirty.view(cache.dtype), table, args[1]), SCALE, q_starts=args[0].to(DEV), scale=None if scale is None else scale.to(DEV))
    # the careful way adds in another order of roundings where it multiplies by vector instructions; these rows have none of it
    out, bound = ref.attention(q, cache, scale, table, lens, args[0].tolist(), SCALE)
    ref.check(got[:7], out[:7], bound[:7])
    assert torch.isnan(got[7:9].float()).any(-1).all()
    assert torch.equal(got[9], clean[9])
    # one infinite value of one row: only its column, and only for those that see it
    if not e4m3:
        dirty = cache.clone()
        dirty[table[0, 4], 73 % 16, 100] = math.inf
        q[..., 100] = 0.5
        got = skg.latent_attention(*_dev(q, dirty, table, args[1]), SCALE, q_starts=args[0].to(DEV))
        out, bound = ref.attention(q, cache, scale, table, lens, args[0].tolist(), SCALE)
        ref.check(got[:7], out[:7], bound[:7])


def test_pages_outside_the_cache_and_shared_ones(skg):
    page, lens = 16, [70, 70, 70, 40]
    cache, _, table = _cache(13, lens, page, False)
    table[0, 1] = -1
    table[1, 4] = cache.shape[0]
    table[2] = table[1]            # the same pages
    table[3, :] = -5               # none
    table[1, 0] = table[0, 0]
    got = _attention_case(skg, [2, 1, 3, 2], lens, 7, page, False, seed=13, table=table)
    assert (got[6:] == 0).all()


def test_rows_behind_the_last_sequence_stay(skg):
    lens, counts = [50, 20], [3, 2]
    cache, _, table = _cache(14, lens, 16, False)
    q = _randn(15, 9, 6, 576).bfloat16()
    out = torch.full((9, 6, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    skg.latent_attention(*_dev(q, cache, table, _ints(lens)), SCALE, q_starts=_starts(counts).to(DEV), out=out)
    want, bound = ref.attention(q, cache, None, table, lens, _starts(counts).tolist(), SCALE)
    ref.check(out, want, bound)
    assert (out[5:] == 3.0).all()


# ------------------------------------------------------------ expanded form

PROMPTS = [
    # new tokens, keys, heads, causal
    ([1], [1], 1, True),
    ([33], [33], 2, True),
    ([130, 1, 0, 5], [130, 40, 7, 5], 3, True),
    ([129], [300], 2, True),
    ([40, 3], [10, 0], 2, True),      # more tokens than keys: some see none
    ([20, 150], [31, 70], 2, False),
    ([300], [300], 8, True),
    # keys of few query tokens shared among workgroups
    ([1, 0, 130, 7], [2100, 700, 530, 0], 2, True), ([64], [1999], 3, False), ([300, 40], [812, 4100], 5, True),
]


def _prompt_inputs(seed, counts, keys, H):
    T, S = sum(counts), sum(keys)
    return ((1.5 * _randn(seed, T, H, 192)).bfloat16(), _randn(seed + 1, S, H, 256).bfloat16(),
            _randn(seed + 2, S, 576).bfloat16(), _starts(counts), _starts(keys))


@pytest.mark.parametrize("counts,keys,H,causal", PROMPTS)
def test_expanded(skg, counts, keys, H, causal):
    q, kv, lat, qs, ks = _prompt_inputs(sum(counts) + H, counts, keys, H)
    out, bound = ref.expanded(q, kv, lat[:, 512:], qs.tolist(), ks.tolist(), SCALE, causal)
    qd, kd, ld, sd, td = _dev(q, kv, lat, qs, ks)
    same = counts == keys
    got = skg.latent_attention_expanded(qd, kd, ld[:, 512:], sd, SCALE, kv_starts=None if same else td, causal=causal)
    ref.check(got, out, bound)
    assert torch.equal(got, skg.latent_attention_expanded(qd, kd, ld[:, 512:], sd, SCALE, kv_starts=td, causal=causal))


def test_expanded_many_sequences(skg):
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 4, (400,), generator=g).tolist()
    q, kv, lat, qs, ks = _prompt_inputs(6, counts, counts, 2)
    out, bound = ref.expanded(q, kv, lat[:, 512:], qs.tolist(), ks.tolist(), SCALE, True)
    qd, kd, ld, sd = _dev(q, kv, lat, qs)
    ref.check(skg.latent_attention_expanded(qd, kd, ld[:, 512:], sd, SCALE), out, bound)


@pytest.mark.parametrize("B,live", [(70, 70), (8192, 6)])
def test_expanded_many_sequences_share_keys(skg, B, live):
    """Batches past a wave, and the largest, whose few query tokens have their keys shared among workgroups."""
    g = torch.Generator().manual_seed(B)
    counts, keys = [0] * B, [0] * B
    for b in torch.randperm(B, generator=g)[:live].tolist():
        counts[b], keys[b] = 1 + b % 2, 500 + 7 * (b % 30)
    q, kv, lat, qs, ks = _prompt_inputs(3, counts, keys, 1)
    out, bound = ref.expanded(q, kv, lat[:, 512:], qs.tolist(), ks.tolist(), SCALE, True)
    qd, kd, ld, sd, td = _dev(q, kv, lat, qs, ks)
    ref.check(skg.latent_attention_expanded(qd, kd, ld[:, 512:], sd, SCALE, kv_starts=td), out, bound)


def test_expanded_unseen_and_behind(skg):
    """Later keys' NaN reach nobody before them; rows behind the last sequence stay; neighbours' keys are not read."""
    counts, H = [50, 70], 3
    q, kv, lat, qs, _ = _prompt_inputs(21, counts, counts, H)
    q = torch.cat((q, q[:4]))
    out, bound = ref.expanded(q, kv, lat[:, 512:], qs.tolist(), qs.tolist(), SCALE, True)
    dirty, dl = kv.clone(), lat.clone()
    dirty[40, 1, 128 + 5] = math.inf
    dirty[45] = math.nan
    dl[46, 512:] = math.nan
    dirty[119] = -math.inf
    o = torch.full((124, H, 128), 2.0, dtype=torch.bfloat16, device=DEV)
    skg.latent_attention_expanded(*_dev(q, dirty, dl[:, 512:], qs), SCALE, out=o)
    for a, b in ((0, 40), (50, 119)):
        ref.check(o[a:b], out[a:b], bound[a:b])
    ref.check(o[40:45, [0, 2]], out[40:45, [0, 2]], bound[40:45, [0, 2]])
    seen = o[40:45, 1].cpu()
    cols = [c for c in range(128) if c != 5]
    ref.check(seen[:, cols], out[40:45, 1][:, cols], bound[40:45, 1][:, cols])
    assert (seen[:, 5] == math.inf).all()
    assert torch.isnan(o[45:50].float()).any(-1).all()
    assert (o[120:] == 2.0).all()


# ------------------------------------------------------------ products per head

@pytest.mark.parametrize("T,H,N,K,pad", [(1, 1, 8, 32, 0), (1, 128, 512, 128, 64), (3, 5, 40, 96, 0), (16, 2, 128, 512, 0),
                                         (17, 3, 512, 128, 8), (130, 4, 128, 512, 0), (300, 2, 72, 480, 32),
                                         (140, 3, 512, 128, 64), (33, 2, 128, 512, 0), (65, 2, 40, 256, 0)])
def test_heads_gemm(skg, T, H, N, K, pad):
    x, w = _randn(T + N, T, H, K + pad).bfloat16(), (_randn(K, H, N, K) * K ** -0.5).bfloat16()
    out, bound = ref.heads(x[..., :K], w)
    xd, wd = _dev(x, w)
    ref.check(skg.heads_gemm(xd[..., :K], wd), out, bound)
    # into a wider tensor, and heads before tokens
    wide = torch.full((T, H, N + 8), 5.0, dtype=torch.bfloat16, device=DEV)
    ref.check(skg.heads_gemm(xd[..., :K], wd, out=wide[..., :N]), out, bound)
    assert (wide[..., N:] == 5.0).all()
    turned = torch.empty(H, T, N, dtype=torch.bfloat16, device=DEV)
    ref.check(skg.heads_gemm(xd[..., :K].transpose(0, 1).contiguous().transpose(0, 1), wd, out=turned.transpose(0, 1)), out, bound)


@pytest.mark.parametrize("K", range(32, 513, 32))
def test_heads_gemm_of_every_depth(skg, K):
    """From the tokens on whose rows are worth a ring in LDS, with a last step that is not full, and below."""
    for T in (19, 16384 // K + 5):
        x, w = _randn(T + K, T, 2, K).bfloat16(), (_randn(K, 2, 136, K) * K ** -0.5).bfloat16()
        out, bound = ref.heads(x, w)
        ref.check(skg.heads_gemm(*_dev(x, w)), out, bound)
