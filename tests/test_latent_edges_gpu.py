"""Latent attention at the ends of its domain on the GPU: scales whose products leave
fp32, rows that hold infinities and NaN in every form of the kernel, long caches.
Against the plain implementations of tests/latent_reference.py and its bounds."""
import pytest
import torch

from tests import latent_reference as ref
from tests import latent_sizes as sizes
from tests.test_latent_gpu import DEV, SCALE, _attention_case, _cache, _dev, _ints, _randn, _starts, skg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,lens,H", [([1], [70], 3), ([40, 7], [300, 9], 20)])
def test_scales_whose_product_leaves_fp32(skg, counts, lens, H):  # noqa: F811
    """Softmax scale 2^126, cache scale 4: scores of zero stay zero, and scores that fit are there."""
    page, softmax = 16, 2.0 ** 126
    cache, _, table = _cache(1, lens, page, True)
    rows = torch.randint(0, 5, cache.shape, generator=torch.Generator().manual_seed(2)).float()
    cache = (rows * (1 - 2 * (torch.arange(576) & 1))).to(torch.float8_e4m3fn)
    scale = torch.tensor([4.0])
    T = sum(counts)
    q = torch.zeros(T, H, 576)
    q[:, 1:, 7] = 2.0 ** -126     # scores 4 times a code; head 0: all zero
    q[:, 2:, 520] = -2.0 ** -126
    q = q.bfloat16()
    out, bound = ref.attention(q, cache, scale, table, lens, _starts(counts).tolist(), softmax)
    got = skg.latent_attention(*_dev(q, cache, table, _ints(lens)), softmax, q_starts=_starts(counts).to(DEV), scale=scale.to(DEV))
    ref.check(got, out, bound)


@pytest.mark.parametrize("counts,lens", [([1], [6205]), ([1, 1], [6205, 40])])
def test_scale_whose_quotient_is_no_normal_number(skg, counts, lens):  # noqa: F811
    """A mean of equal rows is that row: 448 2^-130 is a number of bf16, and every sum on the way (a multiple of 448
    below 2^24 of them) one of fp32.  2^-130 / 6205 is 84.49 times fp32's smallest number, of which 84 is 0.6 % off."""
    page, H = 64, 3
    cache, _, table = _cache(5, lens, page, True)
    cache = torch.full(cache.shape, 448.0).to(torch.float8_e4m3fn)
    cache[..., 1::2] = torch.tensor(-1.0).to(torch.float8_e4m3fn)
    scale = torch.tensor([2.0 ** -130])
    q = torch.zeros(len(lens), H, 576, dtype=torch.bfloat16)
    got = skg.latent_attention(*_dev(q, cache, table, _ints(lens)), SCALE, scale=scale.to(DEV)).cpu()
    assert (got[..., 0::2].double() == 448 * 2.0 ** -130).all()
    assert (got[..., 1::2].double() == -(2.0 ** -130)).all()


# ------------------------------------------------------------ rows that some tokens do not see

NAN = {torch.bfloat16: 0x7FC0, torch.float8_e4m3fn: 0x7F}


def _codes(cache):
    return cache.view(torch.int16 if cache.dtype == torch.bfloat16 else torch.uint8)


def _softmax_over(q, rows, values, seen, scale):
    """ref.softmax_rows with rows that no token of `seen` has taken as zeros, so that their contents touch no bound."""
    clean = torch.where(seen.any(0)[:, None, None], rows, torch.zeros_like(rows))
    vals = torch.where(seen.any(0)[:, None, None], values, torch.zeros_like(values))
    return ref.softmax_rows(q, clean, vals, seen, scale)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("counts,lens,H,page,width,rows", sizes.UNSEEN)
def test_unseen_rows(skg, counts, lens, H, page, width, rows, e4m3):  # noqa: F811
    """The last tokens' rows hold NaN, infinities or both, and so does everything that no sequence has: tokens before
    them get what they would without; those that see a NaN get nothing but NaN; one that sees an infinity where its
    weight is zero gets NaN in that column alone."""
    B, T = len(counts), sum(counts)
    cache, scale, made = _cache(sum(lens) + H, lens, page, e4m3)
    table = made
    if width is not None:
        table = torch.full((B, width), -9, dtype=torch.int32)
        table[:, :made.shape[1]] = made
    q = (1.2 * _randn(T + H, T, H, 576)).bfloat16()
    q[..., 100] = 0.5 + q[..., 100].abs()
    dirty = torch.empty_like(cache)
    _codes(dirty)[:] = NAN[cache.dtype]
    held = [[(int(table[b, p // page]), p % page) for p in range(lens[b])] for b in range(B)]
    for b in range(B):
        for p, (pg, r) in enumerate(held[b]):
            _codes(dirty)[pg, r] = _codes(cache)[pg, r]
    # sequence b: from its last token's row backwards a NaN in column 300, one in the rotated part, and (bf16) an
    # infinity of weight zero before them, all on rows that its first token does not see
    nan_from, minus = [], []
    for b in range(B):
        n, m = counts[b], lens[b]
        bad = [p for p in range(max(m - n + 1, 0), m)][-2:]
        for k, p in enumerate(reversed(bad)):
            pg, r = held[b][p]
            _codes(dirty)[pg, r, 300 if k == 0 else 530] = NAN[cache.dtype]
        nan_from.append(min(bad) if bad else m)
        at = nan_from[b] - 2
        if not e4m3 and at > m - n:
            pg, r = held[b][at]
            dirty[pg, r, 100] = -float("inf")
            minus.append(at)
        else:
            minus.append(None)
    starts = _starts(counts)
    qd, cd, td, ld, sd, zd = _dev(q, dirty, table, _ints(lens), starts, scale)
    got = skg.latent_attention(qd, cd, td, ld, SCALE, q_starts=sd, scale=zd).cpu()
    assert torch.equal(torch.nan_to_num(got.float(), nan=1e9),
                       torch.nan_to_num(skg.latent_attention(qd, cd, td, ld, SCALE, q_starts=sd, scale=zd).cpu().float(), nan=1e9))
    reached = 0
    for b in range(B):
        n, m, t0 = counts[b], lens[b], int(starts[b])
        x = torch.stack([cache[pg, r] for pg, r in held[b]]).double() * (1.0 if scale is None else float(scale))
        for j in range(n):
            own = m - n + j  # the token's own row
            out = got[t0 + j]
            if own >= nan_from[b]:
                assert torch.isnan(out.float()).all(), (b, j)
                reached += 1
                continue
            seen = (torch.arange(m) <= own)[None]
            columns = torch.ones(512, dtype=torch.bool)
            if minus[b] is not None and own >= minus[b]:
                seen[0, minus[b]] = False
                columns[100] = False
                assert torch.isnan(out[:, 100].float()).all(), (b, j)
                reached += 1
            want, bound = _softmax_over(q[t0 + j:t0 + j + 1].double(), x[:, None], x[:, None, :512], seen, SCALE)
            ref.check(out[None][..., columns], want[..., columns], bound[..., columns])
    assert reached


@pytest.mark.parametrize("counts,keys,H,shared", sizes.UNSEEN_KEYS)
def test_unseen_keys(skg, counts, keys, H, shared):  # noqa: F811
    """The same in the expanded form: values and keys of the last tokens, in keys of one workgroup and of several."""
    T, S = sum(counts), sum(keys)
    q, kv, kr = (1.5 * _randn(T, T, H, 192)).bfloat16(), _randn(T + 1, S, H, 256).bfloat16(), _randn(T + 2, S, 64).bfloat16()
    qs, ks = _starts(counts), _starts(keys)
    out, bound = ref.expanded(q, kv, kr, qs.tolist(), ks.tolist(), SCALE, True)
    dirty, dr = kv.clone(), kr.clone()
    end = ks[1:].tolist()
    for b, e in enumerate(end):
        dirty[e - 1] = float("nan")
        dr[e - 3] = float("nan")
        dirty[e - 5, 0, 128 + 77] = float("inf")
    got = skg.latent_attention_expanded(*_dev(q, dirty, dr, qs), SCALE, kv_starts=ks.to(DEV)).cpu()
    for b, (n, m) in enumerate(zip(counts, keys)):
        rows = got[int(qs[b]):int(qs[b]) + n]
        want, lim = out[int(qs[b]):int(qs[b]) + n], bound[int(qs[b]):int(qs[b]) + n]
        ref.check(rows[:n - 5], want[:n - 5], lim[:n - 5])
        # five tokens see the infinity, of head 0's column 77, three the NaN of all heads
        other = [c for c in range(128) if c != 77]
        ref.check(rows[n - 5:n - 3][:, 0][:, other], want[n - 5:n - 3][:, 0][:, other], lim[n - 5:n - 3][:, 0][:, other])
        assert (rows[n - 5:n - 3, 0, 77] == float("inf")).all()
        ref.check(rows[n - 5:n - 3, 1:], want[n - 5:n - 3, 1:], lim[n - 5:n - 3, 1:])
        assert torch.isnan(rows[n - 3:].float()).all()


# ------------------------------------------------------------ tables wider than the sequences, long caches

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("counts,lens,H,page,width,rows", sizes.SHORT + sizes.LONG)
def test_wide_tables_and_long_caches(skg, counts, lens, H, page, width, rows, e4m3):  # noqa: F811
    """Either tile, tables entered by steps and by eight rows; their ends are never read."""
    cache, scale, made = _cache(sum(lens) + 1, lens, page, e4m3)
    table = made
    if width is not None:
        table = torch.full((len(lens), width), -7, dtype=torch.int32)
        table[:, :made.shape[1]] = made
    _attention_case(skg, counts, lens, H, page, e4m3, seed=sum(lens) + 1, single=False, table=table)


# ------------------------------------------------------------ large values

@pytest.mark.parametrize("qscale", [0.5, 40.0])
def test_values_near_the_largest(skg, qscale):  # noqa: F811
    """Half of the columns 2^107 times as large, 600 of them a sequence: sums below 2^119 that scores know nothing of."""
    page, counts, lens, H = 64, [5, 1], [600, 40], 6
    cache, _, table = _cache(31, lens, page, False)
    cache[..., 256:512] *= 2.0 ** 107
    q = (qscale * _randn(32, 6, H, 576)).bfloat16()
    q[..., 256:512] = 0.0
    starts = _starts(counts)
    out, bound = ref.attention(q, cache, None, table, lens, starts.tolist(), SCALE)
    ref.check(skg.latent_attention(*_dev(q, cache, table, _ints(lens)), SCALE, q_starts=starts.to(DEV)), out, bound)
    eq, kv, kr = (qscale * _randn(33, 6, H, 192)).bfloat16(), _randn(34, 640, H, 256).bfloat16(), _randn(35, 640, 64).bfloat16()
    kv[..., 192:] *= 2.0 ** 107
    ks = _starts(lens)
    out, bound = ref.expanded(eq, kv, kr, starts.tolist(), ks.tolist(), SCALE, True)
    ref.check(skg.latent_attention_expanded(*_dev(eq, kv, kr, starts), SCALE, kv_starts=ks.to(DEV)), out, bound)
