"""GPU: attention over the token cache takes every page that exists exactly once, and the right one.

Every kernel form, with more pages than a wave reads of the table at a time (64), more splits than the join holds at
a time (256), lost pages around every 64th entry, and pages that several sequences share.  All of it is exact up to a few
roundings, so that one page too few, too many or in another's place shows, in bf16 too:
  * queries of zeros give every token the same weight, 1; a page's values are one sign a channel, so the sum over n tokens
    is a whole number of at most 2^24, whatever the order, and the output is that number over n;
  * a query aimed at a page (keys are the signs of the page's number) gets that page's values.
"""
import ctypes

import numpy as np
import pytest
import torch

from camera_bev_view_amd import _lib, ops
from gpu_helpers import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
KINDS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def splits_of(B, T, W, Hq, Hk, D, dtype):
    """The parts that a call's rows are split into, from the workspace it asks for (splits x rows x (D + 2) floats)."""
    need = ctypes.c_size_t()
    ad = _lib.CacheAttentionDesc(Hq, _lib.FBEV_DRAFT_NONE, 0, (0, 0, 0), None, 1.0, 0.0)
    _lib.check(_lib.load().fbev_cache_attention_workspace(
        _lib.CacheDesc(0, Hk, D, 0, None, None, None, None), _lib.CacheRows(B, T, W, 16, 16, None), ad,
        _lib.FBEV_DTYPE_F32 if dtype == F32 else _lib.FBEV_DTYPE_BF16, ctypes.byref(need)))
    return max(1, need.value // (4 * B * T * Hq * (D + 2)))


def signed_cache(W, Hk, D, kind, seed):
    """Pages whose 64 tokens have the same keys and values: random signs [pages, Hk, D] each, keys that differ from page to
    page in a fifth of D at least (D of 32 and more)."""
    rng = np.random.default_rng(seed)
    cache = ops.token_cache(W, Hk, D, codes=KINDS[kind])
    keys, values = (rng.choice(np.array([-1, 1], np.int8), (W, Hk, D)) for _ in range(2))
    up = lambda a: torch.from_numpy(a).cuda().to(KINDS[kind]).view(torch.uint8)
    cache.k.view(torch.uint8)[..., :D] = up(keys)[:, :, None, :]
    cache.v.view(torch.uint8)[:, :, :D] = up(values)[..., None]
    cache.k_scale.fill_(0.5)
    cache.v_scale.fill_(0.25)
    return cache, keys, values


# (B, T, Hq, Hk, D, W, splits by type (fp32, bf16)): the form, and what is long about it
FORMS = [
    (24, 1, 8, 8, 32, 600, (1, 1)),        # eight waves with pages of their own, 75 each
    (8, 3, 96, 24, 40, 530, (1, 1)),       # the same, groups of query heads
    (191, 1, 2, 1, 32, 800, (3, 3)),       # four waves of their own, 66 each, splits
    (32, 20, 24, 12, 32, 140, (1, 1)),     # two groups of waves, 70 pages each, not split
    (32, 20, 24, 12, 128, 140, (1, 1)),    # the same, heads of 128
    (8, 20, 16, 8, 32, 1100, (4, 4)),      # two groups (fp32) and four (bf16), 69 pages each and more, splits
    (8, 420, 8, 4, 64, 150, (1, 3)),       # eight row tiles share 150 pages (50 in three splits)
    (16, 800, 8, 4, 32, 75, (1, 1)),       # the same, not split in bf16 either
    (1, 1, 1, 1, 32, 1200, (300, 300)),    # a single row, 300 splits of four pages
    (1, 2, 8, 1, 128, 2100, (512, 512)),   # 16 rows, the most splits
    (1, 70, 1, 1, 128, 1400, (256, 350)),  # row tiles that share pages, 350 splits
    (1, 30, 1, 1, 64, 1100, (256, 256)),   # groups of waves, 256 splits
]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("form", FORMS)
def test_every_page_once(form, dtype, kind):
    B, T, Hq, Hk, D, W, splits = form
    assert splits_of(B, T, W, Hq, Hk, D, dtype) == splits[dtype == BF16]
    say(f"[case] {form} {dtype} {kind}")
    cache, keys, values = signed_cache(W, Hk, D, kind, W + D)
    rng = np.random.default_rng(B + W)
    table = np.stack([rng.permutation(W) for _ in range(B)]).astype(np.int32)
    lost = np.unique([w for n in range(0, W, 64) for w in (n, n + 63) if w < W and n] + [1, W - 2])
    table[:, lost] = np.where(rng.random((B, len(lost))) < 0.5, -1, np.iinfo(np.int32).max)
    # whole tables, and sequences that end inside a page
    start = np.where(np.arange(B) % 2 == 0, 64 * W, 64 * W - 64 * (np.arange(B) % 5) - 27).astype(np.int32)
    to = lambda a: torch.from_numpy(a).cuda()
    q = torch.zeros((B, T, Hq, D), dtype=dtype, device="cuda")
    out = ops.cache_attention(q, cache, to(table), to(start), drafted=False).double().cpu().numpy()
    for b in range(B):
        tokens = np.clip(int(start[b]) - 64 * np.arange(W), 0, 64) * ((table[b] >= 0) & (table[b] < W))
        n = int(tokens.sum())
        sums = np.einsum("w,whd->hd", tokens.astype(np.float64), values[np.where(tokens > 0, table[b], 0)].astype(np.float64))
        assert n <= 1 << 22                             # (times a quarter and powers of two: exact)
        want = np.repeat(sums * 0.25 / n, Hq // Hk, axis=0)
        # 1 / n and the product with it, one rounding each, and the output's own
        bound = np.abs(want) * (3 * 2.0 ** -24 + HALF[dtype]) * 1.01
        err = np.abs(out[b] - want)
        assert (err <= bound).all(), f"sequence {b}: {int((err > bound).sum())} of {err.size} outside"
        # what a page changes an output by is seen: its 64 tokens' part of the channel's sum
        assert 64 * 0.25 / n > 4 * np.median(bound)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("form", FORMS)
def test_every_page_in_its_place(form, dtype, kind):
    """Rows aimed at pages in turn, several calls where a call has fewer rows than the table has pages."""
    B, T, Hq, Hk, D, W, _ = form
    say(f"[case] {form} {dtype} {kind}")
    cache, keys, values = signed_cache(W, Hk, D, kind, W + D + 1)
    rng = np.random.default_rng(B + W + 1)
    table = np.stack([rng.permutation(W) for _ in range(B)]).astype(np.int32)
    start = np.full(B, 64 * W, np.int32)
    to = lambda a: torch.from_numpy(a).cuda()
    # scores are `sharp` times the number of equal signs less that of others: D for the page itself.  Pages that share all but
    # a few signs with it keep a weight of e^(-2 sharp d) at d signs apart: counted below
    sharp = 8.0
    G = Hq // Hk
    order = rng.permutation(W)
    same = np.zeros((Hk, W))                            # signs in common with the nearest other page
    for h in range(Hk):
        c = keys[:, h].astype(np.float32) @ keys[:, h].astype(np.float32).T
        np.fill_diagonal(c, -D)
        same[h] = c.max(axis=1)
    for call in range(min(-(-W // (B * T * G)), 24)):
        at = order[(call * B * T * Hq + np.arange(B * T * Hq)) % W].reshape(B, T, Hk, G)
        page = table[np.arange(B)[:, None, None, None], at]
        head = np.arange(Hk)[None, None, :, None]
        q = keys[page, head].astype(np.float32).reshape(B, T, Hq, D) * 2.0
        out = ops.cache_attention(to(q).to(dtype), cache, to(table), to(start), drafted=False, scale=sharp)
        out = out.float().cpu().numpy().reshape(B, T, Hk, G, D)
        want = values[page, head] * np.float32(0.25)
        gap = sharp * (D - same[head, page])            # of the scores
        # others weigh W e^-gap together at most, twice that of 0.25; weights in two parts leave 2^-17; sums of equal values
        # and the division a few steps more
        bound = 0.25 * (2 * W * np.exp(-gap) + 2.0 ** -16 + HALF[dtype])[..., None]
        err = np.abs(out - want)
        assert (bound < 0.01).all() and (err <= bound).all(), \
            f"call {call}: {int((err > bound).sum())} of {err.size} outside, first at {np.argwhere(err > bound)[:1].tolist()}"


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 2, 2), (3, 8, 1), (40, 2, 1), (90, 2, 1)])
def test_the_widest_table(T, Hq, Hk, dtype):
    """2^24 pages, the most that a table may have, of which a handful exist: the first, the last (which the call's own
    tokens fill up to the table's end) and some between."""
    W, D = 1 << 24, 32
    say(f"[case] table of {W} pages, T={T} {dtype}")
    cache, keys, values = signed_cache(8, Hk, D, "int8", T)
    # the last page's own tokens: the same signs, written by the call
    table = torch.full((1, W), -1, dtype=torch.int32, device="cuda")
    places = [0, 1, 65, 4097, (1 << 23) + 5, W - 66, W - 2, W - 1]
    table[0, places] = torch.arange(8, dtype=torch.int32, device="cuda")
    start = torch.tensor([64 * W - T], dtype=torch.int32, device="cuda")
    old = [cache.k[7].clone(), cache.v[7].clone()]
    rows = lambda a, p: torch.from_numpy(a[p].astype(np.float32)).cuda().expand(1, 1, Hk, D)
    k = torch.cat([rows(keys, 6 + (64 * W - T + t >= 64 * W - 64)) for t in range(T)], 1) * 0.5 * 127
    v = torch.cat([rows(values, 6 + (64 * W - T + t >= 64 * W - 64)) for t in range(T)], 1) * 0.25 * 127
    ops.cache_write(cache, k, v, table, start)
    # rows of one size have the code 127: as values, 1 / 127 of what was written
    own = slice(64 - min(T, 64), 64)
    assert torch.equal(cache.k[7][:, own, :D], old[0][:, own, :D] * 127)
    q = torch.zeros((1, T, Hq, D), dtype=dtype, device="cuda")
    out = ops.cache_attention(q, cache, table, start)[0].double().cpu().numpy()
    for t in range(T):
        tokens = np.array([64] * 6 + [min(64, 128 - T + t + 1), max(0, 64 - T + t + 1)])
        # values: 0.25 a sign from the pages, 0.25 x 127 from the call's rows, exact in codes of 1 / 127 of their scale
        mine = np.array([0] * 6 + [max(0, min(64, 128 - T + t + 1) - min(64, 128 - T)), max(0, min(T, 64) - (T - 1 - t))])
        sums = np.einsum("p,phd->hd", (tokens - mine) + 127.0 * mine, values.astype(np.float64)) * 0.25
        want = np.repeat(sums / tokens.sum(), Hq // Hk, axis=0)
        size = 0.25 * (tokens - mine + 127.0 * mine).sum() / tokens.sum()
        # a scale of 0.25 is one rounding off at most; weights in parts (bf16: 2^-17); 512 sums; the output's rounding
        bound = size * (520 * 2.0 ** -24 + (0 if dtype == F32 else 2.0 ** -17)) + HALF[dtype] * np.abs(want)
        err = np.abs(out[t] - want)
        assert (err <= bound * 1.01).all(), (t, float((err / bound).max()))
