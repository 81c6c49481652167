"""GPU: attention of query tokens over the token cache, every output element against bounds from the arithmetic."""
import numpy as np
import pytest
import torch

import oracle.decoder as dec
from camera_bev_view_amd import _lib, ops
from decoder_bounds import KINDS, attention_bounds, close, f64
from gpu_helpers import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def draw(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def filled(seed, lengths, Hk, D, kind, spare=1, size=1.0):
    """A cache whose sequences hold `lengths` tokens on scattered pages; all else is what memory may hold: any code, NaN
    among them, and NaN for scales.  Returns (cache, model, table)."""
    rng = np.random.default_rng(seed)
    W = max(1, max(-(-n // 64) for n in lengths)) + spare
    pages = len(lengths) * W + 2
    table = rng.permutation(pages)[:len(lengths) * W].reshape(len(lengths), W)
    model = dec.Cache(pages, Hk, D, kind)
    for a in (model.k, model.v):
        a[...] = rng.integers(0, 256, a.shape, dtype=np.uint8)
    for a in (model.k_scale, model.v_scale):
        a[...] = np.nan
    n = dec.numbers(kind)
    for b, length in enumerate(lengths):
        for w in range(-(-length // 64)):
            page, m = table[b, w], min(64, length - 64 * w)
            for codes, scales, view in ((model.k, model.k_scale, lambda c: c[page, :, :m, :]),
                                        (model.v, model.v_scale, lambda c: c[page, :, :, :m].swapaxes(1, 2))):
                x = rng.normal(size=(Hk, m, D)) * size * rng.choice([0.3, 1.0, 3.0], size=(Hk, m, 1))
                c, s = dec.row_codes(x.astype(np.float32), kind)
                view(codes)[..., :D] = c
                view(codes)[..., D:] = 0
                scales[page, :, :m] = s
    up = lambda a: torch.from_numpy(a.copy()).cuda()
    cache = ops.TokenCache(up(model.k).view(KINDS[kind]), up(model.v).view(KINDS[kind]), up(model.k_scale),
                           up(model.v_scale), D)
    return cache, model, table


def random_trees(seed, B, T):
    rng = np.random.default_rng(seed)
    bits = np.zeros((B, T, T), bool)
    for b in range(B):
        for j in range(T):
            p = j - int(rng.integers(1, 6))
            if p >= 0:
                bits[b, j] = bits[b, p]
            bits[b, j, j] = True
    return bits


def pack(bits):
    B, T, _ = bits.shape
    words = max(1, -(-T // 64))
    out = np.zeros((B, T, words), np.uint64)
    for j in range(T):
        out[:, :, j // 64] |= bits[:, :, j].astype(np.uint64) << np.uint64(j % 64)
    return torch.from_numpy(out.view(np.int64)).cuda()


def check(q, cache, model, table, start, drafts, count=None, bits=None, scale=None, cap=0.0, label="", **more):
    out = ops.cache_attention(q, cache, i32(table.tolist() if hasattr(table, "tolist") else table), i32(start),
                              count=i32(count), ancestors=None if bits is None else pack(bits),
                              drafted=drafts != "none", scale=scale, cap=cap, **more)
    qn = f64(q)
    ref = dec.attention(qn, model, np.asarray(table), start, drafts, count, bits, scale, cap)
    bound = attention_bounds(qn, ref, abs(q.shape[3] ** -0.5 if scale is None else scale), cap, q.dtype)
    close(label or drafts, out, ref["out"], bound)
    return out


# (starts, T, Hq, Hk): single tokens, tiles that end inside, row tiles of every kind, no cache, ragged batches
SHAPES = [([0], 1, 1, 1), ([1], 1, 4, 4), ([63, 64, 65], 1, 8, 2), ([1000], 1, 8, 1), ([700, 0, 129], 3, 6, 2),
          ([130], 16, 2, 2), ([127, 5], 17, 4, 1), ([300], 40, 8, 4), ([64, 190], 130, 2, 1), ([0, 0], 70, 4, 2)]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("drafts", ["none", "chain", "tree"])
def test_shapes(shape, drafts, dtype, kind):
    start, T, Hq, Hk = shape
    D = 64 if T < 20 else 32
    say(f"[case] {shape} {drafts} {dtype} {kind}")
    cache, model, table = filled(T + Hq, [n + (0 if drafts == "none" else T) for n in start], Hk, D, kind)
    q = draw(T, len(start), T, Hq, D, dtype=dtype)
    bits = random_trees(T, len(start), T) if drafts == "tree" else None
    out = check(q, cache, model, table, start, drafts, bits=bits)
    if drafts == "none":
        for b, n in enumerate(start):
            assert n > 0 or not out[b].any()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [1, 5, 16, 31, 32, 33, 48, 64, 65, 80, 96, 112, 127, 128])
def test_widths(D, dtype, kind):
    say(f"[case] D={D} {dtype} {kind}")
    cache, model, table = filled(D, [205, 77], 2, D, kind)
    for T, Hq in ((1, 4), (9, 8), (30, 4)):
        q = draw(D + T, 2, T, Hq, D, dtype=dtype)
        check(q, cache, model, table, [205 - T, 77 - T], "chain", label=f"T={T}")
    check(draw(D, 2, 5, 2, D, dtype=dtype) * 4, cache, model, table, [200, 72], "chain", cap=3.0, label="capped")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scales_caps_and_large_scores(dtype):
    cache, model, table = filled(3, [333], 2, 40, "e4m3")
    q = draw(1, 1, 6, 4, 40, dtype=dtype)
    for scale, cap in ((0.0, 0.0), (-0.3, 0.0), (2.0, 0.0), (1.0, 20.0), (0.05, 50.0), (-1.0, 1.0), (1e-6, 1e-3),
                       (1.0, 1e6)):
        check(q, cache, model, table, [327], "chain", scale=scale, cap=cap, label=f"scale={scale} cap={cap}")
    cache, model, table = filled(4, [333], 2, 40, "int8", size=30.0)
    check(q * 3, cache, model, table, [333], "none", label="one token takes all")


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_padded_batches_and_lost_pages(kind):
    """Counts, pages that do not exist, starts beyond the table or negative: the others' results, zeros for padding."""
    cache, model, table = filled(9, [200, 200, 200, 200, 200, 200], 2, 32, kind)
    table = table.copy()
    table[1, 1] = -1
    table[2, 0] = 10 ** 6
    table[3] = -7
    start, T = [150, 150, 150, 150, -3, 2 ** 31 - 1], 50
    # the last sequence's table holds 256 tokens, of which 56 were never written: give it its written pages alone
    table = table[:, :3]
    for drafts in ("none", "chain", "tree"):
        for count in ([50, 50, 30, 50, 50, 50], [0, 1, 49, -4, 50, 2 ** 31 - 1], None):
            if count is None and drafts != "none":
                continue
            st = start[:5] + ([192] if drafts != "none" else [2 ** 31 - 1])
            bits = random_trees(5, 6, T) if drafts == "tree" else None
            out = check(draw(1, 6, T, 4, 32, dtype=BF16), cache, model, table, st, drafts, count, bits,
                        label=f"{drafts} {count}")
            assert out.isfinite().all() and not out[3].any() and not out[4].any()
            if count is not None:
                assert not out[0, max(0, min(50, count[0])):].any() and not out[1, max(0, count[1]):].any()


def test_trees_with_empty_rows_and_wide_words():
    """Bits of any pattern: a query that sees neither itself nor the cache gets zeros; more words than needed; trees over
    word and page borders."""
    rng = np.random.default_rng(6)
    for start, T in (([0, 0], 64), ([50, 13], 65), ([1, 127], 200)):
        cache, model, table = filled(T, [n + T for n in start], 2, 32, "e4m3")
        bits = rng.random((2, T, T)) < 0.2
        bits[:, 3] = False
        bits[0, 10:20] = False
        q = draw(T, 2, T, 4, 32)
        out = check(q, cache, model, table, start, "tree", bits=bits, label=f"{start} {T}")
        if start == [0, 0]:
            assert not out[:, 3].any() and not out[0, 10:20].any()
        wide = torch.cat((pack(bits), torch.full((2, T, 2), -1, dtype=torch.int64, device="cuda")), dim=2)
        again = ops.cache_attention(q, cache, i32(table.tolist()), i32(start), ancestors=wide)
        assert torch.equal(again, out)
        # bits behind the last row are nobody's
        high = wide.clone()
        if T % 64:
            high[:, :, T // 64] |= -1 << (T % 64)
            assert torch.equal(ops.cache_attention(q, cache, i32(table.tolist()), i32(start), ancestors=high), out)
        one = ops.cache_attention(q, cache, i32(table.tolist()), i32(start), ancestors=wide[:1])
        assert torch.equal(one[0], out[0])


def test_a_chain_is_a_tree():
    cache, model, table = filled(8, [300], 2, 64, "int8")
    q = draw(2, 1, 20, 8, 64, dtype=BF16)
    chain = ops.cache_attention(q, cache, i32(table.tolist()), i32([280]))
    tree = ops.cache_attention(q, cache, i32(table.tolist()), i32([280]), ancestors=ops.tree_ancestors(range(-1, 19)))
    assert torch.equal(chain, tree)


def test_odd_tokens_reach_those_that_see_them():
    for kind in ("int8", "e4m3"):
        cache, model, table = filled(12, [140], 1, 32, kind)
        q = draw(3, 1, 10, 2, 32)
        start, t = [130], i32(table.tolist())
        good = ops.cache_attention(q, cache, t, i32(start))
        for scales in (cache.k_scale, cache.v_scale):
            page, slot = int(table[0, 2]), 135 - 128
            old = scales[page, 0, slot].clone()
            scales[page, 0, slot] = float("nan")
            out = ops.cache_attention(q, cache, t, i32(start))
            assert torch.equal(out[:, :5], good[:, :5]) and out[:, 5:].isnan().all()
            assert ops.cache_attention(q, cache, t, i32(start), drafted=False).isfinite().all()
            scales[page, 0, slot] = old
        # every token that a query sees: nothing but NaN, joined over workgroups too
        cache.k_scale[:] = float("nan")
        assert ops.cache_attention(q, cache, t, i32(start)).isnan().all()
    # a query of infinities and NaN is alone with them
    cache, model, table = filled(13, [700], 2, 32, "int8")
    q = draw(4, 1, 9, 4, 32)
    good = ops.cache_attention(q, cache, i32(table.tolist()), i32([691]))
    q[0, 2, 1, 7], q[0, 5, 3, 0] = float("nan"), float("inf")
    out = ops.cache_attention(q, cache, i32(table.tolist()), i32([691]))
    bad = torch.zeros((1, 9, 4), dtype=torch.bool, device="cuda")
    bad[0, 2, 1] = bad[0, 5, 3] = True
    assert torch.equal(out[~bad], good[~bad]) and out[0, 2, 1].isnan().all()


def test_scales_far_apart():
    """Tokens whose values differ by 2^60: the attended one's digits are kept whatever the others' scales are."""
    cache, model, table = filled(14, [192], 1, 32, "int8")
    model.v_scale[table[0, 0], 0] *= np.float32(2.0 ** 60)
    model.v_scale[table[0, 1], 0] *= np.float32(2.0 ** -60)
    cache.v_scale.copy_(torch.from_numpy(model.v_scale))
    k, _ = model.token(int(table[0, 1]), 9)
    q = torch.from_numpy(np.tile(k[0] * 40, (1, 3, 1, 1)).transpose(0, 1, 2, 3)).float().cuda()
    for dtype in (F32, BF16):
        check(q.to(dtype), cache, model, table, [192], "none", label=f"{dtype}")


def test_views_and_addresses():
    cache, model, table = filled(15, [90, 40, 77], 2, 40, "e4m3")
    packed = draw(1, 3, 7, 2, 4, 40, dtype=BF16)
    check(packed[:, :, 1], cache, model, table, [83, 33, 70], "chain", label="packed")
    flat = draw(2, 3 * 7 * 4 * 40 + 1)
    check(flat[1:].view(3, 7, 4, 40), cache, model, table, [83, 33, 70], "chain", label="odd address")
    check(flat[:-1].view(3, 4, 7, 40).transpose(1, 2), cache, model, table, [83, 33, 70], "chain", label="heads first")
    check(draw(3, 1, 1, 4, 40).expand(3, 7, 4, 40), cache, model, table, [83, 33, 70], "chain", label="broadcast")
    check(draw(4, 40, 4, 7, 3).permute(3, 2, 1, 0), cache, model, table, [83, 33, 70], "chain", label="channels apart")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,Hq,Hk,D,n,drafts", [
    (50, 1, 8, 4, 32, 70, "chain"), (64, 3, 6, 3, 64, 200, "tree"), (200, 2, 8, 1, 128, 130, "chain"),
    (70, 40, 4, 4, 40, 64, "chain"), (32, 90, 6, 2, 128, 300, "chain"), (33, 130, 4, 2, 96, 290, "tree"),
    (75, 130, 4, 2, 128, 5, "chain"), (112, 260, 2, 2, 64, 0, "tree"), (100, 70, 2, 2, 32, 63, "none")])
def test_many_sequences(B, T, Hq, Hk, D, n, drafts, dtype):
    """Enough sequences and heads for workgroups of more waves, calls that need no split and those split in two."""
    say(f"[case] {B} sequences of {n} + {T}")
    rng = np.random.default_rng(B)
    start = [int(x) for x in rng.integers(max(0, n - 40), n + 1, B)]
    cache, model, table = filled(B, [s + (0 if drafts == "none" else T) for s in start], Hk, D, "e4m3" if B % 2 else "int8")
    count = [int(x) for x in rng.integers(0, T + 1, B)] if B > 70 else None
    bits = random_trees(B, B, T) if drafts == "tree" else None
    check(draw(B, B, T, Hq, D, dtype=dtype), cache, model, table, start, drafts, count, bits)


def test_long_caches():
    """Splits over workgroups and their join, more than 64 of them."""
    n, D = 40003, 32
    say(f"[case] {n} tokens")
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn((1, n, 1, D), generator=g, device="cuda") for _ in range(2))
    for kind in ("int8", "e4m3"):
        cache = ops.token_cache(700, 1, D, codes=KINDS[kind])
        table = torch.randperm(700, generator=torch.Generator().manual_seed(1))[:626].view(1, 626).int().cuda()
        ops.cache_write(cache, k, v, table, i32([0]))
        kd, vd = ops.cache_read(cache, table, i32([0]), n, dtype=F32)
        for dtype in (F32, BF16):
            for T in (1, 5, 33):
                q = draw(T, 1, T, 2, D, dtype=dtype)
                out = ops.cache_attention(q, cache, table, i32([n - T]))
                s = torch.einsum("thd,nd->htn", q[0].double(), kd[0, :, 0].double()) * D ** -0.5
                seen = torch.arange(n, device="cuda") <= n - T + torch.arange(T, device="cuda")[:, None]
                p = torch.softmax(s.masked_fill(~seen, float("-inf")), dim=-1)
                want = torch.einsum("htn,nd->thd", p, vd[0, :, 0].double())
                size = torch.einsum("htn,nd->thd", p, vd[0, :, 0].double().abs())
                mag = D ** -0.5 * torch.einsum("thd,nd->htn", q[0].double().abs(), kd[0, :, 0].double().abs()).amax(-1)
                U = 2.0 ** -24
                # read values are rounded once more (U each), then as in attention_bounds
                rel = 2 * (3 * D + 36) * U * mag.T[..., None] + 2 * (n + 64) * U + (2 * U if dtype == F32 else 2.0 ** -17)
                bound = rel * size * 1.01
                bound = bound + (U if dtype == F32 else 2.0 ** -8) * (want.abs() + bound)
                err = (out[0].double() - want).abs()
                say(f"[bound] {kind} {dtype} T={T}: share of the bound {float((err / bound).max()):.3f}")
                assert (err <= bound).all()


@pytest.mark.parametrize("Hk,n,B,D", [(8, 7000, 8, 64), (2, 30000, 3, 24), (3, 2500, 4, 128), (16, 3200, 8, 32)])
def test_long_ragged_caches(Hk, n, B, D):
    """Groups of waves that take turns at the pages, of which some are lost, with few rows to a head and several splits."""
    say(f"[case] {B} sequences of up to {n} tokens")
    W, G = -(-n // 64) + 1, 2
    lengths = [n, n // 2 + 3, 0, 1, n - 700, 64, 63, n // 3][:B]
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn((B, n, Hk, D), generator=g, device="cuda") for _ in range(2))
    for kind in ("int8", "e4m3"):
        cache = ops.token_cache(B * W, Hk, D, codes=KINDS[kind])
        table = torch.randperm(B * W, generator=torch.Generator().manual_seed(2)).view(B, W).int()
        table[:, 5::7] = -1
        table = table.cuda()
        ops.cache_write(cache, k, v, table, i32([0] * B), count=i32(lengths))
        kd, vd = (x.double() for x in ops.cache_read(cache, table, i32([0] * B), n, dtype=F32))
        there = (table >= 0).repeat_interleave(64, 1)[:, :n]
        for dtype in (F32, BF16):
            for T in (9, 30, 70):
                q = draw(T, B, T, Hk * G, D, dtype=dtype)
                out = ops.cache_attention(q, cache, table, i32(lengths), drafted=False)
                for b in range(B):
                    seen = there[b] & (torch.arange(n, device="cuda") < lengths[b])
                    if not seen.any():
                        assert not out[b].any()
                        continue
                    kb, vb = kd[b][seen].transpose(0, 1), vd[b][seen].transpose(0, 1)
                    qb = q[b].double().view(T, Hk, G, D).permute(1, 0, 2, 3).reshape(Hk, T * G, D)
                    s = torch.matmul(qb, kb.transpose(1, 2)) * D ** -0.5
                    p = torch.softmax(s, -1)
                    back = lambda x: x.view(Hk, T, G, -1).permute(1, 0, 2, 3).reshape(T, Hk * G, -1)
                    want, size = back(torch.matmul(p, vb)), back(torch.matmul(p, vb.abs()))
                    mag = back((D ** -0.5 * torch.matmul(qb.abs(), kb.abs().transpose(1, 2))).amax(-1, keepdim=True))
                    U = 2.0 ** -24
                    # as in test_long_caches
                    rel = 2 * (3 * D + 36) * U * mag + 2 * (n + 64) * U + (2 * U if dtype == F32 else 2.0 ** -17)
                    bound = rel * size * 1.01
                    bound = bound + (U if dtype == F32 else 2.0 ** -8) * (want.abs() + bound)
                    assert ((out[b].double() - want).abs() <= bound).all(), (kind, dtype, T, b)


def test_pages_beyond_31_bits():
    pages, Hk, D = 33000, 8, 128
    say(f"[case] cache of {pages} pages")
    cache = ops.token_cache(pages, Hk, D)
    small = ops.token_cache(3, Hk, D)
    k, v = draw(1, 1, 150, Hk, D, dtype=BF16), draw(2, 1, 150, Hk, D, dtype=BF16)
    far, near = i32([[32999, 32800, 7]]), i32([[2, 1, 0]])
    for c, t in ((cache, far), (small, near)):
        ops.cache_write(c, k, v, t, i32([0]))
    for T in (1, 60):
        q = draw(T, 1, T, 16, D, dtype=BF16)
        assert torch.equal(ops.cache_attention(q, cache, far, i32([150 - T])),
                           ops.cache_attention(q, small, near, i32([150 - T])))


def test_given_outputs_and_workspaces():
    cache, model, table = filled(16, [500], 2, 64, "int8")
    t, q = i32(table.tolist()), draw(1, 1, 4, 4, 64, dtype=BF16)
    want = ops.cache_attention(q, cache, t, i32([496]))
    out, ws = torch.empty_like(q), torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert ops.cache_attention(q, cache, t, i32([496]), out=out, workspace=ws) is out
        assert torch.equal(out, want)
    assert torch.equal(ops.cache_attention(q, cache, t, i32([496]), workspace=ws[:16]), want)
    with pytest.raises(ValueError, match="overlap"):
        ops.cache_attention(q, cache, t, i32([496]), out=q)
    with pytest.raises(ValueError, match="overlap"):
        ops.cache_attention(q, cache, t, i32([496]), out=ws[:2048].view(BF16).view(1, 4, 4, 64), workspace=ws)


def test_refusals():
    cache, model, table = filled(17, [100], 2, 32, "int8")
    t, q, start = i32(table.tolist()), draw(1, 1, 5, 4, 32), i32([95])
    a = ops.tree_ancestors(range(-1, 4))
    for bad in (dict(q=q[..., :31]), dict(q=q.half()), dict(q=q.cpu()), dict(q=q[0]), dict(start=start.long()),
                dict(count=i32([1, 2])), dict(table=t.long()), dict(ancestors=a[:, :4]), dict(ancestors=a.int()),
                dict(ancestors=a[0]), dict(ancestors=a, drafted=False), dict(ancestors=a[:, :, :0]),
                dict(out=torch.empty_like(q, dtype=BF16)), dict(workspace=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            ops.cache_attention(**{**dict(q=q, cache=cache, table=t, start=start), **bad})
    with pytest.raises(_lib.FlashBevError, match="multiple"):
        ops.cache_attention(q[:, :, :3], cache, t, start)
    with pytest.raises(_lib.FlashBevError, match="scale"):
        ops.cache_attention(q, cache, t, start, scale=float("nan"))
    with pytest.raises(_lib.FlashBevError, match="cap"):
        ops.cache_attention(q, cache, t, start, cap=-2.0)


def test_empty_calls():
    cache = ops.token_cache(2, 1, 16)
    none = i32([]).view(2, 0)
    assert ops.cache_attention(draw(1, 2, 0, 1, 16), cache, i32([[0], [1]]), i32([0, 0])).shape == (2, 0, 1, 16)
    assert ops.cache_attention(draw(1, 2, 1, 1, 16)[:0], cache, none[:0], i32([])).shape == (0, 1, 1, 16)
    assert not ops.cache_attention(draw(1, 2, 3, 1, 16), cache, none, i32([5, 0])).any()
    assert not ops.cache_attention(draw(1, 2, 3, 1, 16), ops.token_cache(0, 1, 16), i32([[0], [1]]), i32([5, 0])).any()


def test_graph_replays_and_streams():
    """A captured step of serving: the new token goes in, attention, the lengths grow; against the same steps run eagerly."""
    def make():
        cache = ops.token_cache(40, 2, 64, codes=torch.int8)
        table = torch.arange(40, device="cuda").view(2, 20).int().contiguous()
        k, v = draw(1, 2, 900, 2, 64, dtype=BF16), draw(2, 2, 900, 2, 64, dtype=BF16)
        ops.cache_write(cache, k, v, table, i32([0, 0]))
        return cache, table, i32([900, 640])

    def step(cache, table, start, x):
        ops.cache_write(cache, x[:, :, :2], x[:, :, 2:4], table, start)
        out = ops.cache_attention(x, cache, table, start)
        start.add_(1)
        return out

    x = draw(3, 2, 1, 8, 64, dtype=BF16)
    a, b = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step(*a, x)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, step(*b, x))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(*a, x)
    for i in range(6):
        x.copy_(draw(30 + i, 2, 1, 8, 64, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, step(*b, x)), i


def test_results_do_not_change_from_run_to_run():
    cache, model, table = filled(18, [3000, 100], 2, 64, "e4m3")
    q = draw(5, 2, 15, 8, 64, dtype=BF16)
    runs = [ops.cache_attention(q, cache, i32(table.tolist()), i32([2985, 85])) for _ in range(3)]
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_two_calls_at_once():
    """Calls that split their tokens, on two streams at the same time, and two captured ones replayed in turn."""
    cases = []
    for i, (n, T, dtype) in enumerate(((6000, 1, BF16), (5000, 40, F32))):
        cache, model, table = filled(20 + i, [n + T], 2, 64, "int8")
        q = draw(i, 1, T, 8, 64, dtype=dtype)
        cases.append((q, cache, i32(table.tolist()), i32([n])))
    want = [ops.cache_attention(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    held = [[], []]
    for _ in range(20):
        for s, c, h in zip(streams, cases, held):
            with torch.cuda.stream(s):
                h.append(ops.cache_attention(*c))
    torch.cuda.synchronize()
    for h, w in zip(held, want):
        assert all(torch.equal(x, w) for x in h)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in cases], []
    for g, c in zip(graphs, cases):
        with torch.cuda.graph(g):
            outs.append(ops.cache_attention(*c))
    for k in range(3):
        for (q, *_), g in zip(cases, graphs):
            q.mul_(-1 if k else 1)
            g.replay()
        torch.cuda.synchronize()
        for o, c in zip(outs, cases):
            assert torch.equal(o, ops.cache_attention(*c)), k
