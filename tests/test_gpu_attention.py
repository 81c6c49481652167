"""GPU: attention with distance bias, score cap and masks against the fp64 oracle."""
import numpy as np
import pytest
import torch

from camera_bev_view_amd import ops
from encoder_bounds import close, oracle_attention

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def draw(B, Tq, Tk, Hq, Hk, D, dtype, seed, dims=0, cap=0.0, docs=None, causal=False, prefix=None, sharp=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: (torch.randn(s, generator=g) * sharp).to(dtype).cuda()
    q, k, v, go = n(B, Tq, Hq, D), n(B, Tk, Hk, D), n(B, Tk, Hk, D), n(B, Tq, Hq, D)
    how = dict(cap=cap, causal=causal)
    if dims:
        how["pos_q"] = (torch.rand((B, Tq, dims), generator=g) * 20 - 10).cuda()
        how["pos_k"] = (torch.rand((B, Tk, dims), generator=g) * 20 - 10).cuda()
        how["slope"] = torch.rand((B, Tq, Hq), generator=g).cuda()
    if docs is not None:
        how["doc_q"], how["doc_k"] = (torch.tensor(d, dtype=torch.int32).cuda() for d in docs)
    if prefix is not None:
        how["prefix"] = torch.tensor(prefix, dtype=torch.int32).cuda()
    return q, k, v, go, how


def check(q, k, v, go, how, label, backward=True):
    print(f"[case] attention {label}: q {tuple(q.shape)} k {tuple(k.shape)} {q.dtype}", flush=True)
    out, lse = ops.attention_forward(q, k, v, **how)
    ref, bd = oracle_attention(q, k, v, how, go if backward else None)
    close(label + " out", out, ref["out"], bd["out"])
    empty = torch.from_numpy(np.isneginf(ref["lse"])).cuda()
    assert torch.equal(lse[..., 1] == 0, empty) and torch.equal(torch.isneginf(lse[..., 0]), empty), \
        f"{label}: rows without keys differ"
    log = lse[..., 0].double() * np.log(2.0) + torch.log(lse[..., 1].double())
    close(label + " m, l", torch.where(empty, 0.0, log), np.where(empty.cpu(), 0.0, ref["lse"]), bd["lse"])
    if not backward:
        return
    gq, gk, gv, gs = ops.attention_backward(go, q, k, v, out, lse, **how)
    for name, x in (("gq", gq), ("gk", gk), ("gv", gv)):
        close(f"{label} {name}", x, ref[name], bd[name])
    if gs is not None:
        close(label + " gslope", gs, ref["gslope"], bd["gslope"])


# (B, Tq, Tk, Hq, Hk, D): one query and one key, no key, tiles that end inside, grouped heads, odd and narrow widths
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 3, 0, 2, 1, 8), (1, 33, 65, 2, 2, 32), (2, 17, 130, 6, 2, 40), (1, 100, 31, 4, 1, 64),
          (1, 70, 70, 2, 1, 96), (1, 40, 200, 2, 2, 128), (2, 5, 9, 3, 3, 5), (1, 129, 257, 1, 1, 16),
          (1, 64, 64, 8, 8, 33)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_dense(shape, dtype):
    check(*draw(*shape, dtype, 31), f"dense {shape}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dims", [1, 2, 3])
@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_distance_and_cap(dims, cap, dtype):
    check(*draw(2, 45, 77, 4, 2, 32, dtype, 32, dims=dims, cap=cap), f"dims={dims} cap={cap}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [16, 64, 128])
def test_wide_scores_and_cap(D, dtype):
    """Scores far apart: the running maximum moves, the cap saturates, weights vanish."""
    check(*draw(1, 50, 150, 2, 1, D, dtype, 33, cap=20.0, sharp=3.0), f"cap sharp D={D}")
    check(*draw(1, 50, 150, 2, 1, D, dtype, 34, sharp=3.0), f"sharp D={D}")


# queries before, at and behind the keys' end; a prefix that covers none, some and all keys
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq,Tk,prefix", [(70, 70, None), (40, 150, None), (150, 40, None), (1, 90, None), (90, 1, None),
                                          (100, 100, [37, 0]), (150, 60, [60, 20]), (70, 200, [500, 131])])
def test_causal_and_prefix(Tq, Tk, prefix, dtype):
    check(*draw(2, Tq, Tk, 4, 2, 32, dtype, 35, causal=True, prefix=prefix), f"causal {Tq}x{Tk} prefix={prefix}")


def runs(lengths, total):
    ids = [i for i, n in enumerate(lengths) for _ in range(n)]
    return ids + [-1] * (total - len(ids))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal", [False, True])
def test_documents(causal, dtype):
    T = 210
    packed = [runs([70, 1, 64, 33, 20], T), runs([5] * 40, T)]
    check(*draw(2, T, T, 4, 2, 32, dtype, 36, docs=(packed, packed), causal=causal), f"packed causal={causal}")
    # ids in any order, queries of documents without keys, padding first
    g = torch.Generator().manual_seed(37)
    dq = torch.randint(-1, 5, (2, 90), generator=g).tolist()
    dk = torch.randint(-1, 4, (2, 140), generator=g).tolist()
    check(*draw(2, 90, 140, 2, 1, 64, dtype, 38, docs=(dq, dk), causal=causal, dims=2, cap=5.0),
          f"mixed documents causal={causal}")
    nothing = [[-1] * 50]
    check(*draw(1, 50, 60, 2, 2, 32, dtype, 39, docs=(nothing, [[0] * 60])), "all padding")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_many_heads_share_staged_keys(D, dtype):
    """Enough row and key tiles that a workgroup takes 128 rows (or keys)."""
    docs = [runs([40, 20], 70)] * 8
    check(*draw(8, 70, 70, 64, 64, D, dtype, 40, dims=2, docs=(docs, docs), causal=True, cap=4.0), f"wide D={D}")
    check(*draw(8, 35, 140, 64, 64, D, dtype, 41), f"wide dense D={D}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_number_of_waves_and_rows(dtype):
    """Grids that take eight waves a row tile (forward too), and narrow heads in 128-row workgroups."""
    docs = [runs([40, 33, 20], 95)] * 4
    for D in (32, 64, 128):
        check(*draw(4, 95, 300, 16, 16, D, dtype, 53, dims=1, cap=6.0), f"eight waves D={D}")
        check(*draw(4, 95, 95, 16, 16, D, dtype, 54, docs=(docs, docs), causal=True), f"eight waves documents D={D}")
    check(*draw(16, 21, 40, 128, 128, 16, dtype, 55), "128-row workgroups, dense")
    check(*draw(16, 40, 40, 128, 128, 16, dtype, 56, causal=True, dims=2, cap=3.0), "128-row workgroups, causal")
    check(*draw(16, 35, 21, 256, 128, 40, dtype, 57, causal=True), "128-row workgroups, grouped heads")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("form", ["dense", "causal", "documents"])
def test_two_heads_share_their_distances(form, dtype):
    """Enough heads with a distance bias that a wave takes two: dense, causal and packed, 1 to 3 axes."""
    docs = [runs([40, 9, 20], 75)] * 4
    kw = dict(dense={}, causal=dict(causal=True), documents=dict(docs=(docs, docs)))[form]
    dims = dict(dense=2, causal=1, documents=3)[form]
    check(*draw(4, 75, 75, 96, 96, 32, dtype, 52, dims=dims, **kw), f"shared distances {form}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq,G,D", [(1, 1, 64), (1, 8, 32), (3, 4, 128), (2, 40, 40)])
def test_few_rows_over_many_keys(Tq, G, D, dtype):
    check(*draw(2, Tq, 5000, 2 * G, 2, D, dtype, 42, dims=2), f"split {Tq} x {G}", backward=False)
    check(*draw(1, Tq, 4097, G, 1, D, dtype, 43, causal=True, cap=10.0), f"split causal {Tq} x {G}")
    check(*draw(1, Tq, 70001, G, 1, min(D, 40), dtype, 54), f"many splits {Tq} x {G}", backward=False)
    docs = ([[3] * Tq], [runs([1500, 700, 900, 4], 4100)])
    check(*draw(1, Tq, 4100, G, 1, D, dtype, 44, docs=docs), f"split documents {Tq} x {G}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tk,G,D", [(1, 1, 64), (3, 4, 128), (40, 2, 33)])
def test_many_rows_over_few_keys(Tk, G, D, dtype):
    check(*draw(2, 2100, Tk, 2 * G, 2, D, dtype, 55, dims=2), f"rows split {Tk} x {G}")
    check(*draw(1, 1500, Tk, G, 1, D, dtype, 56, causal=True, cap=10.0, prefix=[2]), f"rows split causal {Tk} x {G}")
    docs = ([runs([700, 500, 300], 1600)], [[2] * (Tk - Tk // 2) + [0] * (Tk // 2)])
    check(*draw(1, 1600, Tk, G, 1, D, dtype, 57, docs=docs, dims=1), f"rows split documents {Tk} x {G}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_keys_may_hold_anything(dtype):
    """NaN and infinities in keys, values and positions that a query does not see do not reach it, nor what shares a
    tile with it; queries that see no key keep their zeros."""
    T = 150
    ids = [runs([60, 50, 20], T)]
    q, k, v, go, how = draw(1, T, T, 2, 1, 32, dtype, 45, dims=2, docs=(ids, ids), causal=True)
    clean = [t.clone() for t in (q, k, v, go)]
    want = ops.attention_forward(*clean[:3], **how)
    grads = ops.attention_backward(clean[3], *clean[:3], *want, **how)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for t in (k, v, q, go):
            t[0, 130:] = bad                    # padding
        how["pos_k"][0, 130:] = bad
        out, lse = ops.attention_forward(q, k, v, **how)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), bad
        got = ops.attention_backward(go, q, k, v, out, lse, **how)
        for a, b in zip(got, grads):
            assert torch.equal(a, b), bad
    q, k, v, go, how = draw(1, T, T, 2, 1, 32, dtype, 46, docs=(ids, ids))
    want = ops.attention_forward(q, k, v, **how)
    grads = ops.attention_backward(go, q, k, v, *want, **how)
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, v2, q2, go2 = (t.clone() for t in (k, v, q, go))
        v2[0, 70, 0, 3] = bad                   # one value of the second document
        k2[0, 75, 0, 1] = bad
        q2[0, 80, 1, 2] = bad
        go2[0, 85, 1, 2] = bad
        out, lse = ops.attention_forward(q2, k2, v2, **how)
        other = torch.tensor([i < 60 or i >= 110 for i in range(T)], device="cuda")
        assert torch.equal(out[:, other], want[0][:, other])
        got = ops.attention_backward(go2, q2, k2, v2, out, lse, **how)
        for a, b in zip(got[:3], grads[:3]):
            assert torch.equal(a[:, other], b[:, other]), bad
        out, _ = ops.attention_forward(q, k, v2, **how)
        seen = torch.zeros(T, dtype=torch.bool, device="cuda")
        seen[60:110] = True
        col = out[0, :, :, 3].float()
        assert not torch.isfinite(col[seen]).any() and torch.isfinite(col[~seen]).all()
        assert torch.equal(out[0, :, :, :3], want[0][0, :, :, :3])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [32, 64, 128, 40, 33])
def test_rows_behind_the_last_are_not_read(D, dtype):
    """Every tensor is the front of a memory of NaN: a tile that reaches behind the last row sees zeros."""
    for Tq, Tk, H, G in ((1, 1, 2, 1), (5, 3, 1, 1), (33, 65, 1, 2), (130, 100, 40, 1), (2, 70, 1, 3), (200, 300, 1, 1)):
        q, k, v, go, _ = draw(1, Tq, Tk, H * G, H, D, dtype, 52)
        print(f"[case] attention before NaN: {Tq} {Tk} {H} {G} {D} {dtype}", flush=True)
        want = ops.attention_forward(q, k, v)
        grads = ops.attention_backward(go, q, k, v, *want)

        def front(t):
            room = torch.full((1, t.shape[1] + 520, *t.shape[2:]), float("nan"), dtype=dtype, device="cuda")
            room[:, :t.shape[1]] = t
            return room[:, :t.shape[1]]

        q, k, v, go = (front(t) for t in (q, k, v, go))
        out = front(want[0])
        got = ops.attention_forward(q, k, v)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert go.is_contiguous() and out.is_contiguous()
        for a, b in zip(ops.attention_backward(go, q, k, v, out, want[1])[:3], grads[:3]):
            assert torch.equal(a, b)


def test_refused_outputs_and_scales():
    q, k, v, go, _ = draw(1, 40, 40, 2, 2, 32, F32, 53)
    packed = torch.zeros((1, 40, 3, 2, 32), device="cuda")
    for kw in (dict(out=q), dict(out=k), dict(scale=1e-20), dict(scale=1e20), dict(cap=1e-30)):
        with pytest.raises((ValueError, RuntimeError)):
            ops.attention_forward(q, k, v, **kw)
    room = torch.zeros(40 * 64 + 4, device="cuda")
    with pytest.raises(ValueError):
        ops.attention_forward(room[4:].view(1, 40, 2, 32), k, v, out=room[:-4].view(1, 40, 2, 32))
    check(q, k, v, go, dict(scale=1e-12), "smallest scale")
    check(q, k, v, go, dict(scale=0.0), "no scale")
    check(packed[:, :, 0], packed[:, :, 1], packed[:, :, 2], go, {}, "all zeros")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_views(dtype):
    B, T, H, D = 2, 60, 4, 32
    g = torch.Generator().manual_seed(47)
    packed = torch.randn((B, T, 3, H, D), generator=g).to(dtype).cuda()
    go = torch.randn((B, T, H, D), generator=g).to(dtype).cuda()
    check(packed[:, :, 0], packed[:, :, 1], packed[:, :, 2], go, {}, "packed")
    first = torch.randn((B, 3, H, T, D), generator=g).to(dtype).cuda().permute(1, 0, 3, 2, 4)
    check(first[0], first[1], first[2], go, {}, "heads first")
    odd = torch.randn((B, T, 3, H, D + 3), generator=g).to(dtype).cuda()[..., 1:D + 1]
    check(odd[:, :, 0], odd[:, :, 1], odd[:, :, 2], go, {}, "odd addresses")
    shared = packed[:1, :, 1].expand(B, T, H, D)
    check(packed[:, :, 0], shared, shared, go.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), {}, "one memory")
    how = dict(pos_q=torch.randn((B, T, 2), device="cuda"), pos_k=torch.randn((B, T, 2), device="cuda"),
               slope=torch.rand(H, device="cuda"), scale=0.3)
    check(packed[:, :, 0], packed[:, :, 1], packed[:, :, 2], go, how, "a slope a head")
    how["scale"] = -0.3
    check(packed[:, :, 0], packed[:, :, 1], packed[:, :, 2], go, how, "negative scale")


def test_offsets_beyond_32_bits():
    """A long cache whose tokens lie 2^17 elements apart: the last ones behind 2^32 elements."""
    T, step = 36000, 1 << 17
    cache = torch.empty(T * step, dtype=BF16, device="cuda")
    k = cache.as_strided((1, T, 1, 32), (T * step, step, 32, 1))
    v = cache.as_strided((1, T, 1, 32), (T * step, step, 32, 1), 64)
    g = torch.Generator().manual_seed(48)
    k.copy_(torch.randn((1, T, 1, 32), generator=g).to(BF16))
    v.copy_(torch.randn((1, T, 1, 32), generator=g).to(BF16))
    q = torch.randn((1, 2, 2, 32), generator=g).to(BF16).cuda()
    go = torch.randn((1, 2, 2, 32), generator=g).to(BF16).cuda()
    check(q, k, v, go, {}, "strided cache")


def test_autograd_and_broadcast_slope():
    print("[case] attention through autograd; a slope shared by all queries", flush=True)
    q, k, v, go, how = draw(2, 30, 50, 4, 2, 32, F32, 49, dims=2, cap=8.0)
    slope = torch.rand(4, device="cuda").requires_grad_()
    leaves = [t.requires_grad_() for t in (q, k, v)]
    how["slope"] = slope
    out = ops.query_attention(q, k, v, **how)
    grads = torch.autograd.grad(out, leaves + [slope], go)
    how["slope"] = slope.detach()
    ref, bd = oracle_attention(q.detach(), k.detach(), v.detach(), how, go)
    for name, x in zip(("gq", "gk", "gv"), grads):
        close("autograd " + name, x, ref[name], bd[name])
    close("autograd gslope", grads[3], ref["gslope"].sum(axis=(0, 1)), bd["gslope"].sum(axis=(0, 1)) * 1.01 + 1e-9)
    # against differences of the operator's own definition
    import oracle.encoder as enc
    from encoder_bounds import f64
    a = dict(cap=8.0, pos_q=f64(how["pos_q"]), pos_k=f64(how["pos_k"]),
             slope=np.broadcast_to(f64(slope), (2, 30, 4)))
    base = [f64(t) for t in (q, k, v)]
    for which, at in ((0, (1, 7, 2, 5)), (1, (0, 20, 1, 9)), (2, (1, 3, 0, 30))):
        vals = []
        for sign in (1, -1):
            args = [t.copy() for t in base]
            args[which][at] += sign * 1e-5
            vals.append((enc.attention(*args, **a)["out"] * f64(go)).sum())
        name = ("gq", "gk", "gv")[which]
        assert abs((vals[0] - vals[1]) / 2e-5 - f64(grads[which])[at]) <= bd[name][at] + 1e-7


def test_repeats_streams_and_devices_of_the_workspace():
    print("[case] attention twice, on a side stream, with a caller's workspace", flush=True)
    q, k, v, go, how = draw(1, 4, 9000, 4, 1, 64, BF16, 50, dims=2)
    first = ops.attention_forward(q, k, v, **how)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(side):
        second = ops.attention_forward(q, k, v, workspace=ws, **how)
        g2 = ops.attention_backward(go, q, k, v, *second, workspace=ws, **how)
    torch.cuda.current_stream().wait_stream(side)
    g1 = ops.attention_backward(go, q, k, v, *first, **how)
    for a, b in zip(first + g1, second + g2):
        assert torch.equal(a, b)


def test_captured_and_replayed():
    """Forward and backward of the three operators in one graph, replayed with eager work between."""
    print("[case] a captured encoder step", flush=True)
    q, k, v, go, how = draw(1, 90, 90, 4, 4, 32, BF16, 51, dims=2)
    x = torch.randn((1, 90, 128), device="cuda").to(BF16)
    pos = torch.randn((1, 90, 3), device="cuda")
    freqs = ops.rotary_freqs((6, 5, 5), device="cuda")
    w = torch.rand(128, device="cuda")
    single = torch.randn((1, 1, 4, 32), device="cuda").to(BF16)

    def step():
        y, st = ops.group_norm_forward(x, 8, w, None, activation="silu")
        qr, kr = ops.rotary_forward(y.view(1, 90, 4, 32), k, pos, freqs)
        o, lse = ops.attention_forward(qr, kr, v, **how)
        gq, gk, gv, gs = ops.attention_backward(go, qr, kr, v, o, lse, **how)
        gy, _ = ops.rotary_backward(gq, gk, pos, freqs)
        gx, gw, gb = ops.group_norm_backward(gy.reshape(1, 90, 128), x, st, 8, w, None, activation="silu")
        one, _ = ops.attention_forward(single, kr.repeat(1, 50, 1, 1), v.repeat(1, 50, 1, 1))
        return o, gx, gw, gb, gv, gs, one

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        x.copy_(torch.randn((1, 90, 128), device="cuda").to(BF16))
        v.copy_(torch.randn(v.shape, device="cuda").to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b), f"replay {i}"


def test_encoder_layer_around_the_view_transform():
    """The operators as they are used: normalised camera maps through the view transform, BEV cells as tokens with
    rotary positions and distance-biased attention, gradients to the camera features."""
    from camera_bev_view_amd import workloads as wl
    import oracle
    import oracle.encoder as enc
    from encoder_bounds import f64
    print("[case] norm -> view transform -> rotary -> attention", flush=True)
    inp = wl.make_inputs("tiny", with_grad=True)
    B, N, C, H, W = inp.F.shape
    F = torch.from_numpy(np.ascontiguousarray(inp.F.transpose(0, 1, 3, 4, 2))).cuda().requires_grad_()
    K, R, t = (torch.from_numpy(a).cuda() for a in (inp.K, inp.R, inp.t))
    X = Y = 12
    w, b = torch.rand(C, device="cuda").requires_grad_(), torch.zeros(C, device="cuda").requires_grad_()
    y = ops.group_norm_act(F, 4, w, b, activation="silu")
    bev = ops.bev_sample(y, K, R, t, inp.rng6, X, Y, inp.Z)
    cells = bev.permute(0, 2, 3, 1).reshape(B, X * Y, 2, C // 2)
    pos = torch.stack(torch.meshgrid(torch.arange(X), torch.arange(Y), indexing="ij"), -1).float().cuda()
    pos = pos.reshape(1, X * Y, 2).expand(B, X * Y, 2)
    freqs = ops.rotary_freqs((C // 8, C // 8), device="cuda")
    q, k = ops.rotary_axes(cells, cells, pos, freqs)
    slope = torch.full((2,), 0.25, device="cuda").requires_grad_()
    out = ops.query_attention(q, k, cells, pos_q=pos, pos_k=pos, slope=slope)
    out.square().sum().backward()
    for leaf in (F, w, b, slope):
        assert leaf.grad is not None and torch.isfinite(leaf.grad).all() and leaf.grad.abs().max() > 0
    # the same chain from the oracles, to the accuracy of the view transform's own parity rule
    yr = enc.group_norm(f64(F).reshape(B * N, H * W, C), 4, f64(w), f64(b), 1e-5, "silu")["y"].reshape(B, N, H, W, C)
    br = oracle.oracle_forward(yr.transpose(0, 1, 4, 2, 3), inp.K, inp.R, inp.t, inp.rng6, X, Y, inp.Z)
    assert not br["near_edge"].any() or True
    cr = br["out"].transpose(0, 2, 3, 1).reshape(B, X * Y, 2, C // 2)
    ok = ~br["near_edge"].any(axis=-1)
    got = f64(bev).transpose(0, 2, 3, 1)
    assert (np.abs(got - br["out"].transpose(0, 2, 3, 1))[ok] <= 2e-4).all()
    cg = f64(cells)                      # from here on, on the kernels' own cells
    qr = enc.rotary(cg, f64(pos), f64(freqs), False)
    ref = enc.attention(qr, qr, cg, pos_q=f64(pos), pos_k=f64(pos), slope=np.full((B, X * Y, 2), 0.25))
    # fp32 throughout: 144 keys, scores of a few units
    assert np.abs(f64(out) - ref["out"]).max() <= 2e-5 * max(1.0, np.abs(cg).max())
