"""GPU: root-mean-square norm with the residual's addition, its backward and its output in 8 bits, against the fp64
oracle."""
import numpy as np
import pytest
import torch

import oracle.decoder as dec
from camera_bev_view_amd import _lib, ops
from decoder_bounds import HALF, KINDS, U, close, f64, norm_bounds
from gpu_helpers import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def draw(seed, *shape, dtype=F32, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * spread).to(dtype).cuda()


def check(x, residual, weight, eps, gy=None, gh=None, label=""):
    """Forward and backward of x [..., C] against the oracle."""
    C, dtype = x.shape[-1], x.dtype
    y, h, rstd = ops.rms_norm_forward(x, weight, residual=residual, eps=eps)
    if residual is None:
        assert h.data_ptr() == x.data_ptr() or not x.is_contiguous()
    else:
        assert torch.equal(h, (x.float() + residual.float()).to(dtype)), f"{label}: h"
    flat = lambda t: None if t is None else f64(t).reshape(-1, C)
    hn, wn = flat(h), None if weight is None else f64(weight)
    eps = float(np.float32(eps))                        # the call takes it in 32 bits
    ref = dec.rms_norm(hn, wn, eps, flat(gy) if gy is not None else None, flat(gh))
    b = norm_bounds(hn, wn, ref, dtype, flat(gy) if gy is not None else None, flat(gh))
    assert y.shape == x.shape and rstd.shape == x.shape[:-1]
    close(f"{label} y", y.reshape(-1, C), ref["y"], b["y"])
    close(f"{label} rstd", rstd.reshape(-1), ref["rstd"], b["rstd"])
    if gy is not None:
        gx, gw = ops.rms_norm_backward(gy, h, rstd, weight, grad_h=gh)
        # the backward takes the forward's rounded rstd: its error is in the bound
        close(f"{label} gx", gx.reshape(-1, C), ref["gx"], b["gx"])
        close(f"{label} gw", gw, ref["gw"], b["gw"])
        only, none = ops.rms_norm_backward(gy, h, rstd, weight, grad_h=gh, with_weight=False)
        assert none is None and torch.equal(only, gx)
    return y, h, rstd


# every width of a team (4 .. 1024 lanes, one to four pieces a lane), whole pieces and rows that end inside one
WIDTHS = [1, 3, 8, 31, 32, 33, 64, 100, 127, 128, 200, 256, 260, 511, 512, 777, 1001, 1024, 2047, 2048, 4096, 5000, 8192,
          16383, 16384]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C", WIDTHS)
def test_widths(C, dtype):
    rows = 1 if C > 8192 else 37 if C > 600 else 300
    say(f"[case] rms norm C={C} rows={rows} {dtype}")
    x, r, gy, gh = (draw(C + i, rows, C, dtype=dtype) for i in range(4))
    w = draw(C + 9, C) * 0.3 + 1
    check(x, r, w, 1e-6, gy, gh, "with residual")
    check(x, None, w, 1e-3, gy, None, "alone")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C", [(1, 256), (2, 40), (5, 32), (2049, 96), (10007, 24), (4096, 1000)])
def test_row_counts(rows, C, dtype):
    say(f"[case] rms norm rows={rows} C={C} {dtype}")
    x, gy = draw(rows, rows, C, dtype=dtype), draw(rows + 1, rows, C, dtype=dtype)
    check(x, None, None, 1e-5, gy, None, "no weight")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layouts(dtype):
    """Heads of a packed projection, broadcast rows, odd addresses, transposed channels, leading dimensions."""
    w = draw(5, 40)
    packed = draw(1, 6, 7, 3, 4, 40, dtype=dtype)
    for i in range(3):
        check(packed[:, :, i], None, w, 1e-6, draw(2, 6, 7, 4, 40, dtype=dtype), None, f"packed {i}")
    check(packed[:, :, 0], packed[:, :, 1], w, 1e-6, draw(2, 6, 7, 4, 40, dtype=dtype), None, "packed residual")
    row = draw(3, 1, 40, dtype=dtype)
    check(row.expand(9, 40), draw(4, 9, 40, dtype=dtype), w, 1e-6, label="broadcast")
    flat = draw(6, 41 * 40 + 3, dtype=dtype)
    check(flat[1:1 + 41 * 40].view(41, 40), None, w, 1e-6, flat[3:3 + 41 * 40].view(41, 40), None, "odd address")
    check(flat[:8 * 41].view(8, 41)[:, :40], None, w, 1e-6, label="rows 41 apart")
    check(draw(7, 40, 12, dtype=dtype).t(), None, w, 1e-6, draw(8, 12, 40, dtype=dtype), None, "transposed")
    check(draw(9, 40, dtype=dtype), None, w, 1e-6, draw(10, 40, dtype=dtype), None, "one row")
    check(draw(11, 3, 5, 4, 40, dtype=dtype).permute(1, 0, 2, 3), None, w, 1e-6, label="three strides")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_rows(dtype):
    x = torch.empty((0, 24), dtype=dtype, device="cuda")
    y, h, rstd = ops.rms_norm_forward(x, residual=x)
    assert y.shape == h.shape == (0, 24) and rstd.shape == (0,)
    gx, gw = ops.rms_norm_backward(x, h, rstd)
    assert gx.shape == (0, 24) and torch.equal(gw, torch.zeros(24, device="cuda"))
    c, s, _ = ops.rms_norm_codes(x, block=0)
    assert c.shape == (0, 24) and s.shape == (0, 1)


def test_odd_values_stay_in_their_rows():
    x, gy = draw(1, 40, 96), draw(2, 40, 96)
    good = ops.rms_norm_forward(x)
    bad = x.clone()
    bad[3, 5], bad[7, 0], bad[11, 95] = float("nan"), float("inf"), -float("inf")
    y, h, rstd = ops.rms_norm_forward(bad)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[3, 7, 11]] = False
    assert torch.equal(y[keep], good[0][keep]) and torch.equal(rstd[keep], good[2][keep])
    assert y[3].isnan().all() and y[7, 0].isnan() and (y[7, 1:] == 0).all()
    gx, _ = ops.rms_norm_backward(gy, h, rstd)
    assert torch.equal(gx[keep], ops.rms_norm_backward(gy, x, good[2])[0][keep]) and gx[3].isnan().all()
    c, s, _ = ops.rms_norm_codes(bad, block=32)
    cg, sg, _ = ops.rms_norm_codes(x, block=32)
    assert torch.equal(s[keep], sg[keep]) and torch.equal(c[keep].view(torch.uint8), cg[keep].view(torch.uint8))
    assert s[3].isnan().all() and (c[3].view(torch.uint8) == 0).all()
    # an infinity makes 1 / sqrt(mean) zero: its own block holds 0 * inf, the others zeros
    assert s[7, 0].isnan() and (s[7, 1:] == 2.0 ** -126).all() and (c[7].view(torch.uint8) & 127 == 0).all()
    z = torch.zeros((4, 96), device="cuda")
    assert (ops.rms_norm_forward(z)[0] == 0).all() and (ops.rms_norm_codes(z)[0].float() == 0).all()


def test_sizes_far_from_one():
    for k in (1e-15, 1e15):
        x, gy = draw(3, 20, 200) * k, draw(4, 20, 200)
        check(x, None, None, 0.0, gy, None, f"x {k}")


def check_codes(x, residual, weight, kind, block, eps=1e-6):
    C = x.shape[-1]
    codes, scales, h = ops.rms_norm_codes(x, weight, residual=residual, eps=eps, codes=KINDS[kind], block=block)
    if residual is not None:
        assert torch.equal(h, (x.float() + residual.float()).to(x.dtype))
    hn = f64(h).reshape(-1, C)
    eps = float(np.float32(eps))                        # the call takes it in 32 bits
    y = dec.rms_norm(hn, None if weight is None else f64(weight), eps)["y"]
    size = block if 0 < block < C else C
    blocks = -(-C // size)
    assert codes.shape == x.shape and codes.dtype == KINDS[kind] and scales.shape == (*x.shape[:-1], blocks)
    s = f64(scales).reshape(-1, blocks)
    got = dec.numbers(kind)[codes.contiguous().view(torch.uint8).cpu().numpy().reshape(-1, C)]
    assert np.isfinite(got).all()
    ladder = np.sort(np.unique(np.abs(dec.numbers(kind)[:127])))
    for i in range(blocks):
        part, c = y[:, i * size:(i + 1) * size], got[:, i * size:(i + 1) * size]
        want = np.maximum(np.abs(part).max(axis=1) / dec.MOST[kind], 2.0 ** -126)
        # rounded once
        assert (np.abs(s[:, i] - want) <= 1.001 * U * want).all(), f"scales of block {i}"
        q = np.abs(part / want[:, None])
        hi = np.clip(np.searchsorted(ladder, q), 1, len(ladder) - 1)
        least = np.minimum(np.abs(q - ladder[hi - 1]), np.abs(ladder[hi] - q))
        # the number nearest to the exact quotient, unless two are equally near to the fp64 value's last digits
        off = np.abs(np.abs(c) - q)
        assert (off <= least + 2.0 ** -40 * q).all(), f"block {i}: {float((off - least).max())}"
        assert (c * part >= 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("C,block", [(256, 128), (256, 64), (256, 32), (256, 0), (40, 32), (1000, 128), (33, 32),
                                     (100, 128), (4096, 128), (4100, 64), (9000, 32), (16384, 128), (16384, 0), (7, 0)])
def test_codes(C, block, kind, dtype):
    rows = 3 if C > 4000 else 101
    say(f"[case] rms codes C={C} block={block} {kind} {dtype}")
    x, r = draw(C, rows, C, dtype=dtype), draw(C + 1, rows, C, dtype=dtype)
    w = draw(C + 2, C) * 0.5 + 1
    check_codes(x, r, w, kind, block)
    check_codes(x * 1e-3, None, None, kind, block)


def test_codes_of_sizes_far_from_one():
    """Rows and weights near the ends of fp32's range: what the norm takes out or leaves in, scales at their least."""
    for kind in ("int8", "e4m3"):
        for size, weight, eps in ((1e30, 1.0, 1e-6), (1e-30, 1.0, 0.0), (1e-18, 1.0, 1e-6), (1.0, 5e37, 1e-6), (1.0, 1e-35, 1e-6),
                                  (1.0, 1e-37, 0.0), (3e37, 1e-30, 0.0)):
            say(f"[case] {kind} rows of {size}, weights of {weight}")
            x, w = draw(21, 20, 200) * size, (draw(22, 200) * 0.2 + 1).clamp(0.5, 1.5) * weight
            check_codes(x, None, w, kind, 64, eps)
            check_codes(x[:, :130], None, w[:130].clone(), kind, 0, eps)


def test_codes_of_views():
    packed = draw(1, 6, 7, 3, 4, 40, dtype=BF16)
    check_codes(packed[:, :, 1], None, draw(2, 40), "e4m3", 32)
    flat = draw(6, 41 * 45 + 3, dtype=BF16)
    check_codes(flat[1:1 + 41 * 45].view(41, 45), None, None, "int8", 32)


def test_in_place_sum_and_given_outputs():
    x, r, w = draw(1, 50, 96, dtype=BF16), draw(2, 50, 96, dtype=BF16), draw(3, 96)
    y0, h0, s0 = ops.rms_norm_forward(x, w, residual=r)
    for take in (0, 1):
        a, b = x.clone(), r.clone()
        into, out = (a, b)[take], torch.empty_like(x)
        y, h, s = ops.rms_norm_forward(a, w, residual=b, h_out=into, out=out)
        assert y is out and h is into and torch.equal(y, y0) and torch.equal(h, h0) and torch.equal(s, s0)
        assert torch.equal((b, a)[take], (r, x)[take])
    a, b = x.clone(), r.clone()
    c0, cs0, _ = ops.rms_norm_codes(x, w, residual=r)
    c, cs, h = ops.rms_norm_codes(a, w, residual=b, h_out=b)
    assert h is b and torch.equal(h, h0) and torch.equal(c.view(torch.uint8), c0.view(torch.uint8)) and torch.equal(cs, cs0)


def test_refusals():
    x, w = draw(1, 8, 32), draw(2, 32)
    for bad in (dict(weight=w.double()), dict(weight=draw(3, 31)), dict(residual=draw(4, 8, 31)),
                dict(residual=draw(4, 8, 32, dtype=BF16)), dict(h_out=torch.empty_like(x)), dict(out=x),
                dict(out=torch.empty((8, 32), dtype=BF16, device="cuda"))):
        with pytest.raises(ValueError):
            ops.rms_norm_forward(x, **bad)
    r = draw(5, 9, 32)
    with pytest.raises(ValueError, match="overlap"):
        ops.rms_norm_forward(r[:8], residual=x, h_out=r[1:])
    with pytest.raises(ValueError, match="overlap"):
        ops.rms_norm_forward(x, residual=r[:8], h_out=x, out=x)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ops.rms_norm_forward(x.half())
    with pytest.raises(_lib.FlashBevError, match="FBEV_MAX_RMS_CHANNELS"):
        ops.rms_norm_forward(torch.zeros((2, 16385), device="cuda"))
    with pytest.raises(_lib.FlashBevError, match="block"):
        ops.rms_norm_codes(x, block=16)
    with pytest.raises(_lib.FlashBevError, match="eps"):
        ops.rms_norm_forward(x, eps=float("nan"))
    y, h, s = ops.rms_norm_forward(x)
    for bad in (dict(grad_y=draw(1, 8, 31)), dict(grad_h=draw(1, 7, 32)), dict(rstd=s[:7]), dict(weight=w.to(BF16)),
                dict(workspace=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            ops.rms_norm_backward(**{**dict(grad_y=x, h=h, rstd=s), **bad})


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_autograd(dtype):
    x, r = draw(1, 30, 72, dtype=dtype).requires_grad_(), draw(2, 30, 72, dtype=dtype).requires_grad_()
    w = (draw(3, 72) * 0.3 + 1).requires_grad_()
    gy, gh = draw(4, 30, 72, dtype=dtype), draw(5, 30, 72, dtype=dtype)
    y, h = ops.rms_norm_add(x, r, w, eps=1e-3)
    torch.autograd.backward([y, h], [gy, gh])
    _, hd, sd = ops.rms_norm_forward(x.detach(), w.detach(), residual=r.detach(), eps=1e-3)
    gx, gw = ops.rms_norm_backward(gy, hd, sd, w.detach(), grad_h=gh)
    assert torch.equal(x.grad, gx) and torch.equal(r.grad, gx) and torch.equal(w.grad, gw)
    x.grad = w.grad = None
    ops.rms_norm(x, w, eps=1e-3).backward(gy)
    _, hd, sd = ops.rms_norm_forward(x.detach(), w.detach(), eps=1e-3)
    gx, gw = ops.rms_norm_backward(gy, hd, sd, w.detach())
    assert torch.equal(x.grad, gx) and torch.equal(w.grad, gw)
    # the sum alone, the norm alone, no weight
    x.grad = r.grad = None
    ops.rms_norm_add(x, r, eps=1e-3)[1].backward(gh)
    assert torch.equal(x.grad, gh) and torch.equal(r.grad, gh)
    x.grad = r.grad = None
    ops.rms_norm_add(x, r.detach(), eps=1e-3)[0].backward(gy)
    assert x.grad is not None and r.grad is None
    with pytest.raises(RuntimeError):
        g, = torch.autograd.grad(ops.rms_norm(x, w).sum(), x, create_graph=True)
        g.sum().backward()


def test_gradient_against_differences():
    """Central differences of the kernel's own forward, along one direction each for x and w.  Step e: the truncation is
    e^2 / 6 times the third derivative, below 40 r^3 |d|^3 a row here (rows of 64 with r near 1, |d| < 3), and a loss of
    fp32 outputs carries (ROW / 2 + 6) U of its terms over e."""
    x, w, gy = draw(1, 6, 64), draw(2, 64) * 0.3 + 1, draw(3, 6, 64)
    y, h, s = ops.rms_norm_forward(x, w)
    gx, gw = ops.rms_norm_backward(gy, h, s, w)
    e = 2.0 ** -8
    loss = lambda a, b: (ops.rms_norm_forward(a, b)[0].double() * gy.double()).sum().item()
    terms = (y.double() * gy.double()).abs().sum().item()
    for name, g, dx, dw in (("x", gx, draw(4, 6, 64), None), ("w", gw, None, draw(5, 64))):
        d = dx if dx is not None else dw
        d = d.clamp(-3, 3)
        lo, hi = (loss(x - e * d, w), loss(x + e * d, w)) if dx is not None else (loss(x, w - e * d), loss(x, w + e * d))
        want = (g.double() * d.double()).sum().item()
        size = (gy.abs().sum(-1) * w.abs().max()).sum().item()
        bound = 40 * size * 27 * e * e / 6 + 2 * 44 * U * terms * 1.1 / (2 * e) + 200 * U * (g.abs() * d.abs()).sum().item()
        say(f"[bound] differences along {name}: {abs((hi - lo) / (2 * e) - want):.3e} of {bound:.3e}")
        assert abs((hi - lo) / (2 * e) - want) <= bound


def test_graph_replays_and_streams():
    x, r, gy = (draw(i, 300, 256, dtype=BF16) for i in (1, 2, 4))
    w = draw(3, 256)

    def layer():
        y, h, s = ops.rms_norm_forward(x, w, residual=r)
        gx, gw = ops.rms_norm_backward(gy, h, s, w, grad_h=gy)
        return [y, h, s, gx, gw, *ops.rms_norm_codes(x, w, residual=r)[:2]]

    bits = lambda ts: [t.contiguous().view(torch.uint8).clone() for t in ts]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = bits(layer())
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(on_side, bits(layer())):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for k in range(4):
        x.copy_(draw(50 + k, 300, 256, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(bits(held), bits(layer())):
            assert torch.equal(a, b), k


def test_more_workgroups_than_a_launch_dimension_holds():
    rows, C = (1 << 27) + 77, 8
    say(f"[case] rms norm of {rows} rows of {C}")
    x = draw(1, 1, C, dtype=BF16)
    y, h, s = ops.rms_norm_forward(x.expand(rows, C))
    want = ops.rms_norm_forward(x)
    for a in range(0, rows, 1 << 24):
        assert (y[a:a + (1 << 24)] == want[0]).all() and (s[a:a + (1 << 24)] == want[2]).all()
    gx, gw = ops.rms_norm_backward(y, x.expand(rows, C), s)
    wx, w1 = ops.rms_norm_backward(want[0], x, want[2])
    assert (gx[-1000:] == wx).all() and (gx[:1000] == wx).all()
    # equal terms: the sum of n of them by chains of at most n / (1024 * 64) rounds, then 64 + 32 + 32 + 6 shares
    bound = (rows / 65536 + 256) * U * rows * w1.abs().double()
    assert ((gw.double() - rows * w1.double()).abs() <= bound).all()


def test_gradients_of_shared_and_broadcast_inputs():
    w = (draw(3, 96) * 0.3 + 1).requires_grad_()
    x = draw(1, 1, 96).requires_grad_()
    gy, gh = draw(4, 40, 96), draw(5, 40, 96)
    wide = x.expand(40, 96)
    torch.autograd.backward(ops.rms_norm_add(wide, wide, w), [gy, gh])
    _, h, s = ops.rms_norm_forward(wide.detach(), w.detach(), residual=wide.detach())
    gx, gw = ops.rms_norm_backward(gy, h, s, w.detach(), grad_h=gh)
    # both addends: twice the rows' sum, of 80 terms in another order
    want = 2 * gx.double().sum(0)
    assert ((x.grad[0].double() - want).abs() <= 80 * U * 2 * gx.double().abs().sum(0)).all()
    assert torch.equal(w.grad, gw)
    # two leaves of one sum have gradients of their own memory
    a, b = draw(6, 40, 96).requires_grad_(), draw(7, 40, 96).requires_grad_()
    torch.autograd.backward(ops.rms_norm_add(a, b, w), [gy, gh])
    before = b.grad.clone()
    a.grad.mul_(3)
    assert torch.equal(b.grad, before)


def test_captured_training_step():
    """Both directions through autograd in a graph, replayed between eager steps on the same memory."""
    x, r, w = draw(1, 500, 256, dtype=BF16), draw(2, 500, 256, dtype=BF16), draw(3, 256) * 0.2 + 1
    gy, gh = draw(4, 500, 256, dtype=BF16), draw(5, 500, 256, dtype=BF16)

    def step():
        leaves = [t.detach().requires_grad_() for t in (x, r, w)]
        y, h = ops.rms_norm_add(*leaves)
        return [y.detach(), h.detach(), *torch.autograd.grad([y, h], leaves, [gy, gh])]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        x.copy_(draw(60 + k, 500, 256, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b), k
