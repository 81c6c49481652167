"""GPU: group norm with an activation on channels-last maps against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle.encoder as enc
from camera_bev_view_amd import ops
from encoder_bounds import close, f64, norm_bounds

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def draw(shape, dtype, seed, affine=True):
    g = torch.Generator().manual_seed(seed)
    C = shape[-1]
    x = (torch.randn(shape, generator=g) * (0.5 + torch.rand(C, generator=g)) + torch.randn(C, generator=g)).to(dtype)
    gy = torch.randn(shape, generator=g).to(dtype)
    w = (0.5 + torch.rand(C, generator=g)) if affine else None
    b = 0.2 * torch.randn(C, generator=g) if affine else None
    return x, gy, w, b


def check(x, gy, w, b, groups, kind, label, image_dims=None, eps=1e-5):
    dtype, C = x.dtype, x.shape[-1]
    lead = (2 if x.dim() == 5 else 1) if image_dims is None else image_dims
    I = int(np.prod(x.shape[:lead]))
    y, stats = ops.group_norm_forward(x, groups, w, b, eps=eps, activation=kind, image_dims=image_dims)
    gx, gw, gb = ops.group_norm_backward(gy, x, stats, groups, w, b, activation=kind, image_dims=image_dims)
    xs, gs = f64(x).reshape(I, -1, C), f64(gy).reshape(I, -1, C)
    wn, bn = (None if p is None else f64(p) for p in (w, b))
    ref = enc.group_norm(xs, groups, wn, bn, eps, kind, gs)
    bd = norm_bounds(xs, groups, wn, bn, kind, ref, gs, dtype)
    assert y.shape == x.shape and gx.shape == x.shape and y.dtype == dtype and gx.dtype == dtype
    close(label + " y", y.reshape(I, -1, C), ref["y"], bd["y"])
    close(label + " gx", gx.reshape(I, -1, C), ref["gx"], bd["gx"])
    close(label + " gw", gw, ref["gw"], bd["gw"])
    close(label + " gb", gb, ref["gb"], bd["gb"])


# (shape, groups): one pixel, one channel a group, groups that cut the 16-byte pieces, odd channel counts, whole images
# in one workgroup, images in chunks (the last one short), more channels than a workgroup has pieces, one group
SHAPES = [((1, 1, 4), 1), ((3, 5, 7, 6), 6), ((2, 3, 4, 5, 80), 16), ((2, 9, 13, 81), 27), ((1, 8, 22, 64), 8),
          ((3, 300, 12), 4), ((1, 2, 64, 176, 32), 4), ((2, 70, 70, 20), 4), ((1, 5, 9, 2064), 16), ((2, 40, 40, 36), 1),
          ((1, 3000, 10), 5),
          # more chunks than a workgroup joins by itself: forward and backward, backward alone, a wide slab, odd channels
          ((1, 100, 130, 128), 32), ((2, 90, 150, 36), 9), ((2, 1, 700, 1, 1032), 3), ((1, 150, 150, 27), 9),
          # workgroups enough for longer chunks in the backward
          ((9, 70, 60, 128), 32), ((40, 33, 31, 45), 9), ((3, 700, 1032), 43)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_shapes(shape, groups, dtype):
    print(f"[case] group norm {shape} groups={groups} {dtype}", flush=True)
    x, gy, w, b = draw(shape, dtype, 11)
    if shape[-2] == 1:
        gy = gy * 0 + 1     # two elements a group: only the parameters' sums and zeros come back
    check(x.cuda(), gy.cuda(), w.cuda(), b.cuda(), groups, "silu", f"{shape}/{groups}")


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("shape,groups", [((2, 6, 10, 24), 3), ((1, 64, 80, 40), 8)])
def test_activations(kind, shape, groups):
    print(f"[case] group norm {kind} {shape}", flush=True)
    x, gy, w, b = draw(shape, BF16 if shape[0] == 2 else F32, 12)
    check(x.cuda(), gy.cuda(), w.cuda(), b.cuda(), groups, kind, kind)


def test_without_weight_and_bias_and_far_from_zero():
    print("[case] group norm without parameters; values far from zero", flush=True)
    x, gy, _, _ = draw((2, 50, 50, 16), F32, 13, affine=False)
    check(x.cuda(), gy.cuda(), None, None, 4, "gelu", "no parameters")
    check((x + 1000.0).cuda(), gy.cuda(), None, None, 4, "none", "far", eps=1e-3)


def test_strided_maps_and_odd_addresses():
    print("[case] group norm of channel slices, row strides and addresses off 16 bytes", flush=True)
    x, gy, w, b = draw((2, 12, 20, 32), BF16, 14)
    wide = torch.zeros((2, 12, 20, 72), dtype=BF16, device="cuda")
    wide[..., 5:37] = x.cuda()
    check(wide[..., 5:37], gy.cuda(), w.cuda(), b.cuda(), 4, "silu", "slice at 5")
    wide[..., 8:40] = x.cuda()
    check(wide[..., 8:40], gy.cuda(), w.cuda(), b.cuda(), 4, "silu", "slice at 8")
    tall = torch.zeros((2, 12, 30, 32), dtype=BF16, device="cuda")
    tall[:, :, :20] = x.cuda()      # pixels no longer one stride: the binding copies
    check(tall[:, :, :20], gy.cuda(), w.cuda(), b.cuda(), 4, "silu", "cropped rows")
    first = x[:1].cuda().expand(2, 12, 20, 32)
    check(first, gy.cuda(), w.cuda(), b.cuda(), 4, "silu", "one image twice")
    check(x.cuda().reshape(24, 20, 32), gy.cuda().reshape(24, 20, 32), w.cuda(), b.cuda(), 4, "silu", "rows as images")
    check(x.cuda(), gy.cuda(), w.cuda(), b.cuda(), 4, "silu", "all as one image", image_dims=0)
    same = x.cuda()
    with pytest.raises(ValueError):
        ops.group_norm_forward(same, 4, out=same)


def test_empty_and_nan():
    print("[case] group norm of nothing; a NaN stays in its image and group", flush=True)
    w = torch.ones(8, device="cuda")
    for shape in ((0, 4, 8), (3, 0, 8)):
        x = torch.empty(shape, device="cuda")
        y, st = ops.group_norm_forward(x, 2, w, w)
        gx, gw, gb = ops.group_norm_backward(x, x, st, 2, w, w)
        assert y.shape == x.shape and gx.shape == x.shape
        assert (gw == 0).all() and (gb == 0).all()
    x, gy, w, b = draw((2, 40, 16), F32, 15)
    x[1, 7, 5] = float("nan")
    y, _ = ops.group_norm_forward(x.cuda(), 4, w.cuda(), b.cuda(), activation="relu")
    bad = torch.isnan(y.cpu())
    assert bad[1, :, 4:8].all() and not bad[0].any() and not bad[1, :, :4].any() and not bad[1, :, 8:].any()


def test_autograd_and_differences():
    print("[case] group norm through autograd, against central differences", flush=True)
    x, gy, w, b = (t.cuda() for t in draw((1, 3, 4, 12), F32, 16))
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    y = ops.group_norm_act(leaves[0], 3, leaves[1], leaves[2], activation="gelu")
    grads = torch.autograd.grad(y, leaves, gy)
    xs = f64(x).reshape(1, -1, 12)
    ref = enc.group_norm(xs, 3, f64(w), f64(b), 1e-5, "gelu", f64(gy).reshape(1, -1, 12))
    bd = norm_bounds(xs, 3, f64(w), f64(b), "gelu", ref, f64(gy).reshape(1, -1, 12), F32)
    close("autograd gx", grads[0].reshape(1, -1, 12), ref["gx"], bd["gx"])
    close("autograd gw", grads[1], ref["gw"], bd["gw"])
    close("autograd gb", grads[2], ref["gb"], bd["gb"])
    f = lambda a: (enc.group_norm(a, 3, f64(w), f64(b), 1e-5, "gelu")["y"] * f64(gy).reshape(1, -1, 12)).sum()
    for at in ((0, 0, 0), (0, 5, 7), (0, 11, 11)):
        e = np.zeros_like(xs)
        e[at] = 1e-5
        # a central difference of step 1e-5 is off by about 1e-10 of the third derivative and 1e-11 of rounding
        assert abs((f(xs + e) - f(xs - e)) / 2e-5 - f64(grads[0]).reshape(1, -1, 12)[at]) <= bd["gx"][at] + 1e-8


def test_repeats_are_bit_equal_and_streams_do_not_matter():
    print("[case] group norm twice and on a side stream", flush=True)
    x, gy, w, b = (t.cuda() for t in draw((3, 60, 70, 48), BF16, 17))
    run = lambda: (lambda f: f + ops.group_norm_backward(gy, x, f[1], 6, w, b, activation="silu"))(
        ops.group_norm_forward(x, 6, w, b, activation="silu"))
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run()
    torch.cuda.current_stream().wait_stream(side)
    for a, c in zip(first, second):
        assert torch.equal(a, c)
