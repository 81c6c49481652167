"""GPU: rotary positions with several axes against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle.encoder as enc
from camera_bev_view_amd import ops
from encoder_bounds import HALF, U, close, f64

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def draw(B, T, Hq, Hk, D, A, P, dtype, seed, far=50.0):
    g = torch.Generator().manual_seed(seed)
    q, k = torch.randn((B, T, Hq, D), generator=g).to(dtype), torch.randn((B, T, Hk, D), generator=g).to(dtype)
    pos = (torch.rand((B, T, A), generator=g) * 2 - 1) * far
    freqs = torch.rand((A, P), generator=g)
    return q.cuda(), k.cuda(), pos.cuda(), freqs.cuda()


def bound(x, P, interleaved, ref, dtype, theta):
    """A rotated pair of length r: sine and cosine off by 4 U (polynomials, the quarter turn's rounding) and by what
    the double-precision angle is off (2^-50 of it), three fp32 roundings, one rounding to the type."""
    x = np.abs(x)
    e = np.zeros_like(x)
    i1 = np.arange(P) * 2 if interleaved else np.arange(P)
    i2 = i1 + 1 if interleaved else i1 + P
    r = x[..., i1] + x[..., i2]
    e[..., i1] = e[..., i2] = r * (8 * U + 2.0 ** -50 * np.abs(theta)[:, :, None])
    turned = np.zeros(x.shape[-1], bool)
    turned[i1] = turned[i2] = True
    return e + HALF[dtype] * (np.abs(ref) + e) * turned


def check(q, k, pos, freqs, interleaved, label):
    P = freqs.shape[1]
    fwd = ops.rotary_forward(q, k, pos, freqs, interleaved=interleaved)
    bwd = ops.rotary_backward(q, k, pos, freqs, interleaved=interleaved)
    pn, fn = f64(pos), f64(freqs)
    theta = np.abs(pn) @ np.abs(fn)
    for inverse, outs in ((False, fwd), (True, bwd)):
        for name, x, y in (("q", q, outs[0]), ("k", k, outs[1])):
            if x is None:
                assert y is None
                continue
            ref = enc.rotary(f64(x), pn, fn, interleaved, inverse)
            close(f"{label} {name} inverse={inverse}", y, ref, bound(f64(x), P, interleaved, ref, x.dtype, theta))


# one token, one pair, odd channel counts and pairs that fit no wide piece, many tokens, many pairs
CASES = [(1, 1, 1, 1, 2, 1, 1), (2, 7, 3, 1, 40, 3, 18), (1, 900, 8, 8, 32, 3, 16), (3, 33, 4, 2, 64, 2, 32),
         (1, 257, 2, 2, 80, 1, 40), (2, 5, 1, 3, 7, 2, 3), (1, 19, 2, 1, 600, 8, 300), (1, 70, 2, 2, 36, 3, 6)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_shapes(case, interleaved, dtype):
    print(f"[case] rotary {case} interleaved={interleaved} {dtype}", flush=True)
    check(*draw(*case, dtype, 21), interleaved, str(case))


def test_far_positions():
    print("[case] rotary at positions of 1e6 and at multiples of a quarter turn", flush=True)
    check(*draw(1, 300, 2, 1, 32, 3, 16, F32, 22, far=1e6), False, "far")
    q, k, pos, freqs = draw(1, 64, 1, 1, 8, 1, 4, F32, 23)
    pos = (torch.arange(64, device="cuda", dtype=F32) - 32).reshape(1, 64, 1) * (np.pi / 4)
    check(q, k, pos, torch.ones((1, 4), device="cuda"), True, "quarter turns")


def test_one_tensor_views_and_in_place():
    print("[case] rotary of one tensor, of packed and permuted views, in place", flush=True)
    q, k, pos, freqs = draw(2, 31, 4, 4, 32, 3, 12, BF16, 24)
    check(q, None, pos, freqs, False, "q alone")
    check(None, k, pos, freqs, True, "k alone")
    packed = torch.randn((2, 31, 3, 4, 32), device="cuda").to(BF16)
    check(packed[:, :, 0], packed[:, :, 1], pos, freqs, False, "packed")
    heads_first = torch.randn((2, 4, 31, 32), device="cuda").to(BF16).permute(0, 2, 1, 3)
    check(heads_first, k, pos, freqs, True, "heads first")
    odd = torch.randn((2, 31, 4, 37), device="cuda").to(BF16)[..., 3:35]
    check(odd, k, pos, freqs, True, "odd addresses, interleaved")
    check(odd, k, pos, freqs, False, "odd addresses")
    a, b = q.clone(), k.clone()
    want = ops.rotary_forward(q, k, pos, freqs)
    got = ops.rotary_forward(a, b, pos, freqs, q_out=a, k_out=b)
    assert got[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1])
    wide = torch.zeros((2, 31, 4, 40), device="cuda", dtype=BF16)
    ops.rotary_forward(q, None, pos, freqs, q_out=wide[..., :32])
    assert torch.equal(wide[..., :32], want[0]) and (wide[..., 32:] == 0).all()
    # memory that another token's turn still reads
    room = torch.zeros((2 * 31 * 4 * 32 + 8,), device="cuda", dtype=BF16)
    first, later = (room[at:at + 2 * 31 * 4 * 32].view(2, 31, 4, 32) for at in (0, 8))
    for x, out in ((first, later), (q, q.view(2, 31, 4, 32).as_strided((2, 31, 4, 32), (4 * 31 * 32, 32, 31 * 32, 1)))):
        with pytest.raises(ValueError):
            ops.rotary_forward(x, None, pos, freqs, q_out=out)


def test_empty_and_table():
    print("[case] rotary of nothing; the frequency table", flush=True)
    q, k, pos, freqs = draw(2, 0, 4, 4, 32, 3, 12, F32, 25)
    a, b = ops.rotary_forward(q, k, pos, freqs)
    assert a.shape == q.shape and b.shape == k.shape
    t = ops.rotary_freqs((2, 0, 3), base=100.0)
    assert t.shape == (3, 5) and (t[0, 2:] == 0).all() and (t[1] == 0).all() and (t[2, :2] == 0).all()
    assert torch.allclose(t[2, 2:], torch.tensor([1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)]))


def test_autograd_is_the_transpose():
    print("[case] rotary through autograd", flush=True)
    q, k, pos, freqs = draw(1, 20, 2, 1, 16, 2, 8, F32, 26)
    q.requires_grad_()
    k.requires_grad_()
    a, b = ops.rotary_axes(q, k, pos, freqs)
    ga, gb = torch.randn_like(a), torch.randn_like(b)
    gq, gk = torch.autograd.grad((a, b), (q, k), (ga, gb))
    want = ops.rotary_backward(ga, gb, pos, freqs)
    assert torch.equal(gq, want[0]) and torch.equal(gk, want[1])
    # <g, R x> = <R^T g, x>; 16 products of 20 tokens, each off by a few U
    lhs, rhs = (f64(ga) * f64(a)).sum(), (f64(gq) * f64(q)).sum()
    assert abs(lhs - rhs) <= 32 * U * (np.abs(f64(ga)) * (np.abs(f64(a)) + 1)).sum() * 4
    only = torch.autograd.grad(ops.rotary_axes(q, None, pos, freqs)[0], q, ga)[0]
    assert torch.equal(only, want[0])
