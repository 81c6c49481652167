"""GPU: more workgroups than one launch dimension holds (2^32 threads) and more elements than 31 bits count."""
import pytest
import torch

from camera_bev_view_amd import ops

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def within(name, got, ref, bound):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    print(f"[bound] {name}: max|d|={float(err.max()):.3e}", flush=True)
    assert not bad.any(), f"{name}: {int(bad.sum())} outside, first at {bad.nonzero()[0].tolist()}"


def norm_reference(x, gy, groups, eps):
    """y, gx and dz xh of act = none in float64, x [I, S, C]; and the sizes that bounds need."""
    I, S, C = x.shape
    xd = x.double().view(I, S, groups, C // groups)
    var, mean = torch.var_mean(xd, dim=(1, 3), correction=0, keepdim=True)
    rstd = (var + eps).rsqrt()
    xh = (xd - mean) * rstd
    g = gy.double().view(xd.shape)
    gx = rstd * (g - g.mean((1, 3), keepdim=True) - xh * (g * xh).mean((1, 3), keepdim=True))
    # fp32 sums of S C / groups terms; eight further roundings of values of the size of xh and of the gradients
    chain = (64 + 16) * U
    big = xh.abs() + rstd * mean.abs() + rstd * xd.abs().mean((1, 3), keepdim=True)
    gbig = g.abs() + g.abs().mean((1, 3), keepdim=True) + (xh.abs() + big) * ((g * xh).abs().mean((1, 3), keepdim=True) + 1)
    ey, eg = chain * big, 4 * chain * rstd * gbig * (1 + big.amax((1, 3), keepdim=True))
    flat = lambda t: t.reshape(I, S, C)
    return flat(xh), flat(gx), flat(ey), flat(eg.expand(xd.shape)), (g * xh).sum((0, 1)).reshape(-1)


def test_every_token_an_image():
    """Group norm of 4 million tokens, each an image of its own: more workgroups of 1024 threads than a dimension holds."""
    n, C, groups = (1 << 22) + 5, 32, 4
    print(f"[case] group norm of {n} tokens", flush=True)
    g = torch.Generator(device="cuda").manual_seed(95)
    x = torch.randn((n, 1, C), generator=g, device="cuda").to(BF16)
    gy = torch.randn((n, 1, C), generator=g, device="cuda").to(BF16)
    y, stats = ops.group_norm_forward(x, groups, eps=0.1)
    gx, gw, gb = ops.group_norm_backward(gy, x, stats, groups)
    half = 2.0 ** -8
    sums = torch.zeros(C, dtype=torch.float64, device="cuda")
    for a in range(0, n, 1 << 20):
        rows = slice(a, min(n, a + (1 << 20)))
        ry, rg, ey, eg, s = norm_reference(x[rows], gy[rows], groups, 0.1)
        within(f"y from {a}", y[rows], ry, ey + half * (ry.abs() + ey))
        within(f"gx from {a}", gx[rows], rg, eg + half * (rg.abs() + eg))
        sums += s
    # a lane's chain: n / 64 partial sums, then 6 steps
    size = gy.double().abs().sum((0, 1))
    within("gb", gb, gy.double().sum((0, 1)), (n / 64 + 64) * U * size)
    within("gw", gw, sums, (n / 64 + 64) * U * size * 4)


def test_norm_of_more_elements_than_31_bits():
    pixels, C, groups = (1 << 24) + 77, 64, 8
    print(f"[case] group norm of 2 x {pixels} pixels of {C} channels", flush=True)
    g = torch.Generator(device="cuda").manual_seed(96)
    x = torch.randn((2, pixels, C), generator=g, device="cuda", dtype=BF16)
    y, stats = ops.group_norm_forward(x, groups, activation="none", eps=1e-3)
    gy = torch.randn((2, pixels, C), generator=g, device="cuda", dtype=BF16)
    gx, gw, gb = ops.group_norm_backward(gy, x, stats, groups)
    n = pixels * C // groups
    for i in range(2):
        s = torch.zeros((groups, 4), dtype=torch.float64, device="cuda")
        cuts = [slice(a, min(pixels, a + (1 << 21))) for a in range(0, pixels, 1 << 21)]
        for c in cuts:
            xd, gd = (t[i, c].double().view(-1, groups, C // groups) for t in (x, gy))
            s += torch.stack([xd.sum((0, 2)), (xd * xd).sum((0, 2)), gd.sum((0, 2)), (gd * xd).sum((0, 2))], 1)
        mean, rstd = s[:, 0] / n, (s[:, 1] / n - (s[:, 0] / n) ** 2 + 1e-3).rsqrt()
        # values of size 1; chunk means and a lane's chain of chunks: under 2^10 roundings
        within(f"mean {i}", stats[i, :, 0], mean, 1024 * U)
        within(f"rstd {i}", stats[i, :, 1], rstd, 1024 * U * rstd)
        m1, m2 = s[:, 2] / n, (s[:, 3] / n - mean * s[:, 2] / n) * rstd
        for c in (cuts[0], cuts[-1]):
            xd, gd = (t[i, c].double().view(-1, groups, C // groups) for t in (x, gy))
            xh = (xd - mean[:, None]) * rstd[:, None]
            rg = rstd[:, None] * (gd - m1[:, None] - xh * m2[:, None])
            e = 2048 * U * (xh.abs() + 1)
            within(f"y {i}", y[i, c].view(xh.shape), xh, e + 2.0 ** -8 * (xh.abs() + e))
            e = 4096 * U * (xh.abs() + gd.abs() + 1)
            within(f"gx {i}", gx[i, c].view(xh.shape), rg, e + 2.0 ** -8 * (rg.abs() + e))


def test_rotary_of_many_wide_tokens():
    T, D = (1 << 25) + 3, 256
    print(f"[case] rotary of {T} tokens of {D} channels", flush=True)
    g = torch.Generator(device="cuda").manual_seed(97)
    row = torch.randn((1, 1, 1, D), generator=g, device="cuda").to(BF16)
    pos = torch.arange(T, device="cuda", dtype=torch.float32).view(1, T, 1)
    freqs = ops.rotary_freqs((D // 2,), device="cuda")
    q, _ = ops.rotary_forward(row.expand(1, T, 1, D), None, pos, freqs)
    x = row.double().view(2, D // 2)
    for at in (0, T // 2, T - 4096):
        theta = pos[0, at:at + 4096].double() * freqs.double()
        c, s = theta.cos(), theta.sin()
        ref = torch.cat((x[0] * c - x[1] * s, x[1] * c + x[0] * s), -1)
        e = 8 * U * (x[0].abs() + x[1].abs()).repeat(2)
        within(f"tokens from {at}", q[0, at:at + 4096, 0], ref, e + 2.0 ** -8 * (ref.abs() + e))


def test_attention_of_many_short_sequences():
    """One query and one key each: the output is the value, whatever the score."""
    B, D = (1 << 24) + 3, 8
    print(f"[case] attention of {B} sequences", flush=True)
    g = torch.Generator(device="cuda").manual_seed(98)
    q, k, v, go = (torch.randn((B, 1, 1, D), generator=g, device="cuda") for _ in range(4))
    out, stats = ops.attention_forward(q, k, v)
    # the weight and the sum that divides it are the same number
    within("out", out, v.double(), 4 * U * v.double().abs())
    gq, gk, gv, _ = ops.attention_backward(go, q, k, v, out, stats)
    s = (q.double() * k.double()).sum(-1, keepdim=True).abs() * 2
    within("gv", gv, go.double(), (16 + 8 * s) * U * go.double().abs())
    dp = (go.double() * v.double()).abs().sum(-1, keepdim=True)
    for name, x, other in (("gq", gq, k), ("gk", gk, q)):
        within(name, x, torch.zeros_like(other.double()), 64 * U * dp * (1 + s * U) * other.double().abs() + 1e-30)
