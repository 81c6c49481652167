"""GPU: the decoder operators together, as a planner's decoder layer runs them, serving and training."""
import numpy as np
import pytest
import torch

import oracle.decoder as dec
from camera_bev_view_amd import ops
from decoder_bounds import KINDS
from gpu_helpers import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def draw(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).cuda()


class Layer:
    """Norm, projections to heads, rotary positions, cache and attention; then the residual and the next norm."""

    def __init__(self, C=128, Hq=8, Hk=2, D=32):
        self.C, self.Hq, self.Hk, self.D = C, Hq, Hk, D
        self.w1, self.w2 = draw(1, C) * 0.2 + 1, draw(2, C) * 0.2 + 1
        self.proj = draw(3, C, (Hq + 2 * Hk) * D) / C ** 0.5
        self.back = draw(4, Hq * D, C) / (Hq * D) ** 0.5
        self.freqs = ops.rotary_freqs((D // 2,), device="cuda")

    def heads(self, x, pos):
        B, T = x.shape[:2]
        y = ops.rms_norm(x, self.w1)
        qkv = (y @ self.proj).view(B, T, self.Hq + 2 * self.Hk, self.D)
        q, k, v = qkv.split((self.Hq, self.Hk, self.Hk), dim=2)
        q, k = ops.rotary_axes(q, k, pos.view(B, T, 1), self.freqs)
        return q, k, v

    def finish(self, x, a):
        return ops.rms_norm_add(a.flatten(2) @ self.back, x, self.w2)

    def serve(self, x, pos, cache, table, start, **how):
        q, k, v = self.heads(x, pos)
        ops.cache_write(cache, k, v, table, start)
        y, h = self.finish(x, ops.cache_attention(q, cache, table, start, **how))
        return y, h


def test_prompt_then_tokens_then_a_tree():
    """A prompt in one call and the same tokens one by one leave the same cache and (up to the split of the work) the same
    results; a tree of drafted tokens gives each branch what the branch alone would get."""
    layer = Layer()
    B, T = 2, 100
    x, pos = draw(5, B, T, 128), torch.arange(T, device="cuda", dtype=F32).expand(B, T).contiguous()
    table = torch.randperm(8, generator=torch.Generator().manual_seed(2)).int().view(2, 4).cuda().contiguous()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for kind in ("int8", "e4m3"):
        say(f"[case] decoder layer, {kind}")
        whole = ops.token_cache(8, 2, 32, codes=KINDS[kind])
        y, h = layer.serve(x, pos, whole, table, i32([0, 0]))
        steps = ops.token_cache(8, 2, 32, codes=KINDS[kind])
        start = i32([0, 0])
        got = []
        for t in range(T):
            got.append(layer.serve(x[:, t:t + 1], pos[:, t:t + 1].contiguous(), steps, table, start)[0])
            start.add_(1)
        # the projections of one token and of a hundred are other matrix products: keys differ in fp32's last digits, a code by a
        # step now and then, which moves an output by that step's share of a token's weight
        step = 2 / 127 if kind == "int8" else 2 / 16
        assert (torch.cat(got, 1) - y).abs().max() < step * float(y.abs().max())
        # branches 0-1-3 and 0-2 of a tree behind 100 tokens
        draft, dpos = draw(6, B, 4, 128), torch.tensor([[100., 101, 101, 102]] * 2, device="cuda")
        yt, _ = layer.serve(draft, dpos, whole, table, i32([T, T]), ancestors=ops.tree_ancestors([-1, 0, 0, 1]))
        for branch in ([0, 1, 3], [0, 2]):
            alone, _ = layer.serve(draft[:, branch].contiguous(), dpos[:, branch].contiguous(), whole, table, i32([T, T]))
            assert (alone[:, -1] - yt[:, branch[-1]]).abs().max() < step * float(y.abs().max())
            # the branch has replaced the tree's tokens: write the tree again
            layer.serve(draft, dpos, whole, table, i32([T, T]), ancestors=ops.tree_ancestors([-1, 0, 0, 1]))


def test_cached_attention_is_attention_on_what_the_cache_holds():
    """cache_attention against ops.attention_forward on the values that cache_read gives back: fp32 on both sides."""
    layer = Layer()
    x, pos = draw(7, 2, 150, 128), torch.rand((2, 150), generator=torch.Generator().manual_seed(1)).cuda() * 50
    cache = ops.token_cache(6, 2, 32)
    table, start = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with torch.no_grad():
        q, k, v = layer.heads(x, pos)
        ops.cache_write(cache, k, v, table, start)
        out = ops.cache_attention(q, cache, table, start, cap=20.0)
        kd, vd = ops.cache_read(cache, table, start, 150, dtype=F32)
        want, _ = ops.attention_forward(q.contiguous(), kd, vd, causal=True, cap=20.0)
    # both within (3 D + 2 n + 200) 2^-24 times twice the scores' size (at most 20) of the largest value
    bound = 2 * 2 * 20 * (3 * 32 + 2 * 150 + 200) * 2.0 ** -24 * float(vd.abs().max())
    assert (out - want).abs().max() <= bound


def test_training_step_gradients():
    """The layer without its cache: gradients of every parameter against fp64 autograd on the plain operators."""
    layer = Layer()
    x, pos, gy, gh = draw(8, 2, 40, 128), draw(9, 2, 40) * 10, draw(10, 2, 40, 128), draw(11, 2, 40, 128)
    params = dict(x=x, w1=layer.w1, w2=layer.w2, proj=layer.proj, back=layer.back)
    leaves = {n: p.clone().requires_grad_() for n, p in params.items()}
    layer.w1, layer.w2, layer.proj, layer.back = (leaves[n] for n in ("w1", "w2", "proj", "back"))
    q, k, v = layer.heads(leaves["x"], pos)
    y, h = layer.finish(leaves["x"], ops.query_attention(q, k, v, causal=True))
    torch.autograd.backward([y, h], [gy, gh])

    wide = {n: p.double().requires_grad_() for n, p in params.items()}
    norm = lambda a, w: a * torch.rsqrt(a.square().mean(-1, keepdim=True) + 1e-6) * w
    qkv = (norm(wide["x"], wide["w1"]) @ wide["proj"]).view(2, 40, 12, 32)
    theta = (pos.double()[..., None] * layer.freqs.double()).unsqueeze(2)
    def turn(a):
        a1, a2 = a[..., :16], a[..., 16:]
        return torch.cat((a1 * theta.cos() - a2 * theta.sin(), a2 * theta.cos() + a1 * theta.sin()), -1)
    qd, kd, vd = qkv.split((8, 2, 2), dim=2)
    qd, kd = turn(qd).transpose(1, 2), turn(kd).transpose(1, 2).repeat_interleave(4, 1)
    s = qd @ kd.transpose(2, 3) * 32 ** -0.5
    s = s.masked_fill(~torch.ones((40, 40), dtype=torch.bool, device="cuda").tril(), float("-inf"))
    a = (torch.softmax(s, -1) @ vd.transpose(1, 2).repeat_interleave(4, 1)).transpose(1, 2).flatten(2)
    hd = a @ wide["back"] + wide["x"]
    torch.autograd.backward([norm(hd, wide["w2"]), hd], [gy.double(), gh.double()])
    for n in params:
        rel = float((leaves[n].grad.double() - wide[n].grad).norm() / wide[n].grad.norm())
        say(f"[grad] {n}: rel {rel:.2e}")
        # chains of at most 320 products and sums through nine operators, each within a few hundred steps of 2^-24
        assert rel <= 9 * 320 * 2.0 ** -24, n


def test_norm_codes_as_the_left_side_of_a_product():
    """What the 8-bit output stands for, times a weight: within the codes' steps of the norm's own product."""
    x, r, w = draw(12, 64, 512).to(BF16), draw(13, 64, 512).to(BF16), draw(14, 512) * 0.2 + 1
    weight = draw(15, 512, 96) / 512 ** 0.5
    y, h, _ = ops.rms_norm_forward(x.float(), w, residual=r.float())
    codes, scales, h8 = ops.rms_norm_codes(x.float(), w, residual=r.float(), block=128)
    assert torch.equal(h, h8)
    values = (codes.float().view(64, 4, 128) * scales[..., None]).view(64, 512)
    # a code is off by at most 2^-4 of its value, or half of the smallest step
    assert ((values - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * scales.repeat_interleave(128, 1) + 1e-6).all()
    got, want = values.double() @ weight.double(), y.double() @ weight.double()
    bound = ((values - y).abs().double() @ weight.double().abs())
    assert ((got - want).abs() <= bound + 1e-9).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_branches_of_a_tree_get_what_they_would_get_alone(kind):
    """Attention of a tree's tokens against that of each branch as a chain, on the same rows of keys and values (so the same
    codes) behind a short cache, where a wrong mask shows: a chain over the whole tree, a tree without its siblings hidden."""
    say(f"[case] branches, {kind}")
    layer = Layer()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, B, n = i32([[3, 0], [1, 2]]), 2, [5, 62]
    past, draft = draw(20, B, 62, 128), draw(21, B, 5, 128)
    parents, depth = [-1, 0, 0, 1, 2], [0, 1, 1, 2, 2]
    branches = [[0, 1, 3], [0, 2, 4]]
    with torch.no_grad():
        _, pk, pv = layer.heads(past, torch.arange(62., device="cuda").expand(B, 62).contiguous())
        q, k, v = layer.heads(draft, torch.tensor([[m + d for d in depth] for m in n], dtype=F32, device="cuda"))

    def attend(pick, **how):
        cache = ops.token_cache(4, 2, 32, codes=KINDS[kind])
        ops.cache_write(cache, pk, pv, table, i32([0, 0]), count=i32(n))
        ops.cache_write(cache, k[:, pick], v[:, pick], table, i32(n))
        return ops.cache_attention(q[:, pick], cache, table, i32(n), **how)

    every = list(range(5))
    tree = attend(every, ancestors=ops.tree_ancestors(parents))
    # two sums of at most 67 tokens in fp32, scores of 32 products in three parts, all within a few steps of 2^-24 of their
    # sizes: 2 (3 D + 36) 2^-24 of the largest score and 2 (n + 64) 2^-24 of the largest value, twice
    size = float(max(v.abs().max(), pv.abs().max())) * 1.1
    score = float(q.norm(dim=-1).max() * max(k.norm(dim=-1).max(), pk.norm(dim=-1).max())) * 1.1 * 32 ** -0.5
    bound = 2 * (2 * (3 * 32 + 36) * score + 2 * (67 + 64)) * 2.0 ** -24 * size
    for branch in branches:
        alone = attend(branch)
        assert (alone - tree[:, branch]).abs().max() <= bound, branch
    # masks that are wrong: far outside
    chain, all_seen = attend(every), attend(every, ancestors=torch.full((1, 5, 1), 31, dtype=torch.int64, device="cuda"))
    none = attend(every, drafted=False)
    for b in range(B):
        for wrong in (chain, all_seen, none):
            assert (wrong[b, 3:] - tree[b, 3:]).abs().max() > 20 * bound, b
