"""GPU: the gradients of the encoder operators around the view transform, step by step against the oracles."""
import numpy as np
import pytest
import torch

import oracle
import oracle.encoder as enc
from camera_bev_view_amd import ops
from camera_bev_view_amd import workloads as wl
from encoder_bounds import U, close, f64, norm_bounds
from encoder_fine_bounds import oracle as attention_oracle
from gpu_helpers import BWD_REL_L2, rel_l2

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_gradients_from_the_attention_to_the_camera_features():
    """norm -> view transform -> rotary -> attention; each step's gradient from the one that the kernels handed it."""
    print("[case] gradients of norm -> view transform -> rotary -> attention", flush=True)
    inp = wl.make_inputs("tiny", with_grad=True)
    B, N, C, H, W = inp.F.shape
    F = torch.from_numpy(np.ascontiguousarray(inp.F.transpose(0, 1, 3, 4, 2))).cuda().requires_grad_()
    K, R, t = (torch.from_numpy(a).cuda() for a in (inp.K, inp.R, inp.t))
    X = Y = 12
    g = torch.Generator().manual_seed(101)
    w = (0.5 + torch.rand(C, generator=g)).cuda().requires_grad_()
    b = (0.2 * torch.randn(C, generator=g)).cuda().requires_grad_()
    y = ops.group_norm_act(F, 4, w, b, activation="silu")
    bev = ops.bev_sample(y, K, R, t, inp.rng6, X, Y, inp.Z)
    cells = bev.permute(0, 2, 3, 1).reshape(B, X * Y, 2, C // 2)
    pos = torch.stack(torch.meshgrid(torch.arange(X), torch.arange(Y), indexing="ij"), -1).float().cuda()
    pos = pos.reshape(1, X * Y, 2).expand(B, X * Y, 2)
    freqs = ops.rotary_freqs((C // 8, C // 8), device="cuda")
    q, k = ops.rotary_axes(cells, cells, pos, freqs)
    slope = torch.full((2,), 0.25, device="cuda").requires_grad_()
    out = ops.query_attention(q, k, cells, pos_q=pos, pos_k=pos, slope=slope)
    go = torch.randn(out.shape, generator=g).cuda()
    for x in (y, bev, cells, q, k):
        x.retain_grad()
    out.backward(go)

    # attention and rotary: what the cells get as queries, keys and values
    how = dict(pos_q=pos, pos_k=pos, slope=slope.detach().expand(B, X * Y, 2))
    ref, bd = attention_oracle(q.detach(), k.detach(), cells.detach(), how, go)
    close("chain gq", q.grad, ref["gq"], bd["gq"])
    close("chain gk", k.grad, ref["gk"], bd["gk"])
    close("chain gslope", slope.grad, ref["gslope"].sum((0, 1)), bd["gslope"].sum((0, 1)) * 1.01
          + 2 * X * Y * U * np.abs(ref["gslope"]).sum((0, 1)))
    turned = [enc.rotary(f64(x.grad), f64(pos), f64(freqs), False, inverse=True) for x in (q, k)]
    half = C // 4
    pair = lambda x: np.tile(np.abs(x)[..., :half] + np.abs(x)[..., half:2 * half], 2)
    e = 8 * U * (pair(f64(q.grad)) + pair(f64(k.grad)))
    total = turned[0] + turned[1] + ref["gv"]
    close("chain cells", cells.grad, total, e + bd["gv"] + 4 * U * (np.abs(turned[0]) + np.abs(turned[1]) + np.abs(ref["gv"])))
    assert torch.equal(bev.grad, cells.grad.reshape(B, X, Y, C).permute(0, 3, 1, 2))
    # the view transform
    rg = oracle.oracle_backward(f64(bev.grad), inp.K, inp.R, inp.t, inp.rng6, X, Y, inp.Z, H, W)
    err = rel_l2(f64(y.grad), rg.transpose(0, 1, 3, 4, 2))
    print(f"[parity] chain view transform: rel L2 = {err:.3e}", flush=True)
    assert err <= BWD_REL_L2
    # the norm
    xs, gs = f64(F).reshape(B * N, H * W, C), f64(y.grad).reshape(B * N, H * W, C)
    rn = enc.group_norm(xs, 4, f64(w), f64(b), 1e-5, "silu", gs)
    bn = norm_bounds(xs, 4, f64(w), f64(b), "silu", rn, gs, torch.float32)
    close("chain gx", F.grad.reshape(xs.shape), rn["gx"], bn["gx"])
    close("chain gw", w.grad, rn["gw"], bn["gw"])
    close("chain gb", b.grad, rn["gb"], bn["gb"])


def test_most_cells_take_part_in_the_chain_s_comparison():
    """Cells with a sample near an image edge are left out of the comparison with the oracle: they are few."""
    inp = wl.make_inputs("tiny", with_grad=True)
    br = oracle.oracle_forward(inp.F, inp.K, inp.R, inp.t, inp.rng6, 12, 12, inp.Z)
    assert (~br["near_edge"].any(axis=-1)).mean() >= 0.95
    assert (br["out"] != 0).any(axis=1).mean() >= 0.5
