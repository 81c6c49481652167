"""CPU: the encoder operators' oracle against independent forms (torch's own modules in float64, complex rotation)
and its gradients against central differences."""
import numpy as np
import pytest
import torch

import oracle.encoder as enc


def numeric(f, x, g, h=1e-6):
    """Central differences of <g, f(x)>."""
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out[i] = (g * (f(a) - f(b))).sum() / (2 * h)
    return out


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu"])
def test_group_norm_matches_torch(kind):
    r = np.random.default_rng(3)
    x, w, b, g = r.normal(size=(2, 7, 12)), r.normal(size=12), r.normal(size=12), r.normal(size=(2, 7, 12))
    tx = torch.tensor(x.transpose(0, 2, 1).copy(), requires_grad=True)
    tw, tb = torch.tensor(w, requires_grad=True), torch.tensor(b, requires_grad=True)
    z = torch.nn.functional.group_norm(tx, 4, tw, tb, 1e-5)
    fn = dict(none=lambda v: v, relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu)[kind]
    y = fn(z)
    y.backward(torch.tensor(g.transpose(0, 2, 1).copy()))
    ref = enc.group_norm(x, 4, w, b, 1e-5, kind, g)
    np.testing.assert_allclose(ref["y"], y.detach().numpy().transpose(0, 2, 1), atol=1e-12)
    np.testing.assert_allclose(ref["gx"], tx.grad.numpy().transpose(0, 2, 1), atol=1e-11)
    np.testing.assert_allclose(ref["gw"], tw.grad.numpy(), atol=1e-11)
    np.testing.assert_allclose(ref["gb"], tb.grad.numpy(), atol=1e-11)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_complex_turn_and_undone_by_its_inverse(interleaved):
    r = np.random.default_rng(4)
    x, pos, fr = r.normal(size=(2, 5, 3, 10)), r.normal(size=(2, 5, 3)) * 1e4, r.normal(size=(3, 4))
    y = enc.rotary(x, pos, fr, interleaved)
    a = x[..., :8].reshape(2, 5, 3, 4, 2) if interleaved else np.stack((x[..., :4], x[..., 4:8]), -1)
    z = (a[..., 0] + 1j * a[..., 1]) * np.exp(1j * (pos @ fr))[:, :, None]
    b = y[..., :8].reshape(2, 5, 3, 4, 2) if interleaved else np.stack((y[..., :4], y[..., 4:8]), -1)
    np.testing.assert_allclose(b[..., 0] + 1j * b[..., 1], z, atol=1e-12)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    np.testing.assert_allclose(enc.rotary(y, pos, fr, interleaved, inverse=True), x, atol=1e-12)


def test_attention_matches_torch():
    r = np.random.default_rng(5)
    q, k, v = r.normal(size=(2, 6, 4, 8)), r.normal(size=(2, 9, 2, 8)), r.normal(size=(2, 9, 2, 8))
    mask = enc.visible(2, 6, 9, causal=True, prefix=[0, 8])
    t = lambda x: torch.tensor(x).permute(0, 2, 1, 3)
    o = torch.nn.functional.scaled_dot_product_attention(
        t(q), t(k).repeat_interleave(2, 1), t(v).repeat_interleave(2, 1), attn_mask=torch.tensor(mask)[:, None])
    ref = enc.attention(q, k, v, causal=True, prefix=[0, 8])
    np.testing.assert_allclose(ref["out"], o.permute(0, 2, 1, 3).numpy(), atol=1e-12)


def test_attention_gradients_match_differences():
    r = np.random.default_rng(6)
    B, Tq, Tk, Hq, Hk, D = 1, 4, 5, 2, 1, 3
    q, k, v = r.normal(size=(B, Tq, Hq, D)) * 2, r.normal(size=(B, Tk, Hk, D)) * 2, r.normal(size=(B, Tk, Hk, D))
    how = dict(cap=1.5, pos_q=r.normal(size=(B, Tq, 2)), pos_k=r.normal(size=(B, Tk, 2)),
               doc_q=np.array([[0, 0, 1, -1]]), doc_k=np.array([[0, 0, 0, 1, 2]]))
    slope, go = r.uniform(0, 1, (B, Tq, Hq)), r.normal(size=(B, Tq, Hq, D))
    ref = enc.attention(q, k, v, slope=slope, go=go, **how)
    assert (ref["out"][:, 3] == 0).all() and np.isneginf(ref["lse"][:, :, 3]).all()
    f = lambda **n: enc.attention(n.get("q", q), n.get("k", k), n.get("v", v), slope=n.get("slope", slope), **how)["out"]
    for name, x, g in (("q", q, "gq"), ("k", k, "gk"), ("v", v, "gv"), ("slope", slope, "gslope")):
        np.testing.assert_allclose(ref[g], numeric(lambda a: f(**{name: a}), x, go), atol=2e-8)


def test_what_a_masked_key_holds_reaches_nothing():
    r = np.random.default_rng(7)
    q, k, v = r.normal(size=(1, 3, 1, 4)), r.normal(size=(1, 4, 1, 4)), r.normal(size=(1, 4, 1, 4))
    docs = dict(doc_q=np.zeros((1, 3), int), doc_k=np.array([[0, 0, 0, -1]]))
    a = enc.attention(q, k, v, go=np.ones_like(q), **docs)
    k[0, 3], v[0, 3] = np.nan, np.inf
    b = enc.attention(q, k, v, go=np.ones_like(q), **docs)
    for name in ("out", "gq", "gk", "gv"):
        np.testing.assert_array_equal(a[name], b[name])
