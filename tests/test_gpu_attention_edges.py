"""GPU: attention calls at the edges of what its documentation allows."""
import pytest
import torch

from camera_bev_view_amd import ops
from encoder_bounds import close
from encoder_fine_bounds import oracle
from test_gpu_attention import draw, runs

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(q, k, v, go, how, label, skip=()):
    print(f"[case] attention {label}: {tuple(q.shape)} {q.dtype}", flush=True)
    ref, bd = oracle(q, k, v, how, go)
    out, stats = ops.attention_forward(q, k, v, **how)
    grads = ops.attention_backward(go, q, k, v, out, stats, **how)
    for name, x in zip(("out", "gq", "gk", "gv", "gslope"), (out, *grads)):
        if x is not None and name not in skip:
            close(f"{label} {name}", x, ref[name], bd[name])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads,B", [(2, 1), (96, 4)])
def test_a_key_of_minus_infinity_takes_no_weight(heads, B, dtype):
    """A key whose score is minus infinity for every query of its document is as good as masked: the document's other keys
    get the gradients that they have without it."""
    T = 90
    ids = [runs([40, 30], T)] * B
    q, k, v, go, how = draw(B, T, T, heads, heads, 32, dtype, 84, dims=2, docs=(ids, ids))
    q[..., 5] = q[..., 5].abs() + 0.1
    ref_docs = how["doc_k"].clone()
    ref_docs[:, 50] = 99
    ref, bd = oracle(q, k, v, {**how, "doc_k": ref_docs}, go)
    print(f"[case] attention with a key of -inf, {heads} heads {dtype}", flush=True)
    k[:, 50, :, 5] = -float("inf")
    out, stats = ops.attention_forward(q, k, v, **how)
    _, gk, gv, _ = ops.attention_backward(go, q, k, v, out, stats, **how)
    for name, x in (("out", out), ("gk", gk), ("gv", gv)):
        close(f"-inf key {name}", x, ref[name], bd[name])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cap", [65.0, 1e4, 1e6, 1e9, 1e12])
def test_caps_far_above_the_scores(cap, dtype):
    check(*draw(1, 50, 90, 4, 2, 32, dtype, 81, cap=cap, dims=1, sharp=2.0), f"cap {cap}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("prefix", [-2 ** 31, -1, 2 ** 31 - 1])
def test_prefixes_beyond_the_keys(prefix, dtype):
    q, k, v, go, how = draw(1, 40, 70, 2, 1, 32, dtype, 82, causal=True, prefix=[prefix])
    check(q, k, v, go, how, f"prefix {prefix}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_query_row_for_all_tokens(dtype):
    """Queries broadcast over the tokens (stride 0), with scores far beyond what an exponential holds."""
    q, k, v, go, how = draw(1, 33, 45, 2, 2, 32, dtype, 83, sharp=1.0)
    row = k[:, 7:8] * 40
    check(row.expand(1, 33, 2, 32), k, v, go, how, "one row")
    one = k[:, 3:4].expand(1, 45, 2, 32)
    check(q, one, v[:, :1].expand(1, 45, 2, 32), go, how, "one key")
    check(row.as_strided((1, 1, 2, 32), (0, 0, 32, 1)), k, v, go[:, :1].contiguous(), how, "one token of stride 0")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_places_hold_anything_where_a_wave_takes_two_heads(dtype):
    T, B, H = 75, 4, 96
    ids = [runs([40, 9, 20], T)] * B
    q, k, v, go, how = draw(B, T, T, H, H, 32, dtype, 85, dims=2, docs=(ids, ids), causal=True)
    print(f"[case] attention, two heads a wave, padding {dtype}", flush=True)
    want = ops.attention_forward(q, k, v, **how)
    grads = ops.attention_backward(go, q, k, v, *want, **how)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for t in (k, v, q, go):
            t[:, 69:] = bad
        how["pos_k"][:, 69:] = bad
        how["pos_q"][:, 69:] = bad
        out, stats = ops.attention_forward(q, k, v, **how)
        assert torch.equal(out, want[0]) and torch.equal(stats, want[1]), bad
        for a, b in zip(ops.attention_backward(go, q, k, v, out, stats, **how), grads):
            assert torch.equal(a, b), bad
    # one value of a document: the others' rows and gradients stay
    q, k, v, go, how = draw(B, T, T, H, H, 32, dtype, 86, dims=2, docs=(ids, ids))
    want = ops.attention_forward(q, k, v, **how)
    grads = ops.attention_backward(go, q, k, v, *want, **how)
    other = torch.tensor([i < 40 or i >= 49 for i in range(T)], device="cuda")
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, v2, q2, go2 = (t.clone() for t in (k, v, q, go))
        v2[:, 41, :, 3] = k2[:, 42, :, 1] = q2[:, 43, :, 2] = go2[:, 44, :, 2] = bad
        out, stats = ops.attention_forward(q2, k2, v2, **how)
        assert torch.equal(out[:, other], want[0][:, other]), bad
        for a, b in zip(ops.attention_backward(go2, q2, k2, v2, out, stats, **how), grads):
            assert torch.equal(a[:, other], b[:, other]), bad


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_queries(dtype):
    print(f"[case] attention without queries {dtype}", flush=True)
    q, k, v, go, how = draw(2, 0, 50, 4, 2, 32, dtype, 87, dims=2, docs=([[]] * 2, [[0] * 50] * 2))
    out, stats = ops.attention_forward(q, k, v, **how)
    gq, gk, gv, gs = ops.attention_backward(go, q, k, v, out, stats, **how)
    assert out.shape == q.shape and gq.shape == q.shape and gs.shape == (2, 0, 4)
    assert gk.shape == k.shape and (gk == 0).all() and (gv == 0).all()
