"""GPU: attention calls at the edges of what its documentation allows."""
import numpy as np
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
