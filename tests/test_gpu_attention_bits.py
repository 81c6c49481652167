"""GPU: bf16 attention loses nothing but the rounding of its results: outputs and gradients against the fp64 oracle with
bounds that leave no room for operands rounded to bf16 on the way."""
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


def forms():
    """Every form of the kernels: (label, drawing arguments).  Four and eight waves a row tile, 128 rows a workgroup, two
    heads a wave, split keys and split rows, grouped heads, masks, caps, each head width."""
    packed = [runs([40, 33, 20], 95)]
    yield "dense D=32", dict(shape=(1, 33, 65, 2, 2, 32))
    yield "grouped D=64", dict(shape=(2, 17, 130, 6, 2, 64), dims=2)
    yield "odd D=40", dict(shape=(1, 45, 77, 4, 2, 40), cap=3.0, dims=1)
    yield "D=128", dict(shape=(1, 40, 200, 2, 2, 128), causal=True)
    yield "eight waves", dict(shape=(4, 95, 95, 16, 16, 64), docs=(packed * 4, packed * 4), causal=True)
    yield "128 rows", dict(shape=(16, 40, 40, 128, 128, 16), causal=True, dims=2, cap=3.0)
    yield "two heads", dict(shape=(4, 75, 75, 96, 96, 32), dims=2)
    yield "split keys", dict(shape=(1, 2, 2100, 4, 2, 64), dims=2)
    yield "split rows", dict(shape=(1, 1500, 3, 4, 2, 33), dims=1)


FORMS = list(forms())


def make(kw, dtype, seed=71):
    kw = dict(kw)
    return draw(*kw.pop("shape"), dtype, seed, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("label,kw", FORMS, ids=[f[0] for f in FORMS])
def test_outputs(label, kw, dtype):
    q, k, v, _, how = make(kw, dtype)
    print(f"[case] attention outputs {label} {dtype}", flush=True)
    ref, bd = oracle(q, k, v, how)
    close(label + " out", ops.attention_forward(q, k, v, **how)[0], ref["out"], bd["out"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("label,kw", FORMS, ids=[f[0] for f in FORMS])
def test_key_and_value_gradients(label, kw, dtype):
    q, k, v, go, how = make(kw, dtype, 72)
    print(f"[case] attention gk, gv {label} {dtype}", flush=True)
    ref, bd = oracle(q, k, v, how, go)
    _, gk, gv, _ = ops.attention_backward(go, q, k, v, *ops.attention_forward(q, k, v, **how), **how)
    close(label + " gk", gk, ref["gk"], bd["gk"])
    close(label + " gv", gv, ref["gv"], bd["gv"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("label,kw", FORMS, ids=[f[0] for f in FORMS])
def test_query_and_slope_gradients(label, kw, dtype):
    q, k, v, go, how = make(kw, dtype, 73)
    print(f"[case] attention gq {label} {dtype}", flush=True)
    ref, bd = oracle(q, k, v, how, go)
    gq, _, _, gs = ops.attention_backward(go, q, k, v, *ops.attention_forward(q, k, v, **how), **how)
    close(label + " gq", gq, ref["gq"], bd["gq"])
    if gs is not None:
        close(label + " gslope", gs, ref["gslope"], bd["gslope"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("slope", [0.25, 0.5, 2.0])
def test_gradients_of_rows_that_look_at_one_key(slope, dtype):
    """Distances that leave a row one key's weight: its gradients are small differences of large terms, and an output
    rounded to bf16 in their place would be off by many times their size."""
    print(f"[case] attention of peaked rows, slope {slope} {dtype}", flush=True)
    q, k, v, go, how = draw(1, 400, 400, 2, 2, 64, dtype, 74, dims=2)
    how["pos_k"] = how["pos_q"] = how["pos_q"] * 5
    how["slope"] = torch.full_like(how["slope"], slope)
    ref, bd = oracle(q, k, v, how, go)
    gq, gk, gv, gs = ops.attention_backward(go, q, k, v, *ops.attention_forward(q, k, v, **how), **how)
    for name, x in (("gq", gq), ("gk", gk), ("gv", gv), ("gslope", gs)):
        close(f"slope {slope} {name}", x, ref[name], bd[name])
