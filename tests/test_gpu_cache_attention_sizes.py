"""GPU: attention over the token cache where values are as large, or as small, as the cache holds them."""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from test_gpu_cache_attention import check, draw, filled

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def of_size(cache, model, size, kind):
    """Every token's values become positive, their scales as if the largest of each token was `size`."""
    top = np.float32(size / (127.0 if kind == "int8" else 448.0))
    model.v_scale[~np.isnan(model.v_scale)] = top
    model.v[...] = np.abs(model.v.view(np.int8)).view(np.uint8) if kind == "int8" else model.v & 127
    cache.v.view(torch.uint8).copy_(torch.from_numpy(model.v))
    cache.v_scale.copy_(torch.from_numpy(model.v_scale))


# (starts, T, Hq, Hk): waves with pages of their own, four and eight; groups of waves, two and four; shared pages; with
# splits (joined by 32 lanes a row or by a workgroup a row) and without
SHAPES = [([1300], 1, 2, 1), ([6000], 2, 2, 1), ([130] * 50, 1, 8, 4), ([900, 64], 20, 4, 2), ([5000], 30, 1, 1),
          ([400] * 40, 17, 8, 8), ([700, 90], 100, 4, 2)]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_the_largest_values(shape, dtype, kind):
    """A mean of values up to 3e38 is no more than they are: no sum on the way to it may pass fp32's range."""
    start, T, Hq, Hk = shape
    D = 40 if Hk == 2 else 96 if T == 2 else 24
    say(f"[case] {len(start)} x {shape[1:]} {dtype} {kind}")
    cache, model, table = filled(T + Hq, [n + T for n in start], Hk, D, kind)
    of_size(cache, model, 3e38, kind)
    # scores that grow by less than 2^8 from a sequence's first pages to its last
    for b in range(len(start)):
        for w in range(table.shape[1]):
            model.k_scale[table[b, w]] *= np.float32(0.05 + 0.45 * w / table.shape[1])
    cache.k_scale.copy_(torch.from_numpy(model.k_scale))
    out = check(draw(T, len(start), T, Hq, D, dtype=dtype), cache, model, table, start, "chain")
    assert out.isfinite().all() and (out > 1e36).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_small_values(dtype, kind):
    """The range's other end, as far down as the header promises digits: 2^-80 for each page of the table."""
    for start, T in (([1300], 1), ([900, 64], 20), ([700, 90], 100)):
        cache, model, table = filled(T, [n + T for n in start], 2, 40, kind)
        of_size(cache, model, 2.0 ** -80 * table.shape[1], kind)
        out = check(draw(T, len(start), T, 4, 40, dtype=dtype), cache, model, table, start, "chain", label=f"T={T}")
        assert (out > 0).all()
