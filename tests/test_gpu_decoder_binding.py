"""GPU: what the decoder operators' binding keeps and refuses."""
import copy

import pytest
import torch

from camera_bev_view_amd import ops
from gpu_helpers import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def draw(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


NAMES = ("k", "v", "k_scale", "v_scale")


def held_cache():
    """A cache of tensors that the test holds too, with 70 tokens in it; and the call's arguments."""
    made = ops.token_cache(3, 2, 32, codes=torch.int8)
    tensors = {n: getattr(made, n).clone() for n in NAMES}
    cache = ops.TokenCache(*tensors.values(), 32)
    rows, table, start = draw(1, 1, 70, 2, 32), i32([[2, 0, 1]]), i32([0])
    ops.cache_write(cache, rows, rows, table, start)
    return cache, tensors, rows, table, start


@pytest.mark.parametrize("name", NAMES)
def test_a_cache_whose_tensors_have_moved_is_refused(name):
    """Tensors resized or given other memory behind the cache's back: no call goes to the addresses that it was made with."""
    def larger(t):
        t.resize_((4 * t.shape[0], *t.shape[1:]))

    def smaller(t):
        t.resize_((1, *t.shape[1:]))

    def other(t):
        t.set_(t.clone())

    def dropped(t):
        t.untyped_storage().resize_(0)

    for change in (larger, smaller, other, dropped):
        say(f"[case] {name} {change.__name__}")
        cache, tensors, rows, table, start = held_cache()
        kept = {n: getattr(cache, n).clone() for n in NAMES if n != name}
        change(tensors[name])
        for call in (lambda: ops.cache_write(cache, rows, rows, table, start),
                     lambda: ops.cache_read(cache, table, start, 70),
                     lambda: ops.cache_attention(rows[:, :3].contiguous(), cache, table, start)):
            with pytest.raises(ValueError, match="resized or moved"):
                call()
        for n, was in kept.items():
            assert torch.equal(getattr(cache, n), was), n


def test_tensors_written_in_place_are_the_caches():
    cache, tensors, rows, table, start = held_cache()
    for n in NAMES:
        assert getattr(cache, n).data_ptr() == tensors[n].data_ptr() and getattr(cache, n).shape == tensors[n].shape
    assert (cache.D, cache.Hk, cache.pages, cache.device) == (32, 2, 3, rows.device)
    cache.k_scale.mul_(2.0)
    before = ops.cache_read(cache, table, start, 70, dtype=F32)[0]
    tensors["k_scale"].mul_(0.5)
    assert torch.equal(ops.cache_read(cache, table, start, 70, dtype=F32)[0], before / 2)


def test_copies_have_memory_of_their_own():
    cache, tensors, rows, table, start = held_cache()
    deep, shallow = copy.deepcopy(cache), copy.copy(cache)
    was = [x.clone() for x in ops.cache_read(cache, table, start, 70, dtype=F32)]
    ops.cache_write(deep, rows * 3, rows * 5, table, start)
    for got, want in zip(ops.cache_read(cache, table, start, 70, dtype=F32), was):
        assert torch.equal(got, want)
    one = ops.token_cache(3, 2, 32, codes=torch.int8)
    ops.cache_write(one, rows * 3, rows * 5, table, start)
    for got, want in zip(ops.cache_read(deep, table, start, 70), ops.cache_read(one, table, start, 70)):
        assert torch.equal(got, want)
    ops.cache_write(shallow, rows * 3, rows * 5, table, start)          # the same tensors
    for got, want in zip(ops.cache_read(cache, table, start, 70), ops.cache_read(one, table, start, 70)):
        assert torch.equal(got, want)
