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


def test_gradients_are_not_lost_without_a_word():
    """Calls without a backward, on tensors that require gradients: the values are the same, and a gradient is an error."""
    x, r, w = draw(1, 6, 96), draw(2, 6, 96), draw(3, 96)
    want = ops.rms_norm_codes(x, w, residual=r)
    for which in range(3):
        args = [x.clone(), r.clone(), w.clone()]
        args[which].requires_grad_()
        codes, scales, h = ops.rms_norm_codes(args[0], args[2], residual=args[1])
        assert torch.equal(codes.view(torch.uint8), want[0].view(torch.uint8))
        assert torch.equal(scales, want[1]) and torch.equal(h, want[2])
        for out in (scales, h):
            with pytest.raises(RuntimeError, match="rms_norm_codes has no backward"):
                out.sum().backward()
        # the residual stream of a layer behind it too
        with pytest.raises(RuntimeError, match="rms_norm_codes has no backward"):
            ops.rms_norm(h, w).sum().backward()
        with torch.no_grad():
            assert not any(t.requires_grad for t in ops.rms_norm_codes(args[0], args[2], residual=args[1]))
    leaf = x.clone().requires_grad_()
    codes, scales, h = ops.rms_norm_codes(leaf, w)
    assert h is leaf and scales.requires_grad           # h is x itself: its graph is x's
    cache, _, rows, table, start = held_cache()
    q = draw(4, 1, 5, 4, 32)
    want = ops.cache_attention(q, cache, table, i32([65]))
    out = ops.cache_attention(q.requires_grad_(), cache, table, i32([65]))
    assert torch.equal(out, want)
    with pytest.raises(RuntimeError, match="cache_attention has no backward"):
        out.sum().backward()
    with torch.no_grad():
        assert not ops.cache_attention(q, cache, table, i32([65])).requires_grad
    given = torch.empty_like(want)
    out = ops.cache_attention(q, cache, table, i32([65]), out=given)
    assert torch.equal(given, want) and out.data_ptr() == given.data_ptr() and out.requires_grad
    assert ops.cache_attention(q.detach(), cache, table, i32([65]), out=given) is given
