"""CPU: which outputs the encoder operators' binding takes for memory that something else of the call uses."""
import itertools
import random

import pytest
import torch

from camera_bev_view_amd import encoder


def addresses(t):
    at = {0}
    for n, s in zip(t.shape, t.stride()):
        at = {x + i * s for x in at for i in range(n)}
    base = t.data_ptr()
    return {base + x * t.element_size() + i for x in at for i in range(t.element_size())} if t.numel() else set()


def test_slices_of_packed_tensors_lie_apart():
    for shape, cut in (((2, 5, 3, 4, 8), lambda x, i: x[:, :, i]), ((2, 3, 4, 5, 8), lambda x, i: x[:, i].transpose(1, 2)),
                       ((2, 5, 4, 3, 8), lambda x, i: x[:, :, :, i]), ((2, 5, 4, 24), lambda x, i: x[..., 8 * i:8 * i + 8])):
        for dtype in (torch.float32, torch.bfloat16):
            x = torch.zeros(shape, dtype=dtype)
            for i, j in itertools.product(range(3), repeat=2):
                assert encoder._overlap(cut(x, i), cut(x, j)) == (i == j), (shape, i, j)
    grouped = torch.zeros((2, 5, 6, 8))            # four query heads, a key head, a value head
    q, k = grouped[:, :, :4], grouped[:, :, 4:5]
    assert not encoder._overlap(q, k) and not encoder._overlap(k, q)
    assert encoder._overlap(q, grouped[:, :, 3:5])


def test_random_walks_against_their_addresses():
    r = random.Random(5)
    room = torch.zeros(4000)
    apart = 0
    for _ in range(3000):
        pair = []
        for _ in range(2):
            dims = [r.choice([1, 2, 3]) for _ in range(3)] + [r.choice([1, 2, 4])]
            strides = [r.choice([0, 1, 2, 4, 8, 12, 16, 24, 48, 64, 96, 200]) for _ in range(3)] + [1]
            pair.append(room.as_strided(dims, strides, r.randrange(0, 300)))
        x, y = pair
        shared = bool(addresses(x) & addresses(y))
        if shared:
            assert encoder._overlap(x, y), (x.shape, x.stride(), x.storage_offset(), y.shape, y.stride(), y.storage_offset())
        apart += not encoder._overlap(x, y)
        count = 1
        for n, s in zip(x.shape, x.stride()):
            count *= 1 if s == 0 else n
        if encoder._steps_over(encoder._walk(x)):
            assert len(addresses(x)) == count * 4
    assert apart > 500
    assert not encoder._overlap(room[:0], room)


def test_what_is_refused():
    room = torch.zeros(2 * 31 * 4 * 32 + 8)
    first, later = (room[at:at + 2 * 31 * 4 * 32].view(2, 31, 4, 32) for at in (0, 8))
    with pytest.raises(ValueError, match="overlap"):
        encoder._check_apart("out", later, None, first)
    encoder._check_apart("out", later, None, torch.zeros(5))
    window = room.as_strided((5, 8), (4, 1))
    assert not encoder._steps_over(encoder._walk(window))
    assert encoder._steps_over(encoder._walk(first.transpose(1, 2)))
