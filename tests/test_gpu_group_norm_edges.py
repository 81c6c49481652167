"""GPU: group norm calls at the edges of what its documentation allows."""
import pytest
import torch

from camera_bev_view_amd import ops

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_statistics_of_images_without_pixels(dtype):
    """Every element of the statistics is written: memory of another tensor does not show through."""
    print(f"[case] group norm without pixels {dtype}", flush=True)
    x = torch.empty((300, 0, 8), dtype=dtype, device="cuda")
    for _ in range(3):
        held = torch.full((300, 2, 2), float("nan"), device="cuda")       # the allocator hands this memory out next
        del held
        y, stats = ops.group_norm_forward(x, 2, eps=0.25)
        assert y.shape == x.shape and (stats[..., 0] == 0).all() and (stats[..., 1] == 2).all()


# groups of more pieces than a small workgroup has threads: (shape, groups).  Whole slabs, chunks of four pieces a thread
# without and with the launch that joins them, chunks of six, one channel a piece, two slabs of a group each, the widest
# group; last chunks are short
WIDE = [((5, 2, 2056), 1), ((1, 101, 2056), 1), ((1, 701, 2056), 1), ((3, 701, 2056), 1), ((2, 303, 771), 1),
        ((5, 611, 771), 1), ((2, 77, 4112), 2)]
WIDE = [(*c, t) for c in WIDE for t in (F32, BF16)] + [((1, 50, 8192), 1, BF16)]


@pytest.mark.parametrize("shape,groups,dtype", WIDE)
def test_wide_groups(shape, groups, dtype, monkeypatch):
    import encoder_bounds
    from test_gpu_group_norm import check, draw
    # a group's channels are added one after the other in the backward
    monkeypatch.setattr(encoder_bounds, "CHAIN", shape[-1] // groups + 256)
    print(f"[case] group norm of wide groups {shape} {dtype}", flush=True)
    x, gy, w, b = draw(shape, dtype, 17)
    check(x.cuda(), gy.cuda(), w.cuda(), b.cuda(), groups, "silu", f"{shape}/{groups}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_map_one_pixel_wide(dtype):
    from test_gpu_group_norm import check, draw
    print(f"[case] group norm of a map one pixel wide {dtype}", flush=True)
    x, gy, w, b = draw((2, 1, 700, 1, 1032), dtype, 18)
    check(x.cuda(), gy.cuda(), w.cuda(), b.cuda(), 3, "silu", "one pixel wide")
