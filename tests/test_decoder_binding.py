"""CPU: what the binding of the decoder operators does without a device."""
import pytest
import torch

from camera_bev_view_amd import ops


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "D", "Hk", "pages", "device", "desc", "other"])
def test_a_cache_cannot_be_given_other_tensors(name):
    """A cache's descriptor holds addresses: tensors put in the place of its own would leave them behind."""
    cache = object.__new__(ops.TokenCache)
    with pytest.raises(AttributeError):
        setattr(cache, name, None)


def test_ancestors_of_no_trees_and_no_tokens():
    """[B, T] parents give [B, T, words], for a batch of none as for any other."""
    for shape, want in (((0, 5), (0, 5, 1)), ((0, 65), (0, 65, 2)), ((3, 0), (3, 0, 1)), ((0,), (1, 0, 1)), ((0, 0), (0, 0, 1))):
        none = torch.zeros(shape, dtype=torch.int64)
        assert ops.tree_ancestors(none, device="cpu").shape == want, shape
        assert ops.tree_ancestors(none.numpy(), device="cpu").shape == want, shape
    assert ops.tree_ancestors([], device="cpu").shape == (1, 0, 1)
    assert ops.tree_ancestors([[], []], device="cpu").shape == (2, 0, 1)


def test_ancestors_from_lists_arrays_and_tensors():
    parents = [[-1, 0, 0, 2], [-1, -1, 1, 2]]
    want = [[0b0001, 0b0011, 0b0101, 0b1101], [0b0001, 0b0010, 0b0110, 0b1110]]
    for form in (parents, torch.tensor(parents), torch.tensor(parents).numpy(), [torch.tensor(p) for p in parents]):
        assert ops.tree_ancestors(form, device="cpu").squeeze(-1).tolist() == want
    assert ops.tree_ancestors(parents[1], device="cpu").squeeze(-1).tolist() == want[1:]
    chain = ops.tree_ancestors(range(-1, 129), device="cpu")
    assert chain.shape == (1, 130, 3) and chain[0, 129].tolist() == [-1, -1, 3] and chain[0, 63].tolist() == [-1, 0, 0]
    for bad in ([0], [-2], [-1, 1], [[-1, 0], [-1]], [-1, 5]):
        with pytest.raises(ValueError):
            ops.tree_ancestors(bad, device="cpu")
