"""CPU: what the binding of the decoder operators does without a device."""
import pytest

from camera_bev_view_amd import ops


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "D", "Hk", "pages", "device", "desc", "other"])
def test_a_cache_cannot_be_given_other_tensors(name):
    """A cache's descriptor holds addresses: tensors put in the place of its own would leave them behind."""
    cache = object.__new__(ops.TokenCache)
    with pytest.raises(AttributeError):
        setattr(cache, name, None)
