"""Optional tensors without elements: they have no address, which to the library means that they were not
given.  The binding refuses them."""
import pytest
import torch

from tests.test_cache_append import append, rotate
from tests.test_cache_binding import evict, i32


@pytest.mark.parametrize("shape", [(0, 32), (9, 0), (0, 0)])
def test_a_table_of_no_angles_is_not_no_rotation(shape):
    """(Latents would be stored as they came.)"""
    for call in (append, rotate):
        with pytest.raises(ValueError, match="rope"):
            call(rope=torch.zeros(shape))
    with pytest.raises(ValueError, match="rope"):
        append(rope=torch.zeros(shape), rope_offset=0, rope_positions=i32(3))
