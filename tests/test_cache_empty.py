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


def test_a_destination_of_no_pages_is_not_the_source():
    """(Records would be moved in place, or into the pages of kv_cache that dst_table names.)"""
    with pytest.raises(ValueError, match="dst_table"):
        evict(dst_table=i32(2, 0))
    with pytest.raises(ValueError, match="dst_cache"):
        evict(dst_table=i32(2, 3), dst_cache=torch.zeros((0, 16, 80), dtype=torch.uint8))
    a = evict(dst_table=i32(2, 3), dst_cache=torch.zeros((4, 16, 80), dtype=torch.uint8))
    assert a.dst_table and a.dst_cache and a.dst_num_blocks == 4 and a.dst_max_blocks == 3
