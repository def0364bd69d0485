"""np_block_map's binding on the CPU: what it refuses before it looks at a device."""
import pytest
import torch


@pytest.mark.parametrize("positions", [False, True])
def test_a_mapping_without_room_is_not_taken_for_none(positions):
    """None asks for the tables only, whatever the new lengths; a mapping of no tokens has room for none of
    them and is refused, as a slot_mapping with num_tokens 0 is by the library."""
    import paged_kv_decode_np_gb300 as npg
    i32 = dict(dtype=torch.int32)
    tables, lens, free = torch.full((2, 3), -1, **i32), torch.zeros(2, **i32), torch.arange(6, **i32)
    with pytest.raises(ValueError, match="room for no tokens"):
        npg.np_block_map(tables, lens, torch.ones(2, **i32), free, torch.tensor([6], **i32), torch.zeros(3, **i32),
                         torch.zeros(0, dtype=torch.int64), torch.zeros(0, **i32) if positions else None, 2)
