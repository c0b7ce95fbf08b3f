"""The binding's check that an output and an input of one call share no memory."""
import pytest
import torch


def apart(a, b):
    from w4a8_block_quantized_gb300 import binding
    binding._apart(a, b, "out", in_place=False)


def refused(a, b):
    with pytest.raises(ValueError, match="overlaps"):
        apart(a, b)


def test_types_of_two_widths():
    """An fp32 output beside bf16 rows in one array: apart by bytes, not by elements."""
    room = torch.zeros(4096, dtype=torch.uint8)
    for big, small in ((torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        wide, narrow = room.view(big), room.view(small)
        el, sl = wide.element_size(), narrow.element_size()
        # four tokens of 512 bytes: the first 256 to one, the rest to the other
        a = wide.as_strided((4, 2, 256 // el // 2), (512 // el, 256 // el // 2, 1))
        b = narrow.as_strided((4, 2, 256 // sl // 2), (512 // sl, 256 // sl // 2, 1), 256 // sl)
        apart(a, b), apart(b, a)
        refused(a, narrow.as_strided(b.shape, b.stride(), 128 // sl))
        # strides of as many elements, of different bytes
        c = narrow.as_strided((4, 2, 256 // el // 2), (512 // el, 256 // el // 2, 1), 256 // el)
        refused(a, c), refused(c, a)


def test_arrays_that_share_memory_without_sharing_a_storage():
    """Memory imported twice is two storages."""
    import numpy as np
    room = np.zeros((6, 64), dtype=np.float32)
    a, b = torch.from_numpy(room[:4]), torch.from_numpy(room[3:])
    assert a.untyped_storage().data_ptr() != b.untyped_storage().data_ptr()
    refused(a[:, None], b[:, None])
    apart(a[:3, None], b[:, None])


def test_rows_on_top_of_one_another():
    x = torch.zeros(64).as_strided((3, 1, 8), (0, 8, 1))
    refused(x, x)
