"""What the binding of the shared, cross and page calls refuses before it looks for a device."""
import pytest
import torch

import grouped_query_attention_decode_b200 as gqa


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(shape)


CALLS = {
    "decode_shared": (f32(2, 8, 64), f32(1, 4, 2, 64), f32(1, 4, 2, 64), i32(1), i32(2), f32(2, 4, 2, 64), f32(2, 4, 2, 64), i32(2), 0.1),
    "decode_shared_paged": (f32(2, 8, 64), f32(4, 8, 2, 64), f32(4, 8, 2, 64), i32(2, 3), i32(2), i32(2), i32(1), 0.1),
    "cross_attend": (f32(3, 8, 64), f32(2, 4, 2, 64), f32(2, 4, 2, 64), i32(2), i32(3), 0.1),
    "pages_fork": (i32(2), i32(2, 3), i32(2), i32(2, 3), i32(2), i32(4)),
    "pages_free": (i32(1), i32(2, 3), i32(2), i32(4)),
    "pages_reserve": (i32(2, 3), i32(2), i32(4), 1, 8),
    "pages_compact": (i32(2, 3), i32(4)),
    "pages_copy": (f32(4, 8, 2, 64), f32(4, 8, 2, 64), i32(1, 2)),
}


@pytest.mark.parametrize("name", CALLS)
def test_status_is_one_int32_word(name):
    # a kernel ors a 32-bit word into it: one byte, or nothing, must not be handed over
    for status in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64), i32(0)):
        with pytest.raises(ValueError, match="status"):
            getattr(gqa, name)(*CALLS[name], status=status)
    with pytest.raises(ValueError, match="CUDA"):  # the other arguments are in order
        getattr(gqa, name)(*CALLS[name], status=i32(1))
