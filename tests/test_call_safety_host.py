"""What the torch conveniences refuse or arrange around a call, without a GPU: temp
storage that is not one block of memory, the stream a handle stands for, memory that
arrays share, and torch's count of writes to a tensor."""
from __future__ import annotations

import pytest
import torch

import sorting_lsd_radix_sort_amd as lrs
from sorting_lsd_radix_sort_amd import rows

# fake, well-aligned device addresses, far apart: these checks never dereference them
A, B, C, D = (i << 40 for i in range(1, 5))


# ------------------------------------------------------------------ temp storage


def scattered_temps(nbytes):
    """Tensors whose elements are as many bytes as asked for and more, but do not lie in one block."""
    return {"columns": torch.zeros(64, nbytes, dtype=torch.uint8)[:, :nbytes // 2],
            "every other": torch.zeros(4 * nbytes, dtype=torch.uint8)[::2],
            "expanded": torch.zeros(1, dtype=torch.uint8).expand(2 * nbytes),
            "turned": torch.zeros(64, nbytes, dtype=torch.uint8).t()}


@pytest.mark.parametrize("kind", ["columns", "every other", "expanded", "turned"])
def test_temp_that_is_not_one_block_is_refused(kind):
    """A call writes the bytes that follow the tensor's first element: of a column
    slice these are other columns, of an expanded element other memory."""
    need = 4096
    temp = scattered_temps(need)[kind]
    assert temp.numel() >= need and not temp.is_contiguous()
    with pytest.raises(ValueError, match="temp must be contiguous"):
        lrs._temp_tensor(need, temp.device, temp)
    like = torch.zeros(1)
    args = (1, A, 20000, 0, 8, B, C, D)
    with pytest.raises(ValueError, match="temp must be contiguous"):
        rows._temp("lrs_group_tokens", (1, 20000, 8), args, like, temp)
    # one block is taken as it is, by both
    whole = torch.zeros(1 << 20, dtype=torch.uint8)
    assert lrs._temp_tensor(need, whole.device, whole) is whole
    assert rows._temp("lrs_group_tokens", (1, 20000, 8), args, like, whole)[0] is whole
