"""CPU tests of what the binding of the cache and window operators refuses, and
how it names it."""
import ctypes

import pytest
import torch

import token_level_top_hs2_b200 as hs2
from token_level_top_hs2_b200 import build as hs2_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    hs2_build.build()
    return hs2.load()


def test_a_misaligned_tensor_is_named():
    """lengths[1:] of a batch's lengths: the library would say only that some
    argument is invalid."""
    lengths = torch.zeros(9, dtype=torch.int32)
    assert hs2._dense(lengths[:8], "lengths", (torch.int32,), (8,), -1) == lengths.data_ptr()
    assert hs2._dense(lengths[4:8], "lengths", (torch.int32,), (4,), -1) == lengths.data_ptr() + 16
    with pytest.raises(ValueError, match="lengths: must start on a 16-byte boundary"):
        hs2._dense(lengths[1:], "lengths", (torch.int32,), (8,), -1)
    with pytest.raises(ValueError, match="start: must start on a 16-byte boundary"):
        hs2._dense_or_none(lengths[2:], "start", (torch.int32,), (7,), -1)
