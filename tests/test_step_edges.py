"""Edges of the step operators' host side: what is refused before anything is enqueued."""
import ctypes

import pytest
import torch

from paged_kv_cache_47_gb300 import binding as b
from paged_kv_cache_47_gb300 import build

REF = ctypes.byref


@pytest.fixture(scope="module")
def L():
    build.build()
    return b._ops_lib()


def test_block_copy_q4_refuses_a_cache_off_the_gpu(L):
    c = b.Q4Cache.empty(4, 2, 16, 128, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        b.block_copy_q4([[0, 1]], c)
