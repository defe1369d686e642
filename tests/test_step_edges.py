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


def test_select_workspace_refuses_what_the_call_refuses(L):
    ws = lambda S, M, hk=2, nb=8: L.pkv_select_workspace_bytes(REF(b.CacheDesc(nb, 16, hk, 64, b.PKV_BF16)), S, M)  # noqa: E731
    assert ws(3, 5) == 3 * 2 * 8 * 4
    assert ws(1, (1 << 27) - 1) == 2 * (1 << 27) * 4         # the longest row
    assert ws(1, 1 << 27) == 0 and ws(1, (1 << 31) - 1) == 0  # 2^31 tokens and more
    assert ws(1 << 25, 5) == 0                                # too many rows
    assert ws(1, 5, nb=1 << 30) == 0
