"""Edges of the step operators' calls: slots past the pool wherever they lie in a block, one-shot calls
on another stream than the current one."""
import pytest
import torch

from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("off", [0, 3, -1])
def test_block_means_flags_every_slot_past_the_pool(off, B):
    NB = 4
    k = torch.randn(NB, 2, B, 64, device="cuda").bfloat16()
    means = torch.full((NB, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([5, NB * B + off % B], device="cuda")
    b.block_means(slots, k, means)
    assert b.get_error() == b.DEVERR_SLOT and (means == 9).all()
