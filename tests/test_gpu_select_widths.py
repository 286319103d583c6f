"""The choice of blocks: calls that it refuses."""
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [16385, (1 << 31) - 1])
def test_no_room_is_made_for_a_refused_choice(gpu, K):
    scores, table = torch.zeros((64, 4), device=gpu), torch.zeros((64, 4), dtype=torch.int32, device=gpu)
    lens = torch.zeros(64, dtype=torch.int32, device=gpu)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(dsa.DsaError):
        dsa.dsa_block_select(scores, table, lens, K, page_size=16)
    assert torch.cuda.max_memory_allocated() == before
