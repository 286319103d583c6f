"""Block means of steps so long that a block of threads has 32 tokens: several leaders each, blocks that
straddle their borders, a last one that is partly filled."""
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from test_gpu_blocks import check_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [dsa.CACHE_BF16, dsa.CACHE_FP8_SCALED])
@pytest.mark.parametrize("page", [3, 33, 64])
def test_long_steps(gpu, page, kind):
    tokens = 32 * 8 * torch.cuda.get_device_properties(gpu).multi_processor_count + 1
    # prompts that end inside blocks, tokens of one position each between them, padding behind
    lens = [tokens // 3, 1, 2, 1, tokens // 3 + 5, 77, tokens // 3 - 20]
    new = [lens[0], 1, 1, 1, lens[4] - 70, 77, lens[6]]
    check_pool(gpu, lens, new, page, kind, pad=tokens - sum(new) + 45, poison=True)
