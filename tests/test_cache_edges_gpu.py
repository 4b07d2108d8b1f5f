"""The operators around a key-value cache at the ends of their arguments and types:
windows, scores, values and angles that the ordinary tests do not reach."""
import pytest
import torch

from complexity_matmul_tcgen05_gb300 import fgemm
from test_cache_ops_gpu import check_prompt, gen, ints, prompt_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (64, 16)])  # two tiles of a head, two heads
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 100])
def test_prompt_window_without_limit(window, heads, kv_heads):
    """A window that leaves nothing out, also where queries stand in front of the first key."""
    lengths, k_lengths = [5, 130, 100, 1, 40, 300, 129], [300, 77, 50, 1000, 0, 170, 2]
    q, k, v, starts, k_starts = prompt_inputs(gen(60), lengths, k_lengths, heads, kv_heads, 64, torch.bfloat16)
    plain, plain_lse = fgemm.attention(q, k, v, ints(starts), k_starts=ints(k_starts))
    out, lse = fgemm.attention(q, k, v, ints(starts), k_starts=ints(k_starts), window=window)
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)
    group = heads // kv_heads
    for h in (0, heads - 1):
        check_prompt(q[:, h:h + 1], k[:, h // group:h // group + 1], v[:, h // group:h // group + 1], starts, k_starts, True,
                     window, out[:, h:h + 1], lse[:, h:h + 1], what="prompt, window without limit")
