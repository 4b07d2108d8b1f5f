"""The operators of a token step at the edges of what their documentation
admits: long K with few rows, ties behind a long top-k, activations and rows
far from 1, infinities, in-place outputs."""
import pytest
import torch

from complexity_matmul_tcgen05_gb300 import fgemm
from test_token_ops_gpu import DEV, TYPES, check_sample, gen, rand

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- sample


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "two", "steps"])
def test_sample_top_p_behind_a_long_top_k(kind, dtype):
    """Top-k's threshold is found key by key (more than 2048 logits down to
    it), and top-p's search follows at once."""
    g = gen(31)
    rows, vocab = 40, 20011
    if kind == "equal":
        x = torch.full((rows, vocab), 1.5, device=DEV)
    elif kind == "two":
        x = (rand(g, rows, vocab) > 0.5).float()
    else:
        x = torch.floor(4 * rand(g, rows, vocab)) / 4
    x = x.to(TYPES[dtype])
    u = torch.rand(rows, generator=g, device=DEV)
    for kw in (dict(top_k=5000, top_p=0.6), dict(top_k=15000, top_p=0.999, temperature=0.5),
               dict(top_k=3000, top_p=0.01), dict(top_k=9000, top_p=0.9, min_p=0.05)):
        token, prob = check_sample(x, u, **kw)
        for _ in range(20):
            again = fgemm.sample(x, u, **kw)
            assert torch.equal(again[0], token) and torch.equal(again[1], prob)
