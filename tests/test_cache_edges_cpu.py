"""What the calls around a key-value cache do with arguments that their C forms cannot
hold, or may not take: no device needed."""
import pytest
import torch

from complexity_matmul_tcgen05_gb300 import fgemm

MANY = 2 ** 32 + 2  # 2 in 32 bits


def meta(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="meta")


@pytest.mark.parametrize("heads,dim", [(MANY, 8), (2, MANY)])
def test_heads_beyond_32_bits(heads, dim):
    t = meta(1, heads, dim)
    with pytest.raises(fgemm.FgemmError, match="32 bits"):
        fgemm._heads(t, "q", t.shape, t.dtype, -1)


@pytest.mark.parametrize("page,heads", [(MANY, 2), (2, MANY)])
def test_pages_beyond_32_bits(page, heads):
    t = meta(1, page, heads, 8)
    with pytest.raises(fgemm.FgemmError, match="32 bits"):
        fgemm._cache(t, t, None, 8, t.dtype, -1)


def test_windows_beyond_32_bits():
    for window, held in ((0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                         (-1, -1), (-2 ** 32, -1)):
        assert fgemm._softmax(0.5, window, 64) == (0.5, held)
    assert fgemm._softmax(None, 0, 64) == (0.125, 0) and fgemm._softmax(None, 0, 0) == (1.0, 0)
