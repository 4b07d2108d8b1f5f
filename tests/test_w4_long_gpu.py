"""Products with 4-bit weights whose CTAs take many steps: every ring of the
kernel wraps several times, and with warm caches a stage is filled again as
soon as it is handed back."""

import numpy as np
import pytest
import torch

import token_reference as ref
from complexity_matmul_tcgen05_gb300 import fgemm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [5, 16, 30, 64, 128, 200])
def test_many_steps_and_repeated_calls(m, group, dtype):
    n, k = 10240, 4096  # more tiles than halves of the SMs: K is not cut
    g = torch.Generator("cuda").manual_seed(m + group)
    A = torch.randn(m, k, generator=g, device="cuda").to(dtype)
    W = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = ((1 + 0.3 * torch.rand(n, k // group, generator=g, device="cuda")) / 300).to(dtype)
    C = [fgemm.matmul_w4(A, W, s, group=group) for _ in range(12)]
    assert fgemm.default_handle().get_error() == fgemm.OK
    for other in C[1:]:
        assert torch.equal(C[0], other)
    want, bound = ref.w4(A.double().cpu().numpy(), W.cpu().numpy(), s.double().cpu().numpy(), None, group, 1.0, None,
                         "none", dtype)
    assert (np.abs(C[0].double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [16, 32, 48, 128])
def test_many_steps_of_slices(m, group):
    n, k = 8192, 16384  # two slices of 64 steps
    g = torch.Generator("cuda").manual_seed(m + group)
    A = torch.randn(m, k, generator=g, device="cuda").half()
    W = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = ((1 + 0.3 * torch.rand(n, k // group, generator=g, device="cuda")) / 600).half()
    C = [fgemm.matmul_w4(A, W, s, group=group) for _ in range(12)]
    for other in C[1:]:
        assert torch.equal(C[0], other)
    # the bound of the reference for 64 of the columns
    cols = torch.arange(0, n, n // 64, device="cuda")
    want, bound = ref.w4(A.double().cpu().numpy(), W[cols].cpu().numpy(), s[cols].double().cpu().numpy(), None, group, 1.0,
                         None, "none", torch.float16)
    assert (np.abs(C[0][:, cols].double().cpu().numpy() - want) <= bound).all()
