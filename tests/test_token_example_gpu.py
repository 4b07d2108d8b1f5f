"""The example of a token step, at small sizes."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "token_step.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("token_step_example", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("rows", [1, 5, 20])
def test_eager_and_replayed_steps_give_the_same_tokens(ex, rows):
    model = ex.Model(width=256, hidden=352, depth=2, vocab=1000, group=64)
    token = torch.arange(rows, dtype=torch.int32, device="cuda")
    uniform = torch.rand(6, rows, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    kept = dict(temperature=0.9, top_k=40, top_p=0.95)
    eager = ex.generate(model, token, uniform, graph=False, **kept)
    replayed = ex.generate(model, token, uniform, graph=True, **kept)
    assert torch.equal(eager, replayed)
    assert int(eager.min()) >= 0 and int(eager.max()) < 1000
    greedy, prob, logits = model.step(token, uniform[0], temperature=0.0)
    assert torch.equal(greedy.long(), logits.float().argmax(1))
    assert bool((prob == 1).all())


def test_quantised_weights_lie_within_half_a_step(ex):
    # codes -7..7 about the zero point; the scale's rounding to bf16 (2^-8 of
    # it, seven steps at most) comes on top of half a step
    W = torch.randn(33, 200, generator=torch.Generator("cuda").manual_seed(2), device="cuda").bfloat16()
    codes, scales = ex.quantise_w4(W, 64)
    q = torch.stack((codes & 15, codes >> 4), 2).view(33, -1).double() - 8
    s = scales.double().repeat_interleave(64, 1)[:, :200]
    assert float(((q * s - W.double()) / s).abs().max()) <= 0.5 + 7 * 2.0 ** -8


def test_gain_is_fitted_and_8_bit_blocks_multiply(ex):
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(256, 128, generator=g, device="cuda").bfloat16()
    gain = torch.ones(128, device="cuda").bfloat16()
    losses = ex.fit_gain(x, ex.fgemm.rms_norm(x, gain * 1.5)[0], gain)
    assert losses[-1] < 0.01 * losses[0]
    # every weight 1: a row's sum of the 8-bit values, each off by at most 2^-4
    # of itself (or 2^-10 of its block's scale), rounded once to bf16
    B = torch.full((128, 16), 0x38, dtype=torch.uint8, device="cuda")
    C = ex.norm_into_mx(x, gain, B, torch.full((4, 16), 127, dtype=torch.uint8, device="cuda"))
    y = x.double() / (x.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    bound = y.abs().sum(1) * 2.0 ** -4 + 128 * y.abs().amax(1) * 2.0 ** -10 + y.sum(1).abs() * 2.0 ** -8 + 1e-3
    assert bool(((C.double() - y.sum(1, keepdim=True)).abs() <= 2 * bound[:, None]).all())
