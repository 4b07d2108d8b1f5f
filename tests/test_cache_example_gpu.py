"""The operators around a key-value cache as they are used together, and the example."""

import importlib.util
import os

import pytest
import torch

import cache_reference as ref
from complexity_matmul_tcgen05_gb300 import fgemm
from test_cache_ops_gpu import check_paged, check_prompt, gen, ints, rand, within

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "cached_decode.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("cached_decode_example", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dim,page,dtype", [(64, 16, torch.bfloat16), (128, 24, torch.float16), (72, 7, torch.bfloat16)])
def test_prompt_and_steps_share_a_cache(dim, page, dtype):
    """Prompts into the cache; their last queries over the cache give what the prompt
    pass gives; then a few steps, each against its formula."""
    g = gen(40 + dim)
    lengths, heads, kv = [37, 130, 1, 300], 6, 2
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    steps, most = 3, max(lengths) + 3
    width = -(-most // page)
    table = torch.randperm(len(lengths) * width, generator=g, device="cuda").view(-1, width).to(torch.int32)
    k_cache, v_cache = (torch.full((len(lengths) * width, page, kv, dim), float("nan"), dtype=dtype, device="cuda")
                        for _ in range(2))
    freq = (1e4 ** (-2 * torch.arange(dim // 2, device="cuda").double() / dim)).float()

    def slots(seq, at):
        return (table[seq, at // page] * page + at % page).to(torch.int32)

    seq = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), torch.tensor(lengths, device="cuda"))
    at = torch.cat([torch.arange(n, device="cuda") for n in lengths])
    where = slots(seq, at)
    wide = rand(g, starts[-1], (heads + 2 * kv) * dim).to(dtype)
    q, k, v = (x.unflatten(1, (-1, dim)) for x in wide.split((heads * dim, kv * dim, kv * dim), 1))
    turned = fgemm.rotary_cache(q, k, v, at.to(torch.int32), where, freq, k_cache, v_cache)
    keys = k_cache.flatten(0, 1)[where.long()]
    assert torch.equal(v_cache.flatten(0, 1)[where.long()], v)
    out, lse = fgemm.attention(turned, keys, v, ints(starts))
    check_prompt(turned, keys, v, starts, starts, True, 0, out, lse, what="together, prompt")
    last = torch.tensor(starts[1:], device="cuda") - 1
    of_seq = lambda x: [x[a:b] for a, b in zip(starts, starts[1:])]  # noqa: E731
    all_k, all_v = of_seq(keys), of_seq(v)
    n = ints(lengths)
    out, lse = fgemm.attention_paged(turned[last], k_cache, v_cache, table, n)
    check_paged(turned[last], all_k, all_v, 0, None, out, lse, "together, last of the prompt")
    for _ in range(steps):
        n += 1
        where = slots(torch.arange(len(lengths), device="cuda"), n - 1)
        q, k, v = (rand(g, len(lengths), h, dim).to(dtype) for h in (heads, kv, kv))
        turned = fgemm.rotary_cache(q, k, v, n - 1, where, freq, k_cache, v_cache)
        new = k_cache.flatten(0, 1)[where.long()]
        all_k = [torch.cat((a, b[None])) for a, b in zip(all_k, new)]
        all_v = [torch.cat((a, b[None])) for a, b in zip(all_v, v)]
        out, lse = fgemm.attention_paged(turned, k_cache, v_cache, table, n)
        check_paged(turned, all_k, all_v, 0, None, out, lse, "together, a step")


def test_probability_of_a_sampled_token_is_its_logprob():
    g = gen(50)
    logits = (3 * rand(g, 40, 5003)).bfloat16()
    logits[3] = -float("inf")
    token, prob = fgemm.sample(logits, torch.rand(40, generator=g, device="cuda"))
    lp = fgemm.logprobs(logits, token)[0]
    _, _, _, _, bound, _, _ = ref.logprobs(ref.f64(logits), token.cpu().long(), 0)
    assert token[3].item() == -1 and lp[3].item() == -float("inf") and prob[3].item() == 0
    rest = torch.arange(40) != 3
    # prob is rounded to fp32 (2^-24 of itself), so is the logarithm
    want = prob.double().log().cpu()
    within("log of the probability", lp[rest.cuda()], want[rest], bound[rest] + 2.0 ** -24 + want[rest].abs() * 2.0 ** -24)


@pytest.mark.parametrize("kv_heads", [1, 2, 8])
def test_eager_and_replayed_steps_give_the_same_tokens(ex, kv_heads):
    model = ex.Model(kv_heads=kv_heads)
    g = torch.Generator("cuda").manual_seed(2)
    prompts = [torch.randint(0, 8000, (n,), generator=g, device="cuda", dtype=torch.int32) for n in (5, 150, 1)]
    uniform = torch.rand(8, 3, generator=g, device="cuda")
    got = []
    for graph in (False, True):
        cache = ex.Cache(2, 3, 158, kv_heads, model.dim)
        got.append(ex.generate(model, cache, prompts, uniform, graph, temperature=0.9, top_k=40))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    tokens, scores = got[0]
    assert int(tokens.min()) >= 0 and int(tokens.max()) < 8000
    assert bool((scores <= 0).all()) and bool(torch.isfinite(scores).all())
    whole = [torch.cat((x, tokens[:, i])) for i, x in enumerate(prompts)]
    again = ex.score(model, ex.Cache(2, 3, 158, kv_heads, model.dim), whole)
    assert [len(x) for x in again] == [len(x) - 1 for x in whole]
    assert all(bool(torch.isfinite(x).all()) for x in again)
    assert fgemm.default_handle().get_error() == fgemm.OK
