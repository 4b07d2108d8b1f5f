"""The operators around a key-value cache at the ends of their arguments and types:
windows, scores, values and angles that the ordinary tests do not reach."""
import ctypes
import threading

import pytest
import torch

import cache_reference as ref
from complexity_matmul_tcgen05_gb300 import fgemm
from test_cache_ops_gpu import (DEV, TYPES, check_paged, check_prompt, gen, ints, paged_inputs, prompt_inputs, rand,
                                within)

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
        at = slice(h // group, h // group + 1)
        check_prompt(q[:, h:h + 1], k[:, at], v[:, at], starts, k_starts, True, window, out[:, h:h + 1],
                     lse[:, h:h + 1], what="prompt, window without limit")


def far_inputs(dtype, n, dim):
    """Keys of one head whose scores with every query are exact in fp32, far from 0 and,
    times a scale of 64, more than 2^13 apart: a query's output is the value of the
    largest one it sees.  Half of the keys have a score of 0; one query in four has the
    others below it."""
    g = gen(61)
    side = torch.arange(n, device=DEV)
    q, k = torch.zeros(n, 1, dim, device=DEV), torch.zeros(n, 1, dim, device=DEV)
    q[:, 0, 0] = torch.where(side % 4 == 3, -2047.0, 2047.0)  # products of 11 and 9 bits
    order = torch.randperm(n, generator=g, device=DEV)
    k[:, 0, 0] = (256.0 - order % 256) * (16.0 if dtype == torch.float16 else 2.0 ** 20)
    k[order >= 256, 0, 0] = 0.0
    v = rand(g, n, 1, dim).to(dtype)
    if dtype == torch.bfloat16:
        q[:, 0, 0] = q[:, 0, 0].sign() * 255.0
    return q.to(dtype), k.to(dtype), v


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_far_from_zero(dtype, dim, causal, window):
    """Scores of 10^9 and beyond, whose product with log2 e rounds by more than a 16-bit
    weight's exponent holds.  A weight of the largest score rounds by half a step of
    16 bits at most, the output by another, its reciprocal sum by 2^-23."""
    n, scale = 500, 64.0
    q, k, v = far_inputs(TYPES[dtype], n, dim)
    scores = (ref.f64(q)[:, 0] @ ref.f64(k)[:, 0].t()) * scale
    scores = torch.where(ref.seen_by(n, n, causal, window), scores, -torch.inf)
    most = scores.amax(1, keepdim=True)
    # (keys with a score of 0 share the weight where nothing is above them)
    first = torch.softmax(scores, 1)
    values = ref.f64(v)[:, 0]
    want = (first @ values)[:, None]
    half = torch.finfo(TYPES[dtype]).eps / 2
    bound = (first @ values.abs())[:, None] * (2 * half + (n / 16 + 16) * 4 * ref.U32) + ref.store(want, TYPES[dtype])
    want_lse = torch.logsumexp(scores, 1)[:, None]
    # log2 e and ln 2 as fp32 numbers, their two products with the score, the sums of weights
    bound_lse = most.abs() * 6 * ref.U32 + 2.0 ** -12
    out, lse = fgemm.attention(q, k, v, ints([0, n]), causal=causal, window=window, scale=scale)
    within("far scores, prompt", out, want, bound)
    within("far scores, prompt lse", lse, want_lse, bound_lse)
    if causal:
        # the same keys in pages, the last queries one at a time
        pages = -(-n // 16)
        k_cache, v_cache = (torch.zeros(pages, 16, 1, dim, dtype=q.dtype, device=DEV) for _ in range(2))
        k_cache.view(-1, 1, dim)[:n], v_cache.view(-1, 1, dim)[:n] = k, v
        rows = torch.arange(n - 200, n, device=DEV)
        table = torch.arange(pages, device=DEV, dtype=torch.int32).expand(len(rows), pages)
        out, lse = fgemm.attention_paged(q[rows], k_cache, v_cache, table.contiguous(), (rows + 1).to(torch.int32),
                                         window=window, scale=scale)
        within("far scores, paged", out, want[rows.cpu()], bound[rows.cpu()])
        within("far scores, paged lse", lse, want_lse[rows.cpu()], bound_lse[rows.cpu()])


def test_scores_far_from_zero_beside_a_value_that_is_not_finite():
    """Only the queries that see it have it."""
    n, scale, at = 500, 64.0, 301
    q, k, v = far_inputs(torch.float16, n, 64)
    v[at, 0, 5] = torch.inf
    out, lse = fgemm.attention(q, k, v, ints([0, n]), scale=scale)
    plain, plain_lse = fgemm.attention(q, k, torch.where(torch.isinf(v), 0.0, v), ints([0, n]), scale=scale)
    assert torch.equal(lse, plain_lse) and torch.equal(out[:at], plain[:at])
    assert not bool(torch.isfinite(out[at:, 0, 5]).any())
    rest = torch.arange(64, device=DEV) != 5
    assert bool(torch.isfinite(out[:, :, rest]).all())


def test_scores_beside_a_row_far_from_zero():
    """Rows whose scores are in the ten thousands, with two keys of the same score in two
    steps, beside one that becomes far in the second: both keys weigh the same.  A
    weight rounds to fp16 by up to 2^-11 of itself (in the first step it is no power of 2: it
    carries what the reference was rounded by), which moves a value's share of one half by
    up to 2^-12; the sum and the quotient round a few times in fp32."""
    n, dim = 300, 64
    for scale in (1.0, 0.9137, 1.0371):
        q, k = torch.zeros(64, 1, dim, device=DEV), torch.zeros(n, 1, dim, device=DEV)
        q[:, 0, 0] = 1.0 - torch.arange(64, device=DEV) / 128
        q[17, 0, 0], q[17, 0, 1] = 0.0, 2047.0
        k[3, 0, 0] = k[200, 0, 0] = 40000.0
        k[200, 0, 1] = 60000.0
        v = rand(gen(64), n, 1, dim).half()
        out, lse = fgemm.attention(q.half(), k.half(), v, ints([0, 64]), k_starts=ints([0, n]), causal=False,
                                   scale=scale)
        a, b = ref.f64(v[3, 0]), ref.f64(v[200, 0])
        want = ((a + b) / 2).expand(64, 1, dim).clone()
        want[17] = b
        bound = ref.store(want, torch.float16) + (a.abs() + b.abs()) * (2.0 ** -12 + 2.0 ** -20)
        within("beside a far row", out, want, bound)
        most = (q.half().double() @ k.half().double()[:, 0].t()).amax(2).cpu() * scale
        two = torch.full_like(most, 2.0).log()
        two[17] = 0.0
        within("beside a far row, lse", lse, most + two, most * 6 * ref.U32 + 2.0 ** -20)


@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (64, 16)])  # two tiles of a head, two heads
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_exact_scores_of_any_size(dtype, dim, heads, kv_heads):
    """Scores that fp32 holds exactly, each query's and key's of a size of its own from 1 to
    2^40, times a scale of a power of 2: what is left to differ is a weight's exponent, off by
    2^-23 of it (log2 e, the product; below -40 a weight does not count), its exponential,
    its rounding to 16 bits, the sums and the store."""
    t, half = TYPES[dtype], torch.finfo(TYPES[dtype]).eps / 2
    g = gen(70)
    lengths, k_lengths = [300, 130, 5, 700], [300, 260, 400, 600]
    q, k, v, starts, k_starts = prompt_inputs(g, lengths, k_lengths, heads, kv_heads, dim, t)

    def sizes(n, most):
        return 2.0 ** torch.randint(0, most, (n, 1, 1), generator=g, device=DEV).float()

    # three products of 4 and 4 bits for each score
    q, k = (torch.zeros_like(x).index_copy_(2, ints([0, 1, dim - 1]).long(), torch.randint(
        -15, 16, (*x.shape[:2], 3), generator=g, device=DEV).to(t)) for x in (q, k))
    q *= sizes(len(q), 11 if t == torch.float16 else 20).to(t)
    k *= sizes(len(k), 12 if t == torch.float16 else 13).to(t)
    few = [0, 1, heads - 1]
    for scale in (0.125, 2.0 ** -10, 16.0):
        for causal, window in ((True, 0), (False, 0), (True, 150)):
            out, lse = fgemm.attention(q, k, v, ints(starts), k_starts=ints(k_starts), causal=causal, window=window,
                                       scale=scale)
            for s in range(len(lengths)):
                a, b, c, d = starts[s], starts[s + 1], k_starts[s], k_starts[s + 1]
                seen = ref.seen_by(b - a, d - c, causal, window)
                any_seen = seen.any(1)
                for h in few:
                    x = ref.f64(q[a:b, h]) @ ref.f64(k[c:d, h * kv_heads // heads]).t() * scale
                    x = torch.where(seen, x, -torch.inf)
                    z = torch.logsumexp(x, 1)
                    p = torch.where(seen, torch.exp(x - torch.where(any_seen, z, 0.0)[:, None]), 0.0)
                    values = ref.f64(v[c:d, h * kv_heads // heads])
                    want = p @ values
                    off = 2 * half + 2.0 ** -23 * 40 + (8 + 4 * ((d - c) / 16 + 16)) * ref.U32
                    bound = (p @ values.abs()) * off + ref.store(want, t)
                    if t == torch.float16:  # (weights below 2^-14, lifted by 2^6)
                        bound = bound + 2.0 ** -25 * (seen.double() @ values.abs())
                    within("exact scores", out[a:b, h], want, bound)
                    most = torch.where(any_seen, x.amax(1).abs(), 0.0)
                    within("exact scores, lse", lse[a:b, h], z, most * 6 * ref.U32 + off)


def test_large_values_behind_rising_scores():
    """Values near the end of bf16, the second of them behind a score that rises by
    less than 2^8: nothing on the way is larger than the values' sum."""
    n, dim, heads = 300, 8, 320  # (as many heads as leave a share of the cache several blocks)
    scores = torch.full((n,), -60.0, device=DEV)
    scores[3], scores[131] = 0.0, 5.0
    q = torch.ones(1, heads, dim, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros(n, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[..., 0] = scores[:, None]
    v[...] = rand(gen(62), n, heads, dim)
    v[3], v[131] = 1e38, 2e38
    pages = -(-n // 16)
    k_cache, v_cache = (torch.zeros(pages, 16, heads, dim, dtype=q.dtype, device=DEV) for _ in range(2))
    k_cache.view(-1, heads, dim)[:n], v_cache.view(-1, heads, dim)[:n] = k, v
    table = torch.arange(pages, device=DEV, dtype=torch.int32)[None]
    few = [0, 7, heads - 1]
    out, lse = fgemm.attention_paged(q, k_cache, v_cache, table, ints([n]), scale=1.0)
    check_paged(q[:, few], [k[:, few]], [v[:, few]], 0, 1.0, out[:, few], lse[:, few], "large values, paged")
    for h in few:
        got = fgemm.attention(q[:, h:h + 1].contiguous(), k[:, h:h + 1].contiguous(), v[:, h:h + 1].contiguous(),
                              ints([0, 1]), k_starts=ints([0, n]), scale=1.0)
        check_prompt(q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], [0, 1], [0, n], True, 0, *got, 1.0,
                     "large values, prompt")


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_small_angles(interleaved):
    """The sine of a small angle has its bits: pairs (a, 0) and (0, b).  An angle rounds by
    2^-24 of itself and position * 2^-63 turns, the sine by two roundings more."""
    freq = torch.tensor([1e-8, -1e-8, 3e-9, -7e-10, 1e-6, 2e-3, 2.0 ** -30, 1.0], device=DEV)
    positions = [1, -1, 2, 3, -7, 100, 0]
    n, half = len(positions), len(freq)
    q = torch.zeros(n, 2, 2 * half, dtype=torch.bfloat16, device=DEV)
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    q[:, 0, first], q[:, 1, second] = 1.0, 1.0
    cache = [torch.zeros(1, n, 1, 2 * half, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    kv = torch.zeros(n, 1, 2 * half, dtype=torch.bfloat16, device=DEV)
    out = fgemm.rotary_cache(q, kv, kv, ints(positions), ints(range(n)), freq, *cache, interleaved=interleaved)
    at = torch.tensor(positions, dtype=torch.float64)[:, None]
    angle = at * ref.f64(freq)
    sine = torch.sin(angle)
    bound = 4 * ref.U32 * angle.abs() + at.abs() * 2.0 ** -60 + ref.store(sine, torch.bfloat16)
    within("small angles, a sin", out[:, 0, second], sine, bound)
    within("small angles, -b sin", out[:, 1, first], -sine, bound)
    cosine = torch.cos(angle)
    off = 4 * ref.U32 + ref.store(cosine, torch.bfloat16)
    within("small angles, a cos", out[:, 0, first], cosine, off)
    within("small angles, b cos", out[:, 1, second], cosine, off)


def test_sizes_beyond_32_bits():
    """What a C argument of 32 bits cannot hold is held to its largest, or refused; never
    taken less its upper bits."""
    q, k, v, starts, _ = prompt_inputs(gen(63), [90], [90], 2, 1, 64, torch.bfloat16)
    at = ints(starts)
    plain = fgemm.attention(q, k, v, at)
    cache = [x.view(6, 15, 1, 64) for x in (k, v)]
    table, n = ints([range(6)]), ints([90])
    step = fgemm.attention_paged(q[:1], *cache, table, n)
    for window in (2 ** 31, 2 ** 32 + 5, 2 ** 40 + 1):
        got = fgemm.attention(q, k, v, at, window=window)
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
        got = fgemm.attention_paged(q[:1], *cache, table, n, window=window)
        assert torch.equal(got[0], step[0]) and torch.equal(got[1], step[1])
    for call in (
            lambda: fgemm.attention(q, k, v, at, window=-2 ** 32),
            lambda: fgemm.attention_paged(q[:1], *cache, table, n, window=-2 ** 32),
            lambda: fgemm.attention(q[..., :0], k[..., :0], v[..., :0], at),
            lambda: fgemm.attention_paged(q[:1, :, :0], *(x[..., :0] for x in cache), table, n)):
        with pytest.raises(fgemm.FgemmError):
            call()


def test_threads_on_streams_of_their_own():
    """Two threads that share the default handle: each call runs on its thread's stream, so
    it reads what the thread wrote before and its results are there for what comes after."""
    g = gen(65)
    lengths = [700, 31, 1500]
    sets = []
    for i in range(2):
        q, k, v, starts, _ = prompt_inputs(gen(66 + i), lengths, lengths, 8, 2, 64, torch.bfloat16)
        table = torch.arange(140, device=DEV, dtype=torch.int32).view(1, -1)[:, :sum(lengths) // 16]
        logits = 3 * rand(g, 64, 5000)
        sets.append((q, k, v, ints(starts), table, ints([table.shape[1] * 16]), logits,
                     torch.arange(64, device=DEV, dtype=torch.int32)))

    def calls(q, k, v, starts, table, n, logits, tokens):
        """Inputs are written anew on this thread's stream, behind work that takes a while."""
        big = torch.empty(1 << 26, device=DEV).fill_(1.0)
        q, k, v, logits = (x * 1 for x in (q, k, v, logits + big[:1] - 1))
        out, lse = fgemm.attention(q, k, v, starts)
        pages = (k.shape[0] // 16, 16, *k.shape[1:])
        rows = pages[0] * 16
        step = fgemm.attention_paged(out[-1:], k[:rows].view(pages), v[:rows].view(pages), table, n)
        got = fgemm.logprobs(logits, tokens, top=3)
        return [x.clone() for x in (out, lse, *step, *got)]

    want = [calls(*x) for x in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(40):
                got = calls(*sets[i])
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and fgemm.default_handle().get_error() == fgemm.OK


@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (16, 1), (40, 2), (64, 1), (320, 320)])
@pytest.mark.parametrize("dim", [8, 64, 72, 128])
def test_paged_workspace(dim, heads, kv_heads):
    """Nothing is written around the workspace that a call asks for, and less, or one not on 16
    bytes, is refused: query heads of one and two eights and of several tiles, more key heads
    than the device holds shares."""
    few = kv_heads > 100
    lengths = [300, 0, 5000 if not few else 500, 64, 65]
    q, k, v, table, n, keys, values = paged_inputs(gen(heads + dim), lengths, heads, kv_heads, dim, 16, torch.bfloat16)
    L, h = fgemm.lib(), fgemm.default_handle()
    torch.cuda.synchronize()  # (the call below runs on whatever stream the handle has)
    h.set_stream(torch.cuda.current_stream().cuda_stream)
    size = L.fgemm_attention_paged_workspace(h.ptr, len(lengths), heads, kv_heads, dim)
    assert size > 0
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    cache = fgemm._cache(k, v, kv_heads, dim, q.dtype, 0)

    def call(workspace, count):
        return L.fgemm_attention_paged(h.ptr, len(lengths), heads, kv_heads, dim, q.data_ptr(), q.stride(0),
                                       q.stride(1), ctypes.byref(cache), table.data_ptr(), table.stride(0), table.shape[1],
                                       n.data_ptr(), dim ** -0.5, 0, fgemm.BF16, out.data_ptr(), out.stride(0),
                                       out.stride(1), lse.data_ptr(), workspace, count)

    guard = 1 << 16
    space = torch.full((size + 2 * guard,), 0xA5, dtype=torch.uint8, device=DEV)
    at = space.data_ptr() + guard
    for workspace, count, status in ((at, size - 1, fgemm.ERR_INVALID_ARG), (None, size, fgemm.ERR_INVALID_ARG),
                                     (at + 8, size + 8, fgemm.ERR_ALIGNMENT), (at, 0, fgemm.ERR_INVALID_ARG)):
        assert call(workspace, count) == status and "workspace" in h.last_message()
    assert call(at, size) == fgemm.OK
    torch.cuda.synchronize()
    assert bool((space[:guard] == 0xA5).all()) and bool((space[guard + size:] == 0xA5).all())
    for i in (0, heads - 1):
        one, of = slice(i, i + 1), slice(i // (heads // kv_heads), i // (heads // kv_heads) + 1)
        check_paged(q[:, one], [x[:, of] for x in keys], [x[:, of] for x in values], 0, None, out[:, one], lse[:, one],
                    "paged, workspace with guards")


@pytest.mark.parametrize("dim", [64, 128])
def test_outputs_at_the_end_of_f16(dim):
    """Values at +-65504, where many a pipeline saturates: an output is a mean of values and
    no larger, though 16-bit weights and their 32-bit sum differ by up to 2^-11.  Infinite
    values stay what they are."""
    lengths, heads, kv = [40, 300, 1, 700], 6, 2
    q, k, v, starts, _ = prompt_inputs(gen(68), lengths, lengths, heads, kv, dim, torch.float16)
    q *= 2
    k[50] = 0.0  # (the second sequence's eleventh key)
    v = (torch.finfo(torch.float16).max * rand(gen(69), 1, kv, dim).sign()).expand_as(v).half().contiguous()
    out, lse = fgemm.attention(q, k, v, ints(starts))
    check_prompt(q, k, v, starts, starts, True, 0, out, lse, what="largest values, prompt")
    pages = -(-max(lengths) // 16)
    table = torch.arange(len(lengths) * pages, device=DEV, dtype=torch.int32).view(-1, pages)
    caches = [torch.zeros(table.numel(), 16, kv, dim, dtype=q.dtype, device=DEV) for _ in range(2)]
    for s, n in enumerate(lengths):
        for c, x in zip(caches, (k, v)):
            c.view(len(lengths), -1, kv, dim)[s, :n] = x[starts[s]:starts[s + 1]]
    last = torch.tensor(starts[1:], device=DEV) - 1
    step = fgemm.attention_paged(q[last], *caches, table, ints(lengths))
    of = lambda x: [x[a:b] for a, b in zip(starts, starts[1:])]  # noqa: E731
    check_paged(q[last], of(k), of(v), 0, None, *step, "largest values, paged")
    v[50, 0, 3], v[50, 1, 5] = torch.inf, -torch.inf
    caches[1].view(len(lengths), -1, kv, dim)[1, 10] = v[50]
    wild, _ = fgemm.attention(q, k, v, ints(starts))
    assert bool((wild[50:340, :3, 3] == torch.inf).all()) and bool((wild[50:340, 3:, 5] == -torch.inf).all())
    rest = wild.clone()
    rest[50:340, :3, 3], rest[50:340, 3:, 5] = out[50:340, :3, 3], out[50:340, 3:, 5]
    v[50] = v[51]
    check_prompt(q, k, v, starts, starts, True, 0, rest, lse, what="largest values beside infinite ones, prompt")
    got, _ = fgemm.attention_paged(q[last], *caches, table, ints(lengths))
    assert bool((got[1, :3, 3] == torch.inf).all()) and bool((got[1, 3:, 5] == -torch.inf).all())
    assert int(torch.isinf(got).sum()) == heads
