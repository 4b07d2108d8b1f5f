"""The operators around a key-value cache against their formulas in 64 bits
(cache_reference.py), at the sizes, strides, masks and special values where
they can go wrong."""
import math
from fractions import Fraction

import pytest
import torch

import cache_reference as ref
from complexity_matmul_tcgen05_gb300 import fgemm
from parity_util import record

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INF, NAN = math.inf, math.nan


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def within(what, got, want, bound):
    """|got - want| <= bound where want is finite, equal where it is not; records the closest."""
    got = ref.f64(got)
    assert got.shape == want.shape
    finite = torch.isfinite(want)
    assert torch.equal(got[~finite].nan_to_num(nan=7.0), want[~finite].nan_to_num(nan=7.0)), what
    off = (got - want)[finite].abs()
    bound = bound.double()[finite]
    worst = float((off / bound.clamp_min(1e-300)).max()) if off.numel() else 0.0
    record(what, worst, 1.0)
    assert bool((off <= bound).all()), (what, worst)


def laid_out(t, how):
    """The same tokens x heads x dim values in memory of another order."""
    n, heads, dim = t.shape
    if how == "tight":
        return t.contiguous()
    if how == "head major":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((n, heads + 2, dim + 16), NAN, dtype=t.dtype, device=t.device)  # "padded"
    wide[:, 1:-1, 8:8 + dim] = t
    return wide[:, 1:-1, 8:8 + dim]


LAYOUTS = ["tight", "head major", "padded"]

# --------------------------------------------------------------------- rotary


def rotary_inputs(g, n, heads, kv_heads, dim, rot, t, page, spare=3):
    q, k, v = (rand(g, n, x, dim).to(t) for x in (heads, kv_heads, kv_heads))
    positions = torch.randint(0, 1 << 20, (n,), generator=g, device=DEV, dtype=torch.int32)
    pages = -(-n // page) + spare
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:n].to(torch.int32)
    freq = (1e4 ** (-2 * torch.arange(rot // 2, device=DEV).double() / max(rot, 1))).float()
    caches = [torch.full((pages, page, kv_heads, dim), 7.0, dtype=t, device=DEV) for _ in range(2)]
    return q, k, v, positions, slots, freq, *caches


def check_rotary(q, k, v, positions, slots, freq, k_cache, v_cache, interleaved, out, before=7.0):
    t = q.dtype
    pos, f = positions.cpu(), freq.cpu()
    wq, bq = ref.rotate(ref.f64(q), pos, f, interleaved)
    wk, bk = ref.rotate(ref.f64(k), pos, f, interleaved)
    within("rotary q", out, wq, bq + ref.store(wq, t))
    slots = slots.cpu().long()
    kept = (slots >= 0) & (slots < k_cache.shape[0] * k_cache.shape[1])
    kc, vc = ref.f64(k_cache).flatten(0, 1), ref.f64(v_cache).flatten(0, 1)
    at = slots[kept]
    within("rotary k", kc[at], wk[kept], bk[kept] + ref.store(wk[kept], t))
    assert torch.equal(vc[at], ref.f64(v)[kept])
    rest = torch.ones(kc.shape[0], dtype=torch.bool)
    rest[at] = False
    assert bool((kc[rest] == before).all()) and bool((vc[rest] == before).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(8, 8), (64, 64), (128, 128), (128, 96), (80, 80), (72, 36), (72, 2), (96, 0), (16, 14)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rotary_sizes(dtype, dim, rot, interleaved):
    for n, heads, kv_heads, page in ((1, 4, 2, 16), (5, 1, 1, 1), (67, 3, 2, 7)):
        a = rotary_inputs(gen(n * dim + rot), n, heads, kv_heads, dim, rot, TYPES[dtype], page)
        out = fgemm.rotary_cache(*a, interleaved=interleaved)
        check_rotary(*a, interleaved, out)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_layouts_padding_slots_and_in_place(layout, interleaved):
    g = gen(3)
    q, k, v, positions, slots, freq, k_cache, v_cache = rotary_inputs(g, 33, 6, 3, 64, 48, torch.bfloat16, 8)
    slots[4], slots[5], slots[6], slots[7] = -1, 1 << 30, k_cache.shape[0] * 8, -(1 << 31)
    q, k, v = (laid_out(x, layout) for x in (q, k, v))
    # a cache with pages head by head
    k_cache, v_cache = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (k_cache, v_cache))
    a = (q, k, v, positions, slots, freq, k_cache, v_cache)
    before = q.clone()
    out = fgemm.rotary_cache(*a, interleaved=interleaved)
    check_rotary(*a, interleaved, out)
    same = fgemm.rotary_cache(*a, interleaved=interleaved, out=q)
    assert same is q and torch.equal(q, out) and not torch.equal(q, before)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_any_frequency_and_position(interleaved):
    """Against angles reduced exactly: of every size of frequency, at the last positions."""
    freq = torch.tensor([1.0, -0.37, 1e-40, 3.1e-9, 1.9999999, 2.0, -1234.5678, 7.7e22], device=DEV)
    positions = ints([0, 1, -1, 12345, 999999937, 2 ** 31 - 1, -2 ** 31])
    turn = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899"
                        "8628034825342117067982148086513282306647093844609550582231725359408128481117450")
    angle = torch.tensor([[float((Fraction(f) * n) % turn) for f in freq.tolist()] for n in positions.tolist()],
                         dtype=torch.float64)
    n, half = angle.shape
    q, k, v = (rand(gen(29), n, 1, 2 * half).bfloat16() for _ in range(3))
    cache = [torch.zeros(1, n, 1, 2 * half, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    out = fgemm.rotary_cache(q, k, v, positions, ints(range(n)), freq, *cache, interleaved=interleaved)
    # (the reference forms position * frequency: positions of 1 leave the angles as they are)
    for row in range(n):
        want, b = ref.rotate(ref.f64(q[row:row + 1]), torch.ones(1), angle[row], interleaved)
        within("rotary any frequency", out[row:row + 1], want, b + ref.store(want, torch.bfloat16))
    freq[2], freq[5] = NAN, INF
    out = fgemm.rotary_cache(q, k, v, positions, ints(range(n)), freq, *cache, interleaved=interleaved)
    at = torch.tensor([4, 5, 10, 11] if interleaved else [2, 5, half + 2, half + 5])
    lost = torch.zeros(2 * half, dtype=torch.bool)
    lost[at] = True
    assert bool(torch.isnan(out[..., lost.to(DEV)]).all()) and bool(torch.isfinite(out[..., ~lost.to(DEV)]).all())


def test_rotary_many_tokens_far_and_negative_positions():
    q, k, v, positions, slots, freq, k_cache, v_cache = rotary_inputs(gen(9), 4099, 2, 1, 64, 64, torch.float16, 16)
    positions[0], positions[1], positions[2] = (1 << 31) - 1, -5, 0
    a = (q, k, v, positions, slots, freq, k_cache, v_cache)
    check_rotary(*a, False, fgemm.rotary_cache(*a))


# ---------------------------------------------------------------- paged cache


def paged_inputs(g, lengths, heads, kv_heads, dim, page, t, extra_pages=2, table_extra=1):
    """Tokens in scattered pages; slots that hold no token are NaN."""
    need = [-(-max(n, 0) // page) for n in lengths]
    total = sum(need) + extra_pages
    width = max(need + [0]) + table_extra
    k_cache, v_cache = (torch.full((total, page, kv_heads, dim), NAN, dtype=t, device=DEV) for _ in range(2))
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lengths), width), 1 << 30, dtype=torch.int32, device=DEV)
    keys, values, at = [], [], 0
    for s, n in enumerate(lengths):
        n = max(n, 0)
        k, v = (rand(g, n, kv_heads, dim).to(t) for _ in range(2))
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        j = torch.arange(n, device=DEV)
        pages = table[s].long()[j // page]
        k_cache[pages, j % page], v_cache[pages, j % page] = k, v
        keys.append(k)
        values.append(v)
    q = (1.5 * rand(g, len(lengths), heads, dim)).to(t)
    return q, k_cache, v_cache, table, ints(lengths), keys, values


def check_paged(q, keys, values, window, scale, out, lse, what="paged"):
    dim = q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    for s, (k, v) in enumerate(zip(keys, values)):
        seen = ref.seen_by(1, len(k), True, window)
        o, z, bo, bz = ref.attend(ref.f64(q[s:s + 1]), ref.f64(k), ref.f64(v), seen, scale, q.dtype)
        within(f"{what} out", out[s:s + 1], o, bo)
        within(f"{what} lse", lse[s:s + 1], z, bz)


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("dim", [8, 64, 72, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_paged_lengths(dtype, dim, page):
    lengths = [0, 1, 2, 15, 16, 17, 63, 64, 65, 255, 257, 700, 0]
    q, k, v, table, n, keys, values = paged_inputs(gen(dim + page), lengths, 4, 2, dim, page, TYPES[dtype])
    for window in (0, 1, 16, 100):
        out, lse = fgemm.attention_paged(q, k, v, table, n, window=window)
        check_paged(q, keys, values, window, None, out, lse)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 8), (7, 1), (14, 2), (16, 1), (24, 3), (17, 1), (48, 2), (64, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_paged_groups(dtype, heads, kv_heads):
    lengths = [300, 3, 1025]
    q, k, v, table, n, keys, values = paged_inputs(gen(heads), lengths, heads, kv_heads, 128, 16, TYPES[dtype])
    out, lse = fgemm.attention_paged(q, k, v, table, n, scale=0.2)
    check_paged(q, keys, values, 0, 0.2, out, lse)


@pytest.mark.parametrize("heads,kv_heads", [(8, 1), (9, 1), (15, 1), (32, 1), (33, 1), (18, 2)])
@pytest.mark.parametrize("dim", [40, 104])
def test_paged_groups_at_the_edges_of_tiles(heads, kv_heads, dim):
    lengths = [65, 0, 500, 17]
    q, k, v, table, n, keys, values = paged_inputs(gen(27), lengths, heads, kv_heads, dim, 11, torch.float16)
    out, lse = fgemm.attention_paged(q, k, v, table, n, window=300)
    check_paged(q, keys, values, 300, None, out, lse, "paged edges of tiles")


@pytest.mark.parametrize("layout", LAYOUTS)
def test_paged_layouts_and_in_place(layout):
    lengths = [37, 0, 400, 129]
    q, k, v, table, n, keys, values = paged_inputs(gen(1), lengths, 6, 3, 96, 24, torch.bfloat16)
    q = laid_out(q, layout)
    k = k.transpose(1, 2).contiguous().transpose(1, 2)  # pages head by head
    both = torch.stack((v, v), 2)  # values as a part of wider tokens
    v = both[:, :, 1]
    table = torch.cat((table, table), 1)[:, :table.shape[1]]
    into = laid_out(torch.full_like(q, 5.0), layout)
    out, lse = fgemm.attention_paged(q, k, v, table, n, out=into)
    assert out is into
    check_paged(q, keys, values, 0, None, out, lse)
    again, lse2 = fgemm.attention_paged(q, k, v, table, n, out=q)
    assert again is q and torch.equal(q, out) and torch.equal(lse, lse2)


def test_paged_bad_pages_and_lengths():
    lengths = [100, 64, 33, 50]
    q, k, v, table, n, keys, values = paged_inputs(gen(2), lengths, 4, 2, 64, 16, torch.float16, table_extra=0)
    table[0, 2], table[0, 4], table[1, 0] = -1, k.shape[0], (1 << 31) - 1
    table[2] = -(1 << 31)  # not one page is there
    seen = torch.arange(100, device=DEV)
    seen = seen[(seen // 16 != 2) & (seen // 16 != 4)]
    keys[0], values[0] = keys[0][seen], values[0][seen]
    keys[1], values[1] = keys[1][16:], values[1][16:]
    keys[2], values[2] = keys[2][:0], values[2][:0]
    out, lse = fgemm.attention_paged(q, k, v, table, n)
    check_paged(q, keys, values, 0, None, out, lse)
    # a length beyond the table reads what the table has, one below 0 nothing
    full = 16 * table.shape[1]
    q, k, v, table, n, keys, values = paged_inputs(gen(2), [full, full, 5], 4, 2, 64, 16, torch.float16, table_extra=0)
    n[0], n[1], n[2] = (1 << 31) - 1, full + 1, -3
    keys[2], values[2] = keys[2][:0], values[2][:0]
    out, lse = fgemm.attention_paged(q, k, v, table, n)
    check_paged(q, keys, values, 0, None, out, lse)
    empty = k[:0]
    out, lse = fgemm.attention_paged(q, empty, empty, table, n)
    assert bool((out == 0).all()) and bool((lse == -INF).all())
    out, lse = fgemm.attention_paged(q, k, v, table[:, :0], n)
    assert bool((out == 0).all()) and bool((lse == -INF).all())
    assert fgemm.attention_paged(q[:0], k, v, table[:0], n[:0])[0].shape == (0, 4, 64)


def test_paged_special_values():
    q, k, v, table, n, keys, values = paged_inputs(gen(5), [200, 200, 200, 200], 2, 1, 64, 16, torch.bfloat16)
    # a key far above the rest, one far below, an infinite value, a NaN key
    for s, (j, kv, vv) in enumerate(((150, 40.0, None), (0, -40.0, None), (77, None, INF), (199, NAN, None))):
        page, at = table[s, j // 16].long(), j % 16
        if kv is not None:
            keys[s][j] = (kv * q[s, 0] / 8).to(k.dtype) if kv == kv else NAN
            k[page, at] = keys[s][j]
        if vv is not None:
            values[s][j, 0, 3] = vv
            v[page, at] = values[s][j]
    out, lse = fgemm.attention_paged(q, k, v, table, n)
    check_paged(q[:2], keys[:2], values[:2], 0, None, out[:2], lse[:2], "paged far scores")
    assert bool((out[2, :, 3] == INF).all()) and bool(torch.isfinite(out[2, :, 4:]).all())
    assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(lse[3]).all())


def test_paged_only_nan_keys():
    q, k, v, table, n, _, _ = paged_inputs(gen(5), [1, 300], 2, 1, 64, 16, torch.bfloat16)
    k.fill_(NAN)
    out, lse = fgemm.attention_paged(q, k, v, table, n)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


def test_paged_long_context_and_repeatable():
    lengths = [70001, 3, 20000]
    q, k, v, table, n, keys, values = paged_inputs(gen(6), lengths, 8, 2, 64, 64, torch.bfloat16)
    out, lse = fgemm.attention_paged(q, k, v, table, n)
    check_paged(q, keys, values, 0, None, out, lse, "paged long")
    for _ in range(3):
        o2, l2 = fgemm.attention_paged(q, k, v, table, n)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_paged_long_short_and_empty_sequences():
    """More sequences than shares, some of them in many shares."""
    lengths = [0] * 30 + [5000] + [3] * 20 + [0, 700, 0] + [64] * 40 + [9000, 0]
    q, k, v, table, n, keys, values = paged_inputs(gen(28), lengths, 16, 8, 72, 16, torch.bfloat16)
    for _ in range(2):
        out, lse = fgemm.attention_paged(q, k, v, table, n)
        check_paged(q, keys, values, 0, None, out, lse, "paged mixed lengths")
    plain = out.clone()
    out, lse2 = fgemm.attention_paged(q, k, v, table, n, out=q)
    assert out is q and torch.equal(out, plain) and torch.equal(lse, lse2)


def small_weights(n, tops):
    """n keys with scores of 0 at `tops` and -13.8 elsewhere, which many make count: a
    weight is 16.44 * 2^-24, between two of fp16's steps there.  Values are 0 and 1.  Also the
    output and its bound: two roundings to fp16, and half of one for the sums of up to
    n / 4 in 32 bits (2^-24 each step) and the scores (20 * 2^-24)."""
    scores = torch.full((n,), -13.8359375, dtype=torch.float16, device=DEV)
    values = torch.ones(n, dtype=torch.float16, device=DEV)
    scores[tops], values[tops] = 0.0, 0.0
    w = torch.exp(scores.double().cpu())
    want = (w * values.double().cpu()).sum() / w.sum()
    return scores, values, want, want * 2.5 * 2.0 ** -11


def test_paged_small_weights_in_f16():
    n, heads = 16384, 320  # more heads than the device holds shares of: a warp sees a quarter of the keys
    scores, values, want, bound = small_weights(n, [0, 16, 32, 48])
    q = torch.ones(1, heads, 8, dtype=torch.float16, device=DEV)
    k = torch.zeros(n // 64, 64, heads, 8, dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    k[..., 0], v[...] = scores.view(-1, 64, 1), values.view(-1, 64, 1, 1)
    out, _ = fgemm.attention_paged(q, k, v, torch.arange(n // 64, device=DEV, dtype=torch.int32)[None], ints([n]), scale=1.0)
    within("paged small weights", out, want.expand(out.shape), bound.expand(out.shape))


def test_paged_many_sequences():
    g = gen(7)
    lengths = torch.randint(0, 90, (1500,), generator=torch.Generator().manual_seed(1)).tolist()
    q, k, v, table, n, keys, values = paged_inputs(g, lengths, 2, 1, 32, 8, torch.float16)
    out, lse = fgemm.attention_paged(q, k, v, table, n)
    check_paged(q, keys, values, 0, None, out, lse, "paged many")


def test_paged_cache_beyond_32_bit_offsets():
    # two pages more than 2^32 elements apart
    stride = (1 << 32) + 64
    big = torch.empty(stride + 16 * 64, dtype=torch.bfloat16, device=DEV)
    k = big.as_strided((2, 16, 1, 64), (stride, 64, 64, 1))
    g = gen(8)
    k[0], k[1] = rand(g, 16, 1, 64), rand(g, 16, 1, 64)
    q = rand(g, 1, 4, 64).bfloat16()
    table, n = ints([[1, 0]]), ints([25])
    out, lse = fgemm.attention_paged(q, k, k, table, n)
    keys = torch.cat((k[1], k[0]))[:25].clone()
    check_paged(q, [keys], [keys], 0, None, out, lse, "paged far pages")
    v = torch.empty(2, 16, 1, 64, dtype=torch.bfloat16, device=DEV)
    fgemm.rotary_cache(q, keys[:1], keys[1:2], ints([0]), ints([31]), torch.ones(32, device=DEV), k, v)
    assert torch.equal(k[1, 15], keys[0])


def test_paged_in_a_graph_with_other_lengths_and_streams():
    lengths = [40, 900]
    q, k, v, table, n, keys, values = paged_inputs(gen(10), lengths, 8, 4, 128, 16, torch.bfloat16)
    first = fgemm.attention_paged(q, k, v, table, n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fgemm.attention_paged(q, k, v, table, n)
    graph.replay()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    n.copy_(ints([17, 300]))
    graph.replay()
    check_paged(q, [keys[0][:17], keys[1][:300]], [values[0][:17], values[1][:300]], 0, None, out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = fgemm.attention_paged(q, k, v, table, n)
    b = fgemm.attention_paged(q, k, v, table, n)  # two calls at once, a workspace each
    torch.cuda.synchronize()
    assert torch.equal(a[0], out) and torch.equal(b[0], out) and torch.equal(a[1], b[1])


# --------------------------------------------------------------------- prompt


def prompt_inputs(g, lengths, k_lengths, heads, kv_heads, dim, t):
    q = (1.5 * rand(g, sum(lengths), heads, dim)).to(t)
    k, v = (rand(g, sum(k_lengths), kv_heads, dim).to(t) for _ in range(2))
    starts, k_starts = [0], [0]
    for a, b in zip(lengths, k_lengths):
        starts.append(starts[-1] + a)
        k_starts.append(k_starts[-1] + b)
    return q, k, v, starts, k_starts


def check_prompt(q, k, v, starts, k_starts, causal, window, out, lse, scale=None, what="prompt"):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    q, k, v = ref.f64(q), ref.f64(k), ref.f64(v)
    for s in range(len(starts) - 1):
        a, b, c, d = starts[s], starts[s + 1], k_starts[s], k_starts[s + 1]
        if a == b:
            continue
        o, z, bo, bz = ref.attend(q[a:b], k[c:d], v[c:d], ref.seen_by(b - a, d - c, causal, window), scale, out.dtype)
        within(f"{what} out", out[a:b], o, bo)
        within(f"{what} lse", lse[a:b], z, bz)


MASKS = [(True, 0), (False, 0), (True, 1), (True, 100), (True, 129)]


@pytest.mark.parametrize("causal,window", MASKS)
@pytest.mark.parametrize("dim", [8, 64, 72, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prompt_lengths(dtype, dim, causal, window):
    lengths = [1, 2, 63, 64, 65, 127, 128, 129, 0, 255, 256, 257, 300]
    q, k, v, starts, _ = prompt_inputs(gen(dim + window), lengths, lengths, 2, 1, dim, TYPES[dtype])
    out, lse = fgemm.attention(q, k, v, ints(starts), causal=causal, window=window)
    check_prompt(q, k, v, starts, starts, causal, window, out, lse)


@pytest.mark.parametrize("causal,window", MASKS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prompt_keys_of_another_length(dtype, causal, window):
    # prefixes, rows that see nothing (fewer keys than queries), no keys, no queries
    lengths, k_lengths = [5, 130, 200, 1, 0, 40, 129, 3], [300, 131, 77, 1000, 50, 0, 129, 2]
    q, k, v, starts, k_starts = prompt_inputs(gen(11), lengths, k_lengths, 4, 2, 64, TYPES[dtype])
    out, lse = fgemm.attention(q, k, v, ints(starts), k_starts=ints(k_starts), causal=causal, window=window)
    check_prompt(q, k, v, starts, k_starts, causal, window, out, lse)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (7, 1), (16, 2), (20, 1)])
@pytest.mark.parametrize("dim", [32, 96, 128])
def test_prompt_groups(heads, kv_heads, dim):
    lengths = [200, 33, 400]
    q, k, v, starts, _ = prompt_inputs(gen(heads), lengths, lengths, heads, kv_heads, dim, torch.bfloat16)
    out, lse = fgemm.attention(q, k, v, ints(starts), scale=0.3)
    check_prompt(q, k, v, starts, starts, True, 0, out, lse, 0.3)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_prompt_layouts_and_rows_of_no_sequence(layout):
    lengths = [100, 300]
    q, k, v, starts, _ = prompt_inputs(gen(12), [7] + lengths + [30], [7] + lengths + [30], 4, 2, 80, torch.float16)
    starts = starts[1:-1]  # 7 rows before the first sequence, 30 behind the last
    q, k, v = (laid_out(x, layout) for x in (q, k, v))
    out, lse = laid_out(torch.full_like(q, 5.0), layout), torch.full(q.shape[:2], 5.0, device=DEV)
    got = fgemm.attention(q, k, v, ints(starts), out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check_prompt(q, k, v, starts, starts, True, 0, out, lse)
    for rows in (slice(0, 7), slice(starts[-1], None)):
        assert bool((out[rows] == 5).all()) and bool((lse[rows] == 5).all())
    if layout == "padded":  # nothing beside the heads either
        edge = out.as_strided((q.shape[0], 8), (out.stride(0), 1), out.storage_offset() - 8)
        assert bool(torch.isnan(edge).all())


def test_prompt_long():
    lengths = [3000, 1, 1111]
    q, k, v, starts, _ = prompt_inputs(gen(13), lengths, lengths, 2, 1, 128, torch.bfloat16)
    for causal, window in ((True, 0), (True, 777), (False, 0)):
        out, lse = fgemm.attention(q, k, v, ints(starts), causal=causal, window=window)
        check_prompt(q, k, v, starts, starts, causal, window, out, lse, what="prompt long")
        again = fgemm.attention(q, k, v, ints(starts), causal=causal, window=window)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_prompt_many_sequences():
    lengths = torch.randint(0, 40, (700,), generator=torch.Generator().manual_seed(2)).tolist()
    q, k, v, starts, _ = prompt_inputs(gen(14), lengths, lengths, 2, 2, 16, torch.float16)
    out, lse = fgemm.attention(q, k, v, ints(starts))
    check_prompt(q, k, v, starts, starts, True, 0, out, lse, what="prompt many")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("where", [0, 70, 128, 259, 399])
def test_prompt_values_reach_only_queries_that_see_them(where, bad, dim):
    """A key and a value that are not finite: rows that do not see them are as
    without, in the same sequence (causal, window) and in its neighbours."""
    lengths = [100, 400, 60]
    q, k, v, starts, _ = prompt_inputs(gen(15), lengths, lengths, 2, 1, dim, torch.bfloat16)
    for window in (0, 50, 200):
        plain, plain_lse = fgemm.attention(q, k, v, ints(starts), window=window)
        vv, kk = v.clone(), k.clone()
        vv[100 + where, 0, 3] = bad
        out, lse = fgemm.attention(q, k, vv, ints(starts), window=window)
        rows = torch.arange(q.shape[0], device=DEV)
        sees = (rows >= 100 + where) & (rows < 500) & ((rows < 100 + where + window) | (window == 0))
        check_prompt(q, k, v, starts, starts, True, window, torch.where(sees[:, None, None], plain, out), lse,
                     what="beside a value that is not finite")
        assert not bool(torch.isfinite(out[sees][:, :, 3]).any())
        # the other values of those rows do not change (but for another order of the sums)
        rest = out.clone()
        rest[:, :, 3] = plain[:, :, 3]
        check_prompt(q, k, v, starts, starts, True, window, rest, lse, what="beside a value that is not finite")
        kk[100 + where] = NAN
        out, lse = fgemm.attention(q, kk, v, ints(starts), window=window)
        assert bool(torch.isnan(out[sees]).all()) and bool(torch.isnan(lse[sees]).all())
        check_prompt(q, k, v, starts, starts, True, window, torch.where(sees[:, None, None], plain, out),
                     torch.where(sees[:, None], plain_lse, lse), what="beside a NaN key")


def test_prompt_far_scores():
    lengths = [513]
    q, k, v, starts, _ = prompt_inputs(gen(16), lengths, lengths, 2, 1, 64, torch.bfloat16)
    # scores that grow along the keys, and a query whose scores are all far below 0
    k[:, 0] = (torch.arange(513, device=DEV)[:, None] / 513 * 60 * q[500, 0] / q[500, 0].float().norm()).bfloat16()
    q[400] = -q[500] * 4
    for causal in (True, False):
        out, lse = fgemm.attention(q, k, v, ints(starts), causal=causal, scale=1.0)
        check_prompt(q, k, v, starts, starts, causal, 0, out, lse, 1.0, "prompt far scores")


def test_prompt_small_weights_in_f16():
    n = 16384
    scores, values, want, bound = small_weights(n, [0])
    q = torch.ones(3, 2, 8, dtype=torch.float16, device=DEV)
    k, v = torch.zeros(n, 2, 8, dtype=torch.float16, device=DEV), torch.zeros(n, 2, 8, dtype=torch.float16, device=DEV)
    k[..., 0], v[...] = scores[:, None], values[:, None, None]
    out, _ = fgemm.attention(q, k, v, ints([0, 3]), k_starts=ints([0, n]), causal=False, scale=1.0)
    within("prompt small weights", out, want.expand(out.shape), bound.expand(out.shape))


def test_prompt_bad_starts_stay_inside():
    q, k, v, _, _ = prompt_inputs(gen(17), [64], [64], 2, 1, 64, torch.bfloat16)
    out, lse = torch.full_like(q, 5.0), torch.full((64, 2), 5.0, device=DEV)
    fgemm.attention(q, k, v, ints([-10, 20, 1 << 30]), out=out, lse=lse)
    check_prompt(q, k, v, [0, 20, 64], [0, 20, 64], True, 0, out, lse)
    out.fill_(5.0)
    fgemm.attention(q, k, v, ints([40, 20, 10]), out=out, lse=lse)  # not ascending: no rows, or some of them
    fgemm.attention(q, k, v, ints([64, 64]), out=out)
    empty, empty_lse = fgemm.attention(q, k[:0], v[:0], ints([0, 64]))
    assert bool((empty == 0).all()) and bool((empty_lse == -INF).all())
    torch.cuda.synchronize()
    assert fgemm.default_handle().get_error() == fgemm.OK


@pytest.mark.parametrize("causal,window", MASKS)
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 72), ("bf16", 64), ("f16", 128)])
def test_prompt_pairs_of_heads(dtype, dim, causal, window):
    """Enough rows and heads that share their keys for two of them at a time: prefixes,
    rows that see nothing, no keys, no queries, a value that is not finite."""
    lengths, k_lengths = [5, 130, 300, 1, 0, 40, 129, 300], [300, 131, 77, 1000, 50, 0, 129, 333]
    heads, kv = 64, 16
    q, k, v, starts, k_starts = prompt_inputs(gen(23), lengths, k_lengths, heads, kv, dim, TYPES[dtype])
    out, lse = fgemm.attention(q, k, v, ints(starts), k_starts=ints(k_starts), causal=causal, window=window)
    assert fgemm.default_handle().get_error() == fgemm.OK
    looked = [0, 3, 29, 62, 63]
    for h in looked:
        check_prompt(q[:, h:h + 1], k[:, h // 4:h // 4 + 1], v[:, h // 4:h // 4 + 1], starts, k_starts, causal, window,
                     out[:, h:h + 1], lse[:, h:h + 1], what="prompt pairs")
    at = k_starts[-2] + 200  # a key of the last sequence; its queries stand at 33 .. 332 of 333
    v2 = v.clone()
    v2[at, 7, 5] = INF
    wild, wild_lse = fgemm.attention(q, k, v2, ints(starts), k_starts=ints(k_starts), causal=causal, window=window)
    rows = torch.arange(q.shape[0], device=DEV)
    place = rows - starts[-2] + 33
    sees = (rows >= starts[-2]) & ((place >= 200) | (not causal)) & ((place < 200 + window) | (window == 0))
    for h in (28, 31):
        assert not bool(torch.isfinite(wild[sees][:, h, 5]).any())
        rest = wild[:, h:h + 1].clone()
        rest[sees, :, 5] = out[sees, h:h + 1, 5]
        check_prompt(q[:, h:h + 1], k[:, 7:8], v[:, 7:8], starts, k_starts, causal, window, rest, wild_lse[:, h:h + 1],
                     what="prompt pairs beside an infinite value")
    others = [h for h in range(heads) if h // 4 != 7]
    assert torch.equal(wild[:, others], out[:, others]) and torch.equal(wild_lse, lse)


@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_many_jobs_a_cta(dim):
    """More rows than the SMs hold at once, of sequences of very different
    lengths, right behind work that has emptied the caches: no wait runs out."""
    lengths = [700, 0, 3, 900, 130, 1, 257, 0, 400, 2100]
    q, k, v, starts, _ = prompt_inputs(gen(19), lengths, lengths, 32, 8, dim, torch.bfloat16)
    for _ in range(3):
        torch.zeros(1 << 27, device=DEV)
        out, lse = fgemm.attention(q, k, v, ints(starts))
    torch.cuda.synchronize()
    assert fgemm.default_handle().get_error() == fgemm.OK
    few = torch.tensor([0, 13, 31], device=DEV)  # heads that are looked at
    for h in few.tolist():
        check_prompt(q[:, h:h + 1], k[:, h // 4:h // 4 + 1], v[:, h // 4:h // 4 + 1], starts, starts, True, 0,
                     out[:, h:h + 1], lse[:, h:h + 1], what="prompt jobs")


def test_prompt_in_a_graph_and_on_two_streams():
    lengths = [300, 77]
    q, k, v, starts, _ = prompt_inputs(gen(18), lengths, lengths, 4, 2, 128, torch.bfloat16)
    at = ints(starts)
    first = fgemm.attention(q, k, v, at)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fgemm.attention(q, k, v, at)
    graph.replay()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    at.copy_(ints([0, 30, 377]))
    graph.replay()
    check_prompt(q, k, v, [0, 30, 377], [0, 30, 377], True, 0, out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = fgemm.attention(q, k, v, at)
    b = fgemm.attention(q, k, v, at)
    torch.cuda.synchronize()
    assert torch.equal(a[0], out) and torch.equal(b[0], out)


# ------------------------------------------------------------------- logprobs


def check_logprobs(x, tokens, top, got):
    lp, ent, tops, top_lp = got
    g, e, wt, wl, bg, be, bt = ref.logprobs(ref.f64(x), tokens.cpu().long(), top)
    within("logprob", lp, g, bg)
    within("entropy", ent, e, be)
    assert torch.equal(tops.cpu().long(), wt)
    within("top logprobs", top_lp, wl, bt)


@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 255, 1024, 1025, 4099, 50257, 131072, 200001])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_logprobs_sizes(dtype, vocab):
    g = gen(vocab)
    for rows, top in ((1, 5), (3, 32), (2, 0), (5, 1)):
        x = (3 * rand(g, rows, vocab)).to(TYPES[dtype])
        tokens = torch.randint(0, vocab, (rows,), generator=g, device=DEV, dtype=torch.int32)
        check_logprobs(x, tokens, top, fgemm.logprobs(x, tokens, top=top))


@pytest.mark.parametrize("shift", [0, 1, 3, 5])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_strides(dtype, shift):
    g = gen(shift)
    wide = torch.full((9, 5021 + 13), INF, dtype=TYPES[dtype], device=DEV)
    x = wide[:, shift:shift + 5021]
    x.copy_(2 * rand(g, 9, 5021))
    tokens = torch.randint(0, 5021, (9,), generator=g, device=DEV, dtype=torch.int32)
    check_logprobs(x, tokens, 20, fgemm.logprobs(x, tokens, top=20))


@pytest.mark.parametrize("vocab", [40, 5000, 70000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_masks_ties_and_specials(dtype, vocab):
    g = gen(20)
    t = TYPES[dtype]
    x = rand(g, 14, vocab).to(t)
    x[0] = -INF
    x[1] = 0.0  # all equal: the first tokens
    x[2] = -INF
    x[2, vocab - 1] = -50.0  # one token left
    x[3, ::2] = -INF
    x[4, 5] = x[4, vocab - 2] = INF
    x[5, 3::3] = NAN
    x[6] = torch.arange(vocab, device=DEV).to(t)  # rising, with ties in 16 bits
    x[7] = -torch.arange(vocab, device=DEV).float().to(t) / 64
    x[8] = (torch.arange(vocab, device=DEV) % 3).to(t)  # three values
    x[9] = x[9].abs() * -1e-3
    x[9, 11] = 25.0  # a probability near 1
    x[10, ::2], x[10, 1::2] = 0.0, -0.0  # equal
    x[11] = -INF
    x[11, 4:9] = 1.0  # fewer than `top` left
    x[12] = torch.finfo(t).max
    x[13] = torch.finfo(t).min
    tokens = ints([3, 7, vocab - 1, 2, 5, 3, vocab - 1, 0, 1, 11, 8, 2, 9, 9])
    check_logprobs(x, tokens, 32, fgemm.logprobs(x, tokens, top=32))
    check_logprobs(x, tokens, 3, fgemm.logprobs(x, tokens, top=3))
    out = ints([-1, vocab, 1 << 30, -(1 << 31), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0])
    check_logprobs(x, out, 0, fgemm.logprobs(x, out))


def test_logprobs_edges():
    x = torch.zeros(3, 0, device=DEV)
    lp, ent, tops, top_lp = fgemm.logprobs(x, ints([0, 1, -1]), top=4)
    assert bool((lp == -INF).all()) and bool((ent == 0).all()) and bool((tops == -1).all()) and bool((top_lp == -INF).all())
    lp, _, tops, _ = fgemm.logprobs(torch.zeros(0, 5, device=DEV), ints([]), top=2)
    assert lp.shape == (0,) and tops.shape == (0, 2)
    g = gen(21)
    x = (4 * rand(g, 700, 999)).bfloat16()  # more rows than SMs
    tokens = torch.randint(0, 999, (700,), generator=g, device=DEV, dtype=torch.int32)
    check_logprobs(x, tokens, 8, fgemm.logprobs(x, tokens, top=8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fgemm.logprobs(x, tokens, top=8)
    graph.replay()
    check_logprobs(x, tokens, 8, got)


# ------------------------------------------------------------- Python refusals


def test_python_refusals():
    q, k, v, table, n, _, _ = paged_inputs(gen(30), [20], 4, 2, 64, 16, torch.bfloat16)
    flat = [rand(gen(1), 5, 2, 64).bfloat16() for _ in range(3)]
    for call in (
            lambda: fgemm.attention_paged(q[0], k, v, table, n),
            lambda: fgemm.attention_paged(q.float(), k, v, table, n),
            lambda: fgemm.attention_paged(q.cpu(), k, v, table, n),
            lambda: fgemm.attention_paged(q, k.half(), v, table, n),
            lambda: fgemm.attention_paged(q, k, v[:, :8], table, n),
            lambda: fgemm.attention_paged(q, k, v, table.long(), n),
            lambda: fgemm.attention_paged(q, k, v, table, n.long()),
            lambda: fgemm.attention_paged(q, k, v, table[0], n),
            lambda: fgemm.attention_paged(q[:, :3], k, v, table, n),
            lambda: fgemm.attention_paged(q, k, v, table, n, scale=0.0),
            lambda: fgemm.attention_paged(q, k, v, table, n, out=q[:, :2]),
            lambda: fgemm.attention(*flat, ints([0, 5]).long()),
            lambda: fgemm.attention(*flat, ints([[0, 5]])),
            lambda: fgemm.attention(*flat, ints([0, 5]), k_starts=ints([0])),
            lambda: fgemm.attention(*flat, ints([0, 5]), causal=False, window=3),
            lambda: fgemm.attention(*flat, ints([0, 5]), out=flat[0]),
            lambda: fgemm.attention(flat[0], flat[1], flat[2][:4], ints([0, 5])),
            lambda: fgemm.attention(flat[0][..., ::2], flat[1], flat[2], ints([0, 5])),
            lambda: fgemm.attention(flat[0].expand(5, 2, 64), flat[1][:1].expand(5, 2, 64), flat[2], ints([0, 5])),
            lambda: fgemm.attention(*flat, ints([0, 5]), lse=torch.empty(5, 2, device=DEV, dtype=torch.float64)),
            lambda: fgemm.rotary_cache(*flat, ints([0] * 5).float(), ints([0] * 5), torch.ones(32, device=DEV), k, v),
            lambda: fgemm.rotary_cache(*flat, ints([0] * 5), ints([0] * 4), torch.ones(32, device=DEV), k, v),
            lambda: fgemm.rotary_cache(*flat, ints([0] * 5), ints([0] * 5), torch.ones(33, device=DEV), k, v),
            lambda: fgemm.rotary_cache(*flat, ints([0] * 5), ints([0] * 5), torch.ones(32, device=DEV), k[..., :32], v),
            lambda: fgemm.logprobs(flat[0], ints([0] * 5)),
            lambda: fgemm.logprobs(flat[0][:, 0].double(), ints([0] * 5)),
            lambda: fgemm.logprobs(flat[0][:, 0], ints([0] * 5), top=33),
            lambda: fgemm.logprobs(flat[0][:, 0], ints([0] * 5).long())):
        with pytest.raises(fgemm.FgemmError):
            call()
