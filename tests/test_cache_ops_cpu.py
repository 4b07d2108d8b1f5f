"""CPU tests of the operators around a key-value cache: every refusal of the C
entry points (the handle is checked last, so they need no device), and the
references the GPU tests use, on worked cases."""
import ctypes
import math

import pytest
import torch

import cache_reference as ref
from complexity_matmul_tcgen05_gb300 import fgemm

BAD, ALIGN, UNSUP = fgemm.ERR_INVALID_ARG, fgemm.ERR_ALIGNMENT, fgemm.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    from complexity_matmul_tcgen05_gb300 import build
    build.build()
    return fgemm.lib()


def refused(L, status, got, text):
    said = L.fgemm_last_message(None).decode()
    assert got == status and text in said, (got, said)


CACHE = dict(k=16, v=16, pages=10, page_size=16, k_page=16 * 128, k_token=128, k_head=64, v_page=16 * 128, v_token=128,
             v_head=64)


def cache_of(kw):
    c = {**CACHE, **{name: kw.pop(name) for name in CACHE if name in kw}}
    return ctypes.byref(fgemm.KvCache(*c.values())) if kw.pop("cache", True) else None


CACHE_REFUSALS = [
    (dict(cache=None), BAD, "cache must not be NULL"),
    (dict(pages=-1), BAD, "page_size"),
    (dict(page_size=0), BAD, "page_size"),
    (dict(pages=1 << 30, page_size=2), BAD, "page_size"),
    (dict(pages=1 << 62, page_size=4), BAD, "page_size"),
    (dict(k=None), BAD, "k and v"),
    (dict(v=None), BAD, "k and v"),
    (dict(k_page=56), BAD, "stride of the cache"),
    (dict(v_token=-128), BAD, "stride of the cache"),
    (dict(v_head=(1 << 36) + 8), BAD, "stride of the cache"),
    (dict(k_token=132), ALIGN, "cache"),
    (dict(k=24), ALIGN, "cache"),
    (dict(v=8), ALIGN, "cache"),
]


@pytest.mark.parametrize("kw,status,text", [
    (dict(), BAD, "handle is NULL"),
    (dict(T=0), BAD, "handle is NULL"),
    (dict(T=1, ldq=1), BAD, "handle is NULL"),
    (dict(heads=1, hsq=1, ldq=64), BAD, "handle is NULL"),
    (dict(pages=0, k=None, v=None), BAD, "handle is NULL"),
    (dict(rot=0, inv_freq=None), BAD, "handle is NULL"),
    (dict(dtype=2), BAD, "dtype"),
    (dict(T=-1), BAD, "sizes"),
    (dict(T=1 << 31), BAD, "sizes"),
    (dict(heads=0), BAD, "heads"),
    (dict(kv_heads=1025), BAD, "heads"),
    (dict(dim=0), BAD, "dim"),
    (dict(dim=60), BAD, "dim"),
    (dict(dim=136), BAD, "dim"),
    (dict(rot=63), BAD, "rot"),
    (dict(rot=66), BAD, "rot"),
    (dict(rot=-2), BAD, "rot"),
    (dict(positions=None), BAD, "NULL"),
    (dict(slots=None), BAD, "NULL"),
    (dict(inv_freq=None), BAD, "NULL"),
    (dict(slots=18), ALIGN, "4-byte"),
    (dict(q=None), BAD, "NULL"),
    (dict(k_in=None), BAD, "NULL"),
    (dict(v_in=None), BAD, "NULL"),
    (dict(out=None), BAD, "NULL"),
    (dict(ldq=56), BAD, "stride"),
    (dict(hsq=-64), BAD, "stride"),
    (dict(ldo=(1 << 36) + 8), BAD, "stride"),
    (dict(ldo=64), BAD, "overlap"),
    (dict(hso=64, ldo=192), BAD, "overlap"),
    (dict(T=(1 << 31) - 1024, heads=1024, kv_heads=1024, hso=1 << 30, ldo=1 << 36), BAD, "overlap"),  # (2^67 values)
    (dict(hsq=68), ALIGN, "16-byte"),
    (dict(q=24), ALIGN, "16-byte"),
    (dict(out=40), ALIGN, "16-byte"),
    (dict(out=16, ldo=512), BAD, "q's strides"),
] + CACHE_REFUSALS)
def test_rotary_refusals(L, kw, status, text):
    kw = dict(kw)
    c = cache_of(kw)
    a = {**dict(T=4, heads=4, kv_heads=2, dim=64, q=16, ldq=256, hsq=64, k_in=16, ldk=128, hsk=64, v_in=16, ldv=128,
                hsv=64, positions=16, slots=16, inv_freq=16, rot=64, inter=0, dtype=fgemm.BF16, out=32, ldo=256,
                hso=64), **kw}
    refused(L, status, L.fgemm_rotary_cache(None, *a.values(), c), text)


SOFTMAX_REFUSALS = [
    (dict(scale=0.0), BAD, "scale"),
    (dict(scale=-1.0), BAD, "scale"),
    (dict(scale=math.nan), BAD, "scale"),
    (dict(scale=math.inf), BAD, "scale"),
    (dict(scale=2.0 ** 65), BAD, "scale"),
    (dict(window=-1), BAD, "window"),
    (dict(lse=18), ALIGN, "lse"),
    (dict(heads=3), BAD, "multiple"),
    (dict(heads=0), BAD, "heads"),
    (dict(dim=12), BAD, "dim"),
    (dict(dim=256), BAD, "dim"),
    (dict(dtype=2), BAD, "dtype"),
    (dict(q=None), BAD, "NULL"),
    (dict(out=None), BAD, "NULL"),
    (dict(ldq=56), BAD, "stride"),
    (dict(ldq=260), ALIGN, "16-byte"),
    (dict(ldo=64), BAD, "overlap"),
]


@pytest.mark.parametrize("kw,status,text", [
    (dict(), BAD, "handle is NULL"),
    (dict(seqs=0), BAD, "handle is NULL"),
    (dict(table_pages=0, page_table=None), BAD, "handle is NULL"),
    (dict(lse=None), BAD, "handle is NULL"),
    (dict(seqs=-1), BAD, "sizes"),
    (dict(seqs=(1 << 20) + 1), BAD, "2^20"),
    (dict(table_pages=-1), BAD, "sizes"),
    (dict(lengths=None), BAD, "NULL"),
    (dict(page_table=None), BAD, "NULL"),
    (dict(ld_table=7), BAD, "ld_table"),
    (dict(lengths=18), ALIGN, "4-byte"),
    (dict(page_table=18), ALIGN, "4-byte"),
    (dict(out=16, ldo=512), BAD, "q's strides"),
] + SOFTMAX_REFUSALS + CACHE_REFUSALS)
def test_paged_refusals(L, kw, status, text):
    kw = dict(kw)
    c = cache_of(kw)
    a = {**dict(seqs=4, heads=4, kv_heads=2, dim=64, q=16, ldq=256, hsq=64, cache=c, page_table=16, ld_table=8,
                table_pages=8, lengths=16, scale=0.125, window=0, dtype=fgemm.BF16, out=32, ldo=256, hso=64, lse=16,
                work=None, size=0), **kw}
    a["cache"] = c
    refused(L, status, L.fgemm_attention_paged(None, *a.values()), text)


def test_paged_workspace_without_handle(L):
    assert L.fgemm_attention_paged_workspace(None, 4, 8, 2, 64) == 0


@pytest.mark.parametrize("kw,status,text", [
    (dict(), BAD, "handle is NULL"),
    (dict(T=0), BAD, "handle is NULL"),
    (dict(seqs=0), BAD, "handle is NULL"),
    (dict(T_k=0, k=None, v=None), BAD, "handle is NULL"),
    (dict(k_starts=None), BAD, "handle is NULL"),
    (dict(T=-1), BAD, "sizes"),
    (dict(T_k=1 << 31), BAD, "sizes"),
    (dict(seqs=-1), BAD, "seqs"),
    (dict(window=5, causal=0), BAD, "window needs"),
    (dict(starts=None), BAD, "starts"),
    (dict(starts=18), ALIGN, "4-byte"),
    (dict(k_starts=18), ALIGN, "4-byte"),
    (dict(k=None), BAD, "NULL"),
    (dict(v=None), BAD, "NULL"),
    (dict(hsk=32), BAD, "stride"),
    (dict(v=40), ALIGN, "16-byte"),
    (dict(out=16), BAD, "out must not be"),
    (dict(out=64), BAD, "out must not be"),
] + SOFTMAX_REFUSALS)
def test_prompt_refusals(L, kw, status, text):
    a = {**dict(seqs=2, T=8, T_k=8, heads=4, kv_heads=2, dim=64, q=16, ldq=256, hsq=64, k=64, ldk=128, hsk=64, v=80,
                ldv=128, hsv=64, starts=16, k_starts=16, causal=1, window=0, scale=0.125, dtype=fgemm.F16, out=32,
                ldo=256, hso=64, lse=16), **kw}
    refused(L, status, L.fgemm_attention(None, *a.values()), text)


@pytest.mark.parametrize("kw,status,text", [
    (dict(), BAD, "handle is NULL"),
    (dict(rows=0), BAD, "handle is NULL"),
    (dict(top=0, top_tokens=None, top_logprobs=None), BAD, "handle is NULL"),
    (dict(rows=1, ld=0), BAD, "handle is NULL"),
    (dict(type=3), BAD, "logits_type"),
    (dict(rows=-1), BAD, "rows"),
    (dict(vocab=-1), BAD, "rows"),
    (dict(vocab=(1 << 19) + 1, ld=1 << 20), UNSUP, "FGEMM_SAMPLE_MAX_VOCAB"),
    (dict(top=33), BAD, "top"),
    (dict(top=-1), BAD, "top"),
    (dict(logits=None), BAD, "NULL"),
    (dict(tokens=None), BAD, "NULL"),
    (dict(logprob=None), BAD, "NULL"),
    (dict(top_tokens=None), BAD, "NULL"),
    (dict(top_logprobs=None), BAD, "NULL"),
    (dict(ld=99), BAD, "ld"),
    (dict(type=2, logits=18), ALIGN, "aligned"),
    (dict(type=1, logits=17), ALIGN, "aligned"),
    (dict(entropy=18), ALIGN, "aligned"),
    (dict(top_tokens=18), ALIGN, "aligned"),
])
def test_logprobs_refusals(L, kw, status, text):
    a = {**dict(rows=2, vocab=100, logits=16, ld=100, type=2, tokens=16, top=5, logprob=16, entropy=16, top_tokens=16,
                top_logprobs=16), **kw}
    refused(L, status, L.fgemm_logprobs(None, *a.values()), text)


# ------------------------------------------------------------- the references


def test_reference_attention_on_worked_rows():
    # two keys with scores log 3 and 0: weights 3/4 and 1/4
    q, k = torch.ones(1, 1, 1).double(), torch.tensor([[[math.log(3)]], [[0.0]]], dtype=torch.float64)
    v = torch.tensor([[[4.0]], [[8.0]]]).double()
    out, lse, b, _ = ref.attend(q, k, v, torch.ones(1, 2, dtype=torch.bool), 1.0, torch.bfloat16)
    assert abs(out.item() - 5.0) < 1e-12 and abs(lse.item() - math.log(4)) < 1e-12 and 0 < b.item() < 0.1
    out, lse, _, _ = ref.attend(q, k, v, torch.zeros(1, 2, dtype=torch.bool), 1.0, torch.bfloat16)
    assert out.item() == 0 and lse.item() == -math.inf
    seen = ref.seen_by(3, 5, True, 2)
    assert seen.tolist() == [[False, True, True, False, False], [False, False, True, True, False],
                             [False, False, False, True, True]]
    assert ref.seen_by(3, 1, True, 0).tolist() == [[False], [False], [True]]


def test_reference_rotation_is_one():
    x = torch.randn(3, 2, 8, dtype=torch.float64, generator=torch.Generator().manual_seed(0))
    pos, freq = torch.tensor([0, 1, 1000]), torch.tensor([1.0, 0.1, 0.01])
    for interleaved in (False, True):
        y, _ = ref.rotate(x, pos, freq, interleaved)
        assert torch.equal(y[0], x[0]) and torch.equal(y[..., 6:], x[..., 6:])
        assert torch.allclose(y.square().sum(-1), x.square().sum(-1))
    y, _ = ref.rotate(x, pos, freq, True)
    assert torch.allclose(y[1, :, 2], x[1, :, 2] * math.cos(0.1) - x[1, :, 3] * math.sin(0.1), atol=1e-7)


def test_reference_logprobs_on_worked_rows():
    inf = math.inf
    x = torch.tensor([[math.log(0.5), math.log(0.25), math.log(0.25), -inf], [-inf] * 4, [inf, 0.0, inf, math.nan]]).double()
    given, entropy, tops, lp, *_ = ref.logprobs(x, torch.tensor([0, 1, 2]), 3)
    assert abs(given[0] - math.log(0.5)) < 1e-7 and given[1] == -inf and abs(given[2] + math.log(2)) < 1e-12
    assert abs(entropy[0] - 1.5 * math.log(2)) < 1e-7 and entropy[1] == 0 and abs(entropy[2] - math.log(2)) < 1e-12
    assert tops.tolist() == [[0, 1, 2], [-1, -1, -1], [0, 2, 1]]
    assert lp[2, 2] == -inf
