"""CPU tests of the token-step operators: every refusal of the C entry points
(the handle is checked last, so they need no device), and the gradient
formula of the norm against differences."""
import ctypes

import numpy as np
import pytest

import token_reference as ref
from complexity_matmul_tcgen05_gb300 import fgemm

BAD, ALIGN, UNSUP = fgemm.ERR_INVALID_ARG, fgemm.ERR_ALIGNMENT, fgemm.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    from complexity_matmul_tcgen05_gb300 import build
    build.build()
    return fgemm.lib()


def said(L):
    return L.fgemm_last_message(None).decode()


def refused(L, status, got, text):
    assert got == status and text in said(L), (got, said(L))


NORM = dict(M=4, N=64, x=16, ldx=64, res=None, ldr=0, gain=16, eps=1e-6, dtype=fgemm.BF16, total=None, ldt=0)


def norm(L, y=16, ldy=64, inv=16, **kw):
    a = {**NORM, **kw}
    return L.fgemm_rms_norm(None, *a.values(), y, ldy, inv)


def norm_mx(L, fmt=0, q=16, ldq=64, scales=16, lds=2, inv=16, **kw):
    a = {**NORM, **kw}
    return L.fgemm_rms_norm_mx(None, *a.values(), fmt, q, ldq, scales, lds, inv)


@pytest.mark.parametrize("call", [norm, norm_mx])
@pytest.mark.parametrize("kw,status,text", [
    (dict(), BAD, "handle is NULL"),
    (dict(M=0), BAD, "handle is NULL"),
    (dict(dtype=2), BAD, "dtype"),
    (dict(M=-1), BAD, "sizes"),
    (dict(N=1 << 31), BAD, "sizes"),
    (dict(N=0), BAD, "at least one value"),
    (dict(eps=-1.0), BAD, "eps"),
    (dict(eps=float("nan")), BAD, "eps"),
    (dict(eps=float("inf")), BAD, "eps"),
    (dict(x=None), BAD, "NULL"),
    (dict(gain=None), BAD, "NULL"),
    (dict(ldx=63), BAD, "leading dimension"),
    (dict(res=16, ldr=63), BAD, "leading dimension"),
    (dict(total=16, ldt=63), BAD, "leading dimension"),
    (dict(x=17), ALIGN, "aligned"),
    (dict(gain=17), ALIGN, "aligned"),
    (dict(inv=18), ALIGN, "aligned"),
])
def test_norm_refusals(L, call, kw, status, text):
    refused(L, status, call(L, **kw), text)


def test_norm_output_refusals(L):
    refused(L, BAD, norm(L, y=None), "NULL")
    refused(L, BAD, norm(L, ldy=63), "leading dimension")
    refused(L, ALIGN, norm(L, y=17), "aligned")
    refused(L, BAD, norm_mx(L, fmt=2), "format")
    refused(L, BAD, norm_mx(L, q=None), "NULL")
    refused(L, BAD, norm_mx(L, scales=None), "NULL")
    refused(L, BAD, norm_mx(L, ldq=63), "ldq")
    refused(L, BAD, norm_mx(L, lds=1), "lds")


@pytest.mark.parametrize("kw,status,text", [
    (dict(), BAD, "handle is NULL"),
    (dict(M=0), BAD, "handle is NULL"),
    (dict(dtype=7), BAD, "dtype"),
    (dict(M=-1), BAD, "sizes"),
    (dict(N=0), BAD, "at least one value"),
    (dict(dy=None), BAD, "NULL"),
    (dict(total=None), BAD, "NULL"),
    (dict(gain=None), BAD, "NULL"),
    (dict(inv=None), BAD, "NULL"),
    (dict(dx=None), BAD, "NULL"),
    (dict(lddy=63), BAD, "leading dimension"),
    (dict(dt=16, lddt=63), BAD, "leading dimension"),
    (dict(lddx=63), BAD, "leading dimension"),
    (dict(dgain=18), ALIGN, "dgain"),
    (dict(dy=17), ALIGN, "aligned"),
])
def test_norm_backward_refusals(L, kw, status, text):
    a = {**dict(M=4, N=64, dy=16, lddy=64, total=16, ldt=64, gain=16, inv=16, dt=None, lddt=0, dtype=fgemm.F16, dx=16,
                lddx=64, dgain=16, work=16, size=1 << 20), **kw}
    refused(L, status, L.fgemm_rms_norm_backward(None, *a.values()), text)


def test_norm_backward_workspace_without_handle(L):
    assert L.fgemm_rms_norm_backward_workspace(None, 4, 64) == 0


@pytest.mark.parametrize("kw,status,text", [
    (dict(), BAD, "handle is NULL"),
    (dict(M=0), BAD, "handle is NULL"),
    (dict(dtype=3), BAD, "dtype"),
    (dict(K=-1), BAD, "sizes"),
    (dict(K=(1 << 30) + 1), BAD, "sizes"),
    (dict(group=16), BAD, "group"),
    (dict(kind=9), BAD, "epilogue"),
    (dict(kind=3, N=63), BAD, "even N"),
    (dict(kind=1), BAD, "bias"),
    (dict(C=None), BAD, "C must"),
    (dict(ldc=63), BAD, "ldc"),
    (dict(C=17), ALIGN, "C and the bias"),
    (dict(bias=17), ALIGN, "C and the bias"),
    (dict(A=None), BAD, "NULL"),
    (dict(W=None), BAD, "NULL"),
    (dict(scales=None), BAD, "NULL"),
    (dict(lda=255), BAD, "lda"),
    (dict(ldw=127), BAD, "ldw"),
    (dict(lds=1), BAD, "lds"),
    (dict(zeros=16, ldz=1), BAD, "ldz"),
    (dict(A=18), ALIGN, "16-byte"),
    (dict(W=24), ALIGN, "16-byte"),
    (dict(lda=257), ALIGN, "16-byte"),
    (dict(ldw=136), ALIGN, "16-byte"),
    (dict(scales=17), ALIGN, "scales"),
    (dict(M=100), BAD, "workspace"),
    (dict(M=100, work=256, size=1000), BAD, "workspace"),
    (dict(M=100, work=272, size=1 << 20), ALIGN, "workspace"),
    (dict(M=100, work=256, size=1 << 20), BAD, "handle is NULL"),
])
def test_w4_refusals(L, kw, status, text):
    a = {**dict(M=4, N=64, K=256, A=16, lda=256, W=16, ldw=128, scales=16, lds=2, zeros=None, ldz=0, group=128, C=16,
                ldc=64, dtype=fgemm.BF16, kind=0, bias=None, work=None, size=0), **kw}
    epi, work = fgemm.Epilogue(a.pop("kind"), 1.0, a.pop("bias")), (a.pop("work"), a.pop("size"))
    refused(L, status, L.fgemm_matmul_w4(None, *a.values(), ctypes.byref(epi), *work), text)


@pytest.mark.parametrize("kw,status,text", [
    (dict(), BAD, "handle is NULL"),
    (dict(rows=0), BAD, "handle is NULL"),
    (dict(type=3), BAD, "logits_type"),
    (dict(rows=-1), BAD, "rows"),
    (dict(vocab=-1), BAD, "rows"),
    (dict(vocab=(1 << 19) + 1, ld=1 << 20), UNSUP, "FGEMM_SAMPLE_MAX_VOCAB"),
    (dict(logits=None), BAD, "NULL"),
    (dict(u=None), BAD, "NULL"),
    (dict(token=None), BAD, "NULL"),
    (dict(ld=99), BAD, "ld"),
    (dict(type=2, logits=18), ALIGN, "aligned"),
    (dict(type=0, logits=17), ALIGN, "aligned"),
    (dict(u=18), ALIGN, "aligned"),
    (dict(prob=18), ALIGN, "aligned"),
])
def test_sample_refusals(L, kw, status, text):
    a = {**dict(rows=2, vocab=100, logits=16, ld=100, type=2, u=16, token=16, prob=None), **kw}
    how = fgemm.Sampling(1.0, 0, 1.0, 0.0, None, None, None, None)
    got = L.fgemm_sample(None, a["rows"], a["vocab"], a["logits"], a["ld"], a["type"], a["u"], ctypes.byref(how),
                         a["token"], a["prob"])
    refused(L, status, got, text)


def test_sample_settings_refusals(L):
    refused(L, BAD, L.fgemm_sample(None, 2, 100, 16, 100, 2, 16, None, 16, None), "how")
    how = fgemm.Sampling(1.0, 0, 1.0, 0.0, 18, None, None, None)
    refused(L, ALIGN, L.fgemm_sample(None, 2, 100, 16, 100, 2, 16, ctypes.byref(how), 16, None), "aligned")


def test_norm_gradient_formula_against_differences():
    rng = np.random.default_rng(1)
    m, n, eps = 3, 17, 1e-3
    x, gain, dy, dt = (rng.standard_normal(s) for s in ((m, n), (n,), (m, n), (m, n)))

    def loss(x, gain):  # y enters through dy, the sum itself through dt
        return np.sum(ref.norm(x, gain, eps)[1] * dy) + np.sum(x * dt)

    inv, _ = ref.norm(x, gain, eps)
    dx, dgain = ref.norm_backward(dy, x, gain, inv, dt)
    h = 1e-6
    for i in range(m):
        for j in range(n):
            e = np.zeros((m, n))
            e[i, j] = h
            # central differences: h^2 of the third derivative and 2^-52 / h of the loss
            assert abs((loss(x + e, gain) - loss(x - e, gain)) / (2 * h) - dx[i, j]) < 1e-8
    for j in range(n):
        e = np.zeros(n)
        e[j] = h
        assert abs((loss(x, gain + e) - loss(x, gain - e)) / (2 * h) - dgain[j]) < 1e-8


def test_sample_reference_on_worked_rows():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    pick = lambda u, **kw: ref.sample_row(x, u, **{**dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **kw})[:2]  # noqa: E731
    assert pick(0.05)[0] == 0 and pick(0.3)[0] == 1 and pick(0.6)[0] == 2 and pick(0.9)[0] == 3
    assert pick(0.0, top_k=2)[0] == 1 and pick(0.99, top_k=2)[0] == 3
    assert abs(pick(0.0, top_k=2)[1] - 4 / 7) < 1e-12
    assert pick(0.0, top_p=0.65)[0] == 1 and pick(0.99, top_p=0.65)[0] == 3
    assert pick(0.99, top_p=0.35) == (1, 1.0)
    assert pick(0.0, min_p=0.6)[0] == 1 and pick(0.99, min_p=0.6)[0] == 3
    assert pick(0.5, temperature=0.0) == (1, 1.0)
    assert ref.sample_row(np.full(5, -np.inf), 0.5, 1.0, 0, 1.0, 0.0)[0] == -1
