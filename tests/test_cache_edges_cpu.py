"""What the calls around a key-value cache do with arguments that their C forms cannot
hold, or may not take: no device needed."""
import threading
import time

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


# ------------------------------------------------- refusals of the C entry points


@pytest.fixture(scope="module")
def L():
    from complexity_matmul_tcgen05_gb300 import build
    build.build()
    return fgemm.lib()


def refused(L, status, got, text):
    said = L.fgemm_last_message(None).decode()
    assert got == status and text in said, (got, said)


@pytest.mark.parametrize("kw,status,text", [
    (dict(seqs=(1 << 20) + 1), fgemm.ERR_INVALID_ARG, "seqs must be"),
    (dict(seqs=1 << 20), fgemm.ERR_INVALID_ARG, "handle is NULL"),
    (dict(T=(1 << 31) - 1024, heads=128), fgemm.ERR_UNSUPPORTED, "below 2^31"),
    (dict(T=128, seqs=1 << 20, heads=1024, ldq=1024 * 64, ldo=1024 * 64), fgemm.ERR_INVALID_ARG, "handle is NULL"),
    (dict(T=(1 << 31) - 1024, heads=126, ldq=126 * 64, ldo=126 * 64), fgemm.ERR_INVALID_ARG, "handle is NULL"),
    (dict(lse=None), fgemm.ERR_INVALID_ARG, "handle is NULL"),
])
def test_prompt_sizes_that_a_launch_cannot_have(L, kw, status, text):
    a = {**dict(seqs=2, T=8, T_k=8, heads=4, kv_heads=2, dim=64, q=16, ldq=256, hsq=64, k=64, ldk=128, hsk=64, v=80,
                ldv=128, hsv=64, starts=16, k_starts=16, causal=1, window=0, scale=0.125, dtype=fgemm.F16, out=32,
                ldo=256, hso=64, lse=16), **kw}
    refused(L, status, L.fgemm_attention(None, *a.values()), text)


@pytest.mark.parametrize("rows,text", [((1 << 27) + 1, "rows must be"), (1 << 27, "handle is NULL")])
def test_logprobs_of_too_many_rows(L, rows, text):
    refused(L, fgemm.ERR_INVALID_ARG, L.fgemm_logprobs(None, rows, 100, 16, 100, 2, 16, 5, 16, 16, 16, 16), text)


# ------------------------------------------------------------------------ threads


class OnDevice(torch.Tensor):
    """A CPU tensor that the binding takes for one on cuda:0."""

    def get_device(self):
        return 0


class Library:
    """Stands for the C library: a call notes the stream that the handle has then.  The
    first thread that sets a stream waits a while for the second to set its own."""

    def __init__(self):
        self.stream, self.seen, self.both, self.sets = None, {}, threading.Event(), 0

    def fgemm_set_stream(self, handle, stream):
        self.stream = stream
        self.sets += 1
        if self.sets == 1:
            self.both.wait(0.5)
        else:
            self.both.set()
        return fgemm.OK

    def called(self, *args):
        self.seen[threading.get_ident()] = self.stream
        return fgemm.OK

    fgemm_logprobs = fgemm_rms_norm = called


def in_two_threads(call):
    threads = [threading.Thread(target=call) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


def test_threads_share_a_handle(monkeypatch):
    """Each call runs on its own thread's stream."""
    for call in (lambda x, n, h: fgemm.logprobs(x, n, handle=h), lambda x, n, h: fgemm.rms_norm(x, x[0], handle=h)):
        library = Library()
        monkeypatch.setattr(fgemm, "_lib", library)
        monkeypatch.setattr(fgemm, "_raw_stream", lambda dev: threading.get_ident())
        handle = fgemm.Handle.__new__(fgemm.Handle)
        handle._h, handle.device, handle.lock = None, 0, threading.Lock()
        x, n = torch.zeros(2, 8).half().as_subclass(OnDevice), torch.zeros(2, dtype=torch.int32).as_subclass(OnDevice)
        in_two_threads(lambda: call(x, n, handle))
        assert len(library.seen) == 2 and all(thread == stream for thread, stream in library.seen.items())


def test_threads_get_one_default_handle(monkeypatch):
    class Slow:
        def __init__(self):
            time.sleep(0.2)

    monkeypatch.setattr(fgemm, "Handle", Slow)
    monkeypatch.setattr(fgemm, "_handles", {})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    got = []
    in_two_threads(lambda: got.append(fgemm.default_handle()))
    assert len(got) == 2 and got[0] is got[1]
