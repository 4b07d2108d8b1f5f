"""The operators of a token step at the edges of what their documentation
admits: long K with few rows, ties behind a long top-k, activations and rows
far from 1, infinities, in-place outputs."""
import ctypes
import math

import numpy as np
import pytest
import torch

import token_reference as ref
from complexity_matmul_tcgen05_gb300 import fgemm
from test_token_ops_gpu import DEV, TYPES, check_mx, check_sample, gen, padded, rand, w4_inputs, within

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


@pytest.mark.parametrize("top_k", [(1 << 31) + 7, (1 << 32) + 1, 1 << 40, -(1 << 31) - 1, -(1 << 32) + 1])
def test_sample_top_k_beyond_32_bits(top_k):
    """All of them keep every token: above the vocabulary, or not above 0."""
    g = gen(32)
    x, u = rand(g, 5, 300), torch.rand(5, generator=g, device=DEV)
    want = fgemm.sample(x, u)
    got = fgemm.sample(x, u, top_k=top_k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ----------------------------------------------------------------------- w4


def w4_terms(A, W, scales, zeros, group):
    """(C, magnitude, lost) in 64 bits: the product, the sum of its terms'
    magnitudes |A| |q - z| |s|, and what fp16's range drops of a group's small
    values: 2^-39 of its largest for each term."""
    k = A.shape[1]
    at = np.arange(k) // group
    s = scales[:, at]
    z = np.full_like(s, 8.0) if zeros is None else zeros.astype(np.float64)[:, at]
    q = ref.w4_codes(W, k) - z
    lost = np.zeros((A.shape[0], W.shape[0]))
    for k0 in range(0, k, group):
        most = np.max(np.abs(A[:, k0:k0 + group]), axis=1)
        lost += np.outer(most, np.sum(np.abs(q[:, k0:k0 + group] * s[:, k0:k0 + group]), axis=1))
    return A @ (q * s).T, np.abs(A) @ np.abs(q * s).T, lost * 2.0 ** -39


def w4_close(C, A, W, scales, zeros, group, cols=None):
    """C is the product to what its own terms allow, nothing wider: a product
    step adds 16 terms and the running sum, each cut to 24 bits; then one
    addition a group, and at most 32 over warps, slices and the epilogue."""
    if cols is not None:
        C, W, scales = C[:, cols], W[cols], scales[cols]
        zeros = None if zeros is None else zeros[cols]
    k = A.shape[1]
    want, mag, lost = w4_terms(ref.f64(A), W.cpu().numpy(), ref.f64(scales), None if zeros is None else zeros.cpu().numpy(),
                               group)
    within("w4 terms", C, want, (17 / 16 * group + k / group + 32) * ref.U32 * mag + lost + ref.store(want, A.dtype))


@pytest.mark.parametrize("k", [20736, 22016, 24576, 45056, 180224])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_one_row_of_a_long_k(k, zeros):
    n = 64 if k > 100000 else 8192  # many columns: K is cut only as far as A has to be
    A, W, s, z, _ = w4_inputs(1, n, k, "bf16", 32, zeros, k)
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=32)
    w4_close(C, A, W, s, z, 32, torch.arange(0, n, n // 64, device=DEV))


@pytest.mark.parametrize("m,k,group", [(8, 28672, 32), (8, 33000, 32), (5, 53248, 128), (8, 53248, 128), (7, 40000, 64),
                                       (1, 200000, 32), (2, 140000, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_w4_few_rows_whose_a_is_loaded_in_parts(m, k, group, dtype):
    """K above what eight CTAs keep of A in shared memory."""
    n = 100  # an odd number of tiles, the last of them ragged
    A, W, s, z, bias = w4_inputs(m, n, k, dtype, group, True, m + k)
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=group)
    w4_close(C, A, W, s, z, group)
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=group, bias=bias, epilogue="swiglu")
    want, bound = ref.w4(ref.f64(A), W.cpu().numpy(), ref.f64(s), z.cpu().numpy(), group, 1.0, ref.f64(bias), "swiglu",
                         A.dtype)
    within("w4 swiglu", C, want, bound)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 33, 100), (3, 64, 1023), (8, 96, 4096), (9, 128, 257), (17, 64, 700), (40, 72, 4096),
                                   (65, 40, 300), (150, 136, 2304)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_w4_to_what_its_terms_allow(m, n, k, dtype, group, zeros):
    A, W, s, z, _ = w4_inputs(m, n, k, dtype, group, False, m + n + k)
    if zeros:  # a byte, not four bits
        z = torch.randint(0, 256, s.shape, generator=gen(k), device=DEV, dtype=torch.uint8)
        s = s / 16
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=group)
    w4_close(C, A, W, s, z, group)


@pytest.mark.parametrize("m", [1, 9])
@pytest.mark.parametrize("first,second,third", [(0, 2, 4), (1, 3, 5), (0, 1, 7), (3, 8, 12)])
def test_w4_terms_that_cancel_leave_the_rest(first, second, third, m):
    """L - L + x, all with weights of one step: x comes back whole, as long as
    24 bits hold it beside L."""
    k, x = 64, 1 + 513 / 1024
    for log_l in range(0, 13):
        A = torch.zeros((m, k), device=DEV, dtype=torch.float16)
        A[:, [first, second]] = 2.0 ** log_l
        A[:, third] = x
        q = torch.full((8, k), 8, device=DEV, dtype=torch.uint8)
        q[:, first], q[:, second], q[:, third] = 9, 7, 9
        C = fgemm.matmul_w4(A, q[:, 0::2] | (q[:, 1::2] << 4), torch.ones((8, 1), device=DEV).half(), group=64)
        assert torch.all(C == x), log_l


@pytest.mark.parametrize("m,n,k,group", [(26, 65, 213, 32), (142, 359, 290, 128), (7, 125, 46, 64), (174, 323, 22, 32),
                                         (56, 129, 877, 32), (4, 509, 2266, 64), (35, 261, 3, 64), (278, 120, 45, 32),
                                         (1, 96, 4096, 128), (100, 65, 4096, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_w4_small_terms_beside_large_ones(m, n, k, group, dtype):
    A, W, s, _, _ = w4_inputs(m, n, k, "f16", group, False, m + n)
    hot = torch.rand(A.shape, generator=gen(m), device=DEV) < 0.01
    A = torch.nn.functional.pad(torch.where(hot, A * 64, A / 128), (0, -k % 8)).to(TYPES[dtype])[:, :k]
    C = fgemm.matmul_w4(A, W, s.to(A.dtype), group=group)
    w4_close(C, A, W, s.to(A.dtype), None, group)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 4, 8, 9, 40, 150])
@pytest.mark.parametrize("dtype,small,large", [("bf16", 1.0, 2.0 ** 20), ("bf16", 1.0, 1e30), ("f16", 0.02, 60000.0)])
def test_w4_large_activations_of_codes_at_the_zero_point(m, group, dtype, small, large):
    """A weight of 0 takes nothing of its activation, however large."""
    n, k = 72, 1024
    A, W, s, _, _ = w4_inputs(m, n, k, dtype, group, False, m + group)
    z = torch.randint(0, 16, s.shape, generator=gen(m), device=DEV, dtype=torch.uint8)
    A = (A * small).contiguous()
    # one such activation in a row, in the first half of K; a whole group of them for the largest
    hot = (torch.arange(m, device=DEV) * 131 + 64) % (k // 2)
    width = group if large > 2.0 ** 34 else 1
    q = torch.stack((W & 15, W >> 4), 2).flatten(1)
    for i, h in enumerate(hot.tolist()):
        h = h // width * width
        A[i, h:h + width] = large
        q[:, h:h + width] = z[:, h // group, None]
    W = q[:, 0::2] | (q[:, 1::2] << 4)
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=group)
    w4_close(C, A, W, s, z, group)


@pytest.mark.parametrize("m", [1, 5, 20, 140])
def test_w4_large_finite_rows(m):
    A, W, s, z, _ = w4_inputs(m, 72, 600, "bf16", 64, True, m)
    A = A.contiguous()
    for i in range(0, m, 2):
        A[i] = (A[i].float() * 2.0 ** 122).to(A.dtype)
    s = (s.float() * 2.0 ** -8).to(s.dtype)
    assert torch.all(torch.isfinite(A))
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=64)
    w4_close(C, A, W, s, z, 64)


@pytest.mark.parametrize("m", [1, 5, 20, 140])
def test_w4_large_groups_with_small_scales(m):
    """Sums of a group beyond fp32 whose scale brings them back."""
    n, k, group = 40, 512, 128
    A, W, s, _, _ = w4_inputs(m, n, k, "bf16", group, False, m)
    A = torch.full_like(A, 2.0 ** 127)
    z = torch.full(s.shape, 255, device=DEV, dtype=torch.uint8)
    s = (s.float() * 2.0 ** -15).to(s.dtype)
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=group)
    assert torch.all(torch.isfinite(C))
    w4_close(C, A, W, s, z, group)


@pytest.mark.parametrize("k", [300, 4072])  # one CTA a tile, and slices of K
@pytest.mark.parametrize("m", [1, 3, 9, 200])
def test_w4_infinite_and_nan_scales(m, k):
    n = 48
    A, W, s, z, _ = w4_inputs(m, n, k, "bf16", 64, True, 5)
    A, s = torch.nn.functional.pad(A.abs() + 0.5, (0, -k % 8))[:, :k], s.clone()  # rows of whole 16 bytes
    s[3, 1] = math.inf
    s[17, 4] = -math.inf
    s[40, 2] = math.nan
    z[3, 1] = z[17, 4] = 20  # every weight of the group is infinite, with one sign
    z[20, 0], s[20, 0] = 7, math.inf  # some are 0 times infinity
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=64)
    q = torch.stack((W & 15, W >> 4), 2).flatten(1)[:, :k].double()
    at = torch.arange(k, device=DEV) // 64
    want = (A.double().cpu() @ ((q - z.double()[:, at]) * s.double()[:, at]).T.cpu())
    got = C.double().cpu()
    bad = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and bool(bad[:, [3, 17, 20, 40]].all())
    assert torch.equal(got[bad & ~torch.isnan(want)], want[bad & ~torch.isnan(want)])
    ok = torch.tensor([j for j in range(n) if j not in (3, 17, 20, 40)], device=DEV)
    w4_close(C, A, W, s, z, 64, ok)
    # a gate with such a column spoils its own output and no other
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=64, epilogue="swiglu")
    lost = torch.tensor([j in (3, 17, 20, 16) for j in range(n // 2)], device=DEV)
    assert torch.all(torch.isfinite(C[:, ~lost]))
    assert torch.all(torch.isnan(C[:, [20, 16]]))


@pytest.mark.parametrize("kind", ["nan", "inf", "large"])
@pytest.mark.parametrize("m", [8, 256])
def test_w4_time_of_rows_that_are_not_finite(m, kind):
    """Rows of a batch that diverged, or that pad it, take what others take."""
    n = k = 4096
    A, W, s, _, _ = w4_inputs(m, n, k, "bf16", 128, False, m)
    B = A.clone()
    if kind == "nan":
        B[:, 1::7] = math.nan
    elif kind == "inf":
        B[:, -1] = math.inf
    else:
        B = (B.float() * 2.0 ** 122).to(B.dtype)

    def us(X):
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(5):
                fgemm.matmul_w4(X, W, s)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 200)
        return sorted(times)[2]

    us(A)
    assert us(B) < 4 * us(A)


# --------------------------------------------------------------------- norm

FAR = [3e38, 1e20, 1e18, 1e-18, 1e-25, 1e-38, 2.0 ** -130]


@pytest.mark.parametrize("layout", ["tight", "shifted", "odd"])
@pytest.mark.parametrize("n", [7, 64, 1000, 4096, 16392, 70000])
def test_norm_of_rows_far_from_one(n, layout):
    """bf16 holds values whose squares fp32 does not."""
    t = torch.bfloat16
    g = gen(n)
    rows = len(FAR)
    scale = torch.tensor(FAR, device=DEV, dtype=torch.float64)[:, None]
    x = (torch.rand((rows, n), generator=g, device=DEV, dtype=torch.float64) * 2 - 1)
    x[:, 0] = 1
    x = (x * scale).to(t)
    gain = (1 + 0.3 * rand(g, n)).to(t)
    assert torch.all(torch.isfinite(x))
    if layout == "shifted":
        x = padded(x, 16 - n % 8, 3)
    elif layout == "odd":
        x = padded(x, 1 if n % 2 == 0 else 2, 1)
    zero = torch.zeros_like(x)
    for eps in (0.0, 1e-6):
        inv64, y64 = ref.norm(ref.f64(x), ref.f64(gain), float(np.float32(eps)))
        for residual in (None, zero):
            y, total, inv = fgemm.rms_norm(x, gain, residual=residual, eps=eps)
            assert torch.equal(total, x)
            with np.errstate(over="ignore"):
                want = torch.from_numpy(inv64).float()
            fits = torch.isfinite(want)
            within("inv_rms", inv.cpu()[fits], inv64[fits.numpy()],
                   (inv64 * (ref.norm_chain(n) / 2 + 6) * ref.U32 + 2.0 ** -149)[fits.numpy()])
            assert torch.all(torch.isinf(inv.cpu()[~fits]))
            # (2^-140: products of fp32 numbers near its end)
            within("y", y, y64, ref.store(y64, t) + ref.norm_bound(y64, n) + 2.0 ** -140)
            for fmt in ("e4m3", "e5m2"):
                q, scales, total2, inv2 = fgemm.rms_norm_mx(x, gain, residual=residual, eps=eps, fmt=fmt)
                assert torch.equal(total2, total) and torch.equal(inv2, inv)
                if eps == 0.0:
                    check_mx(q, scales, y64, ref.norm_bound(y64, n), fmt)


@pytest.mark.parametrize("layout", ["tight", "shifted"])
@pytest.mark.parametrize("n", [64, 1000, 4096, 8200, 16400])
def test_norm_backward_of_rows_far_from_one(n, layout):
    t = torch.bfloat16
    g = gen(n + 1)
    far = [1e37, 1e20, 1.0, 1e-18, 1e-25, 1e-36]
    rows = len(far)
    scale = torch.tensor(far, device=DEV, dtype=torch.float64)[:, None]
    total = (rand(g, rows, n).double() * scale).to(t)
    dy, gain = (0.2 * rand(g, rows, n)).to(t), (1 + 0.3 * rand(g, n)).to(t)
    dy[-1] *= 2.0 ** -30  # dx is dy / rms: within bf16
    dt = (0.1 * rand(g, rows, n).double() / scale.clamp(1e-30, 1e30)).to(t)
    inv = (1 / total.double().square().mean(1).sqrt()).float()
    if layout == "shifted":
        total, dy, dt = (padded(v, 8, 1) for v in (total, dy, dt))
    for dtotal in (None, dt):
        dx, dgain = fgemm.rms_norm_backward(dy, total, gain, inv, dtotal=dtotal)
        args = [ref.f64(v) for v in (dy, total, gain, inv, dtotal)]
        dx64, dg64 = ref.norm_backward(*args)
        ex, eg = ref.norm_backward_bound(*args, 1, rows)
        within("dx", dx, dx64, ref.store(dx64, t) + ex + 2.0 ** -140)
        within("dgain", dgain, dg64, eg + np.abs(dg64) * ref.U32)


@pytest.mark.parametrize("rows,n,layout", [(3, 256, "tight"), (1, 100, "tight"), (3, 100, "shifted"), (2, 70000, "tight")])
def test_norm_in_place_keeps_the_total(rows, n, layout):
    """y over x: the total that comes back, which the backward pass takes, is x as it was."""
    g = gen(n)
    x, gain = rand(g, rows, n).bfloat16(), (1 + 0.3 * rand(g, n)).bfloat16()
    if layout == "shifted":
        x = padded(x, 8, 1)
    want = fgemm.rms_norm(x, gain)
    before = x.clone()
    y, total, inv = fgemm.rms_norm(x, gain, out=x)
    assert y is x and torch.equal(y, want[0]) and torch.equal(inv, want[2])
    assert torch.equal(total, before)


def test_norm_refuses_one_memory_for_both_outputs():
    x, gain = torch.randn(3, 64, device=DEV).half(), torch.ones(64, device=DEV).half()
    for kw in (dict(out=x, total=x), dict(out=x, total=x, residual=x.clone())):
        with pytest.raises(fgemm.FgemmError):
            fgemm.rms_norm(x, gain, **kw)


# ------------------------------------------------------------------- errors


def test_an_error_is_reported_once():
    """A call that failed leaves nothing behind for the next one to report."""
    x, gain = torch.randn(3, 64, device=DEV).half(), torch.ones(64, device=DEV).half()
    want = fgemm.rms_norm(x, gain)[0]
    torch.cuda.synchronize()
    rt = ctypes.CDLL("libcudart.so.13")
    h, L = fgemm.default_handle(), fgemm.lib()
    side = torch.cuda.Stream()
    stream, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(stream, 2) == 0  # relaxed
    L.fgemm_set_stream(h._h, stream)
    failed = L.fgemm_get_error(h._h)  # it would wait for a stream that is being captured
    rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
    rt.cudaGetLastError()  # torch's own copy of the runtime
    assert failed == fgemm.ERR_CUDA
    assert torch.equal(fgemm.rms_norm(x, gain)[0], want)
    assert h.get_error() == fgemm.OK
