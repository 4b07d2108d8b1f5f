"""The operators of a token step against their formulas in 64 bits
(token_reference.py), at the sizes, strides, masks and special values where
they can go wrong."""
import math

import numpy as np
import pytest
import torch

import token_reference as ref
from complexity_matmul_tcgen05_gb300 import fgemm
from parity_util import record

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def within(what, got, want, bound):
    """|got - want| <= bound everywhere; records the closest."""
    off = np.abs(ref.f64(got) - want)
    worst = float(np.max(off / np.maximum(bound, 1e-300), initial=0.0))
    record(what, worst, 1.0)
    assert np.all(off <= bound), (what, worst, np.unravel_index(np.argmax(off / np.maximum(bound, 1e-300)), off.shape))


def padded(t, extra, shift=0):
    """The same values in rows of a wider buffer, `shift` elements in."""
    wide = torch.full((t.shape[0], t.shape[1] + extra + shift), 7, dtype=t.dtype, device=t.device)
    wide[:, shift:shift + t.shape[1]] = t
    return wide[:, shift:shift + t.shape[1]]


# --------------------------------------------------------------------- norm

NORM_SHAPES = [(1, 1), (3, 7), (1, 8), (5, 32), (2, 33), (7, 255), (4, 256), (9, 1000), (6, 1024), (2, 1032), (3, 1537),
               (2, 4096), (1, 5127), (2, 16384), (1, 16392), (1, 20000), (1, 65544), (1, 70001)]


@pytest.mark.parametrize("layout", ["tight", "padded", "shifted"])
@pytest.mark.parametrize("rows,n", NORM_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_norm_forward(rows, n, dtype, layout):
    t, eps = TYPES[dtype], 1e-5
    g = gen(rows * 1000 + n)
    x, res = rand(g, rows, n).to(t), (3 * rand(g, rows, n)).to(t)
    gain = (1 + 0.3 * rand(g, n)).to(t)
    if layout != "tight":
        x, res = (padded(v, 16 - n % 8, 0 if layout == "padded" else 3) for v in (x, res))
    for residual in (None, res):
        y, total, inv = fgemm.rms_norm(x, gain, residual=residual, eps=eps)
        exact = ref.f64(x) if residual is None else ref.f64(x) + ref.f64(res)
        if residual is None:
            assert total is x
        else:  # the sum in fp32, then its rounding
            within("total", total, exact, ref.store(exact, t) + np.abs(exact) * ref.U32)
        tt = ref.f64(total)
        inv64, y64 = ref.norm(tt, ref.f64(gain), eps)
        within("inv_rms", inv, inv64, inv64 * (ref.norm_chain(n) / 2 + 5) * ref.U32)
        within("y", y, y64, ref.store(y64, t) + ref.norm_bound(y64, n))
        for fmt in ("e4m3", "e5m2"):
            q, scales, total2, inv2 = fgemm.rms_norm_mx(x, gain, residual=residual, eps=eps, fmt=fmt)
            assert torch.equal(total2, total) and torch.equal(inv2, inv)
            check_mx(q, scales, y64, ref.norm_bound(y64, n), fmt)


def check_mx(q, scales, y64, err, fmt):
    """Scales and elements are those of some y within err of y64."""
    emax, bits, low, top = ref.F8[fmt]
    e = scales.cpu().numpy().astype(np.int64) - 127
    rel = float(np.max(err / np.maximum(np.abs(y64), 1e-300)))
    for b in range(e.shape[1]):
        most = np.max(np.abs(y64[:, 32 * b:32 * b + 32]), axis=1)
        lo = np.where(most > 0, np.frexp(most * (1 - rel))[1] - 1 - emax, -127).clip(-127, 127)
        hi = np.where(most > 0, np.frexp(most * (1 + rel))[1] - 1 - emax, -127).clip(-127, 127)
        assert np.all((lo <= e[:, b]) & (e[:, b] <= hi))
    scale = np.repeat(np.ldexp(1.0, e), 32, axis=1)[:, :y64.shape[1]]
    v = y64 / scale
    spacing = np.ldexp(1.0, np.maximum(np.frexp(v * (1 + rel))[1] - 1, low) - bits)
    want = np.clip(v, -top, top)
    off = np.abs(ref.f64(q.view(F8[fmt])) - want)
    assert np.all(off <= spacing / 2 + err / scale)
    assert np.all(np.abs(ref.f64(q.view(F8[fmt]))) <= top)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("n", [64, 96, 50])
def test_norm_mx_is_what_matmul_mx_reads(n, fmt):
    g = gen(n)
    x, gain = rand(g, 37, n).bfloat16(), (1 + 0.1 * rand(g, n)).bfloat16()
    q, scales, _, _ = fgemm.rms_norm_mx(x, gain, fmt=fmt)
    v = fgemm.mx_to_bf16(q, scales, fmt)
    assert torch.equal(v.double(), q.view(F8[fmt]).double() *
                       scales.view(torch.float8_e8m0fnu).double().repeat_interleave(32, 1)[:, :n])


def test_norm_mx_blocks_of_zeros_subnormals_and_specials():
    x = torch.ones(1, 192, device=DEV, dtype=torch.bfloat16)
    gain = torch.ones(192, device=DEV, dtype=torch.bfloat16)
    gain[:32] = 0
    gain[32:64] = 2.0 ** -130
    gain[64:96] = 3e38
    gain[70] = float("inf")
    gain[100] = float("nan")
    q, scales, _, inv = fgemm.rms_norm_mx(x, gain, eps=0.0)
    assert inv.item() == 1.0
    v = q.view(F8["e4m3"]).float()[0]
    assert scales[0, 0].item() == 0 and torch.all(v[:32] == 0)
    assert scales[0, 1].item() == 0 and torch.all(v[32:64] == 2.0 ** -3)
    assert scales[0, 2].item() == 255 and scales[0, 3].item() == 255  # not finite: the NaN scale
    assert scales[0, 4].item() == 127 - 8 and torch.all(v[128:] == 256)
    gain[70] = 3e38
    q, scales, _, _ = fgemm.rms_norm_mx(x, gain, eps=0.0)
    assert scales[0, 2].item() == 127 + 127 - 8
    big = float(gain[64].double()) / 2.0 ** 119
    assert torch.all(q.view(F8["e4m3"]).float()[0][64:96] == min(448.0, round(big / 32) * 32))


def test_norm_special_rows():
    g = gen(3)
    x = rand(g, 5, 64).bfloat16()
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 6] = float("nan")
    gain = torch.ones(64, device=DEV, dtype=torch.bfloat16)
    y, _, inv = fgemm.rms_norm(x, gain, eps=1e-6)
    assert torch.all(y[1] == 0) and abs(inv[1].item() - 1e3) < 1e3 * 8 * ref.U32
    assert inv[2].item() == 0 and torch.isnan(y[2, 5]) and torch.all(y[2, :5] == 0)
    assert torch.all(torch.isnan(y[3]))
    assert torch.all(torch.isfinite(y[[0, 4]]))
    y0, _, _ = fgemm.rms_norm(x[1:2], gain, eps=0.0)
    assert torch.all(torch.isnan(y0))


def test_norm_in_place_and_out_arguments():
    g = gen(4)
    for n in (256, 100, 70000):
        x, res, gain = rand(g, 3, n).half(), rand(g, 3, n).half(), rand(g, n).half()
        want = fgemm.rms_norm(x, gain, residual=res)
        x2, res2 = x.clone(), res.clone()
        y, total, inv = fgemm.rms_norm(x2, gain, residual=res2, out=x2, total=res2)
        assert y is x2 and total is res2
        for a, b in zip((y, total, inv), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("layout", ["tight", "shifted"])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 7), (5, 64), (700, 33), (400, 1000), (33, 2048), (310, 4096), (9, 8200),
                                    (3, 14336), (2, 16384), (5, 16400), (2, 9001), (1000, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_norm_backward(rows, n, dtype, layout):
    t, eps = TYPES[dtype], 1e-5
    g = gen(rows * 77 + n)
    total, dy, dt = rand(g, rows, n).to(t), (0.2 * rand(g, rows, n)).to(t), (0.1 * rand(g, rows, n)).to(t)
    gain = (1 + 0.3 * rand(g, n)).to(t)
    if layout == "shifted":
        total, dy, dt = (padded(v, 8, 1) for v in (total, dy, dt))
    inv = torch.rsqrt(total.double().square().mean(1) + eps).float()
    ctas = min(rows, 2 * torch.cuda.get_device_properties(0).multi_processor_count)
    for dtotal in (None, dt):
        dx, dgain = fgemm.rms_norm_backward(dy, total, gain, inv, dtotal=dtotal)
        args = [ref.f64(v) for v in (dy, total, gain, inv, dtotal)]
        dx64, dg64 = ref.norm_backward(*args)
        ex, eg = ref.norm_backward_bound(*args, math.ceil(rows / ctas), ctas)
        within("dx", dx, dx64, ref.store(dx64, t) + ex)
        within("dgain", dgain, dg64, eg + np.abs(dg64) * ref.U32)
    # in place of dy, and the same bits again
    again, dgain2 = fgemm.rms_norm_backward(dy, total, gain, inv, dtotal=dt, out=dy)
    assert again is dy and torch.equal(again, dx) and torch.equal(dgain, dgain2)


def test_norm_backward_against_differences():
    """The kernels' own forward, differenced along one direction in fp32-sized steps."""
    g = gen(9)
    rows, n, eps = 4, 512, 1e-3
    x, gain, dy = rand(g, rows, n).half(), (1 + 0.2 * rand(g, n)).half(), rand(g, rows, n).half()
    _, _, inv = fgemm.rms_norm(x, gain, eps=eps)
    dx, dgain = fgemm.rms_norm_backward(dy, x, gain, inv)
    d = torch.sign(rand(g, rows, n)).half() / 16
    hi, lo = (fgemm.rms_norm(x + s * d, gain, eps=eps)[0] for s in (1, -1))
    # steps as taken: x +- d rounds in fp16
    step = ((x + d).double() - (x - d).double())
    slope = float(((hi.double() - lo.double()) * dy.double()).sum())
    # y is off by half a step each side; the third derivative enters with (1/16)^2 of the slope's scale
    noise = 2 * float((dy.double().abs() * hi.double().abs()).sum()) * 2.0 ** -11
    curve = float((dy.double().abs() * step.abs() * inv.double()[:, None]).sum()) / 256
    assert abs(slope - float((dx.double() * step).sum())) < noise + curve
    bump = torch.full_like(gain, 0.0625)
    hi, lo = (fgemm.rms_norm(x, gain + s * bump, eps=eps)[0] for s in (1, -1))
    step = (gain + bump).double() - (gain - bump).double()
    slope = float(((hi.double() - lo.double()) * dy.double()).sum())
    assert abs(slope - float((dgain.double() * step).sum())) < noise


def test_norm_empty():
    for shape in ((0, 64), (0, 0)):
        x = torch.empty(shape, device=DEV, dtype=torch.bfloat16)
        gain = torch.ones(shape[1], device=DEV, dtype=torch.bfloat16)
        assert fgemm.rms_norm(x, gain)[0].shape == shape
        assert fgemm.rms_norm_mx(x, gain)[0].shape == shape
        inv = torch.empty(0, device=DEV)
        dx, dgain = fgemm.rms_norm_backward(x, x, gain, inv)
        assert dx.shape == shape and torch.all(dgain == 0)


# ----------------------------------------------------------------------- w4


def w4_inputs(m, n, k, dtype, group, zeros, seed, scale_spread=0.3):
    t = TYPES[dtype]
    g = gen(seed)
    A = rand(g, m, max(-(-k // 8) * 8, 8)).to(t)[:, :k]
    W = torch.randint(0, 256, (n, max(-(-k // 32) * 16, 16)), generator=g, device=DEV, dtype=torch.uint8)[:, :(k + 1) // 2]
    groups = -(-k // group)
    scales = ((1 + scale_spread * rand(g, n, groups)) / (5 * math.sqrt(max(k, 1)))).to(t)
    z = torch.randint(0, 16, (n, groups), generator=g, device=DEV, dtype=torch.uint8) if zeros else None
    bias = (0.1 * rand(g, n)).to(t)
    return A, W, scales, z, bias


def check_w4(A, W, scales, z, bias, group, epilogue, alpha=1.0):
    C = fgemm.matmul_w4(A, W, scales, zeros=z, group=group, bias=bias, alpha=alpha, epilogue=epilogue)
    want, bound = ref.w4(ref.f64(A), W.cpu().numpy(), ref.f64(scales), None if z is None else z.cpu().numpy(), group,
                         alpha, ref.f64(bias), epilogue, A.dtype)
    within(f"w4 {epilogue}", C, want, bound)
    return C


W4_SHAPES = [(1, 1, 1), (1, 8, 32), (1, 16, 256), (2, 33, 100), (3, 64, 511), (5, 100, 512), (8, 96, 1024), (9, 128, 257),
             (1, 1000, 4096), (16, 200, 2304), (17, 64, 700), (33, 72, 640), (64, 256, 1024), (65, 40, 300),
             (100, 130, 384), (129, 256, 512), (300, 520, 1032), (1, 4096, 33)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", W4_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_w4_sizes(m, n, k, dtype, group, zeros):
    A, W, s, z, bias = w4_inputs(m, n, k, dtype, group, zeros, m * 7 + n + k)
    check_w4(A, W, s, z, None, group, "none")


@pytest.mark.parametrize("epilogue", ["none", "scale_bias", "silu", "swiglu"])
@pytest.mark.parametrize("m,n,k", [(1, 66, 512), (7, 160, 1000), (20, 98, 384), (70, 256, 640), (260, 128, 512)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_w4_epilogues(m, n, k, dtype, epilogue):
    A, W, s, z, bias = w4_inputs(m, n, k, dtype, 64, True, m + n)
    check_w4(A, W, s, z, bias, 64, epilogue, alpha=-1.5)
    check_w4(A, W, s, z, None if epilogue != "scale_bias" else bias, 64, epilogue)


@pytest.mark.parametrize("m", [1, 8, 12, 40, 150])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_w4_every_code_and_zero_point_exactly(m, dtype):
    """A of one-hot rows and power-of-two scales: C is (q - z) s, exactly."""
    k, n, group = 128, 32, 32
    t = TYPES[dtype]
    g = gen(m)
    W = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    z = torch.randint(0, 16, (n, k // group), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.exp2(torch.randint(-3, 3, (n, k // group), generator=g, device=DEV).float()).to(t)
    codes = torch.stack((W & 15, W >> 4), 2).flatten(1)
    for first in range(0, k, m):
        A = torch.zeros(m, k, device=DEV, dtype=t)
        hot = (torch.arange(m, device=DEV) + first) % k
        A[torch.arange(m, device=DEV), hot] = 1
        C = fgemm.matmul_w4(A, W, s, zeros=z, group=group)
        want = ((codes.double() - z.double().repeat_interleave(group, 1)) * s.double().repeat_interleave(group, 1))[:, hot].T
        assert torch.equal(C.double(), want)


@pytest.mark.parametrize("m", [1, 9, 40, 200])
def test_w4_infinities_and_nan_in_a(m):
    A, W, s, z, _ = w4_inputs(m, 48, 300, "bf16", 64, True, 5)
    A = A.clone()
    A = torch.nn.functional.pad(A, (0, 4))[:, :300]
    A[0, 17] = float("inf")
    if m > 2:
        A[2, 5] = float("nan")
        A[m - 1, 299] = -float("inf")
    C = fgemm.matmul_w4(A, W, s, zeros=z, group=64)
    q = torch.stack((W & 15, W >> 4), 2).flatten(1)[:, :300].double()
    at = torch.arange(300, device=DEV) // 64
    Wv = (q - z.double()[:, at]) * s.double()[:, at]
    want = A.double().cpu() @ Wv.T.cpu()
    for i in range(m):
        bad = ~torch.isfinite(want[i])
        got = C[i].double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want[i]))
        assert torch.equal(got[bad & ~torch.isnan(want[i])], want[i][bad & ~torch.isnan(want[i])])
    assert torch.all(torch.isfinite(C[1:2]))


@pytest.mark.parametrize("m", [1, 20, 140])
def test_w4_strided_operands(m):
    A, W, s, z, bias = w4_inputs(m, 80, 512, "f16", 128, True, 6)
    want = fgemm.matmul_w4(A, W, s, zeros=z, group=128, bias=bias, epilogue="scale_bias")
    A2, W2, s2, z2 = padded(A, 24), padded(W, 48), padded(s, 3, 1), padded(z, 5, 1)
    out = padded(torch.zeros(m, 80, device=DEV, dtype=torch.float16), 7, 1)
    got = fgemm.matmul_w4(A2, W2, s2, zeros=z2, group=128, bias=bias, epilogue="scale_bias", out=out)
    assert got is out and torch.equal(out, want)


def test_w4_ends_of_memory_and_repeatability():
    """W's last row ends with the tensor; two calls give the same bits."""
    for m in (1, 30, 140):
        A, _, s, _, _ = w4_inputs(m, 5, 72, "bf16", 32, False, 8)
        flat = torch.randint(0, 256, (4 * 48 + 36,), generator=gen(1), device=DEV, dtype=torch.uint8)
        W = flat.as_strided((5, 36), (48, 1))
        C = check_w4(A, W, s, None, None, 32, "none")
        assert torch.equal(C, fgemm.matmul_w4(A, W, s, group=32))


def test_w4_empty():
    A, W, s, z, bias = w4_inputs(3, 16, 0, "bf16", 128, False, 1)
    C = fgemm.matmul_w4(A, W, s, bias=bias, epilogue="scale_bias")
    assert torch.equal(C, bias.expand(3, 16))
    assert fgemm.matmul_w4(A[:0], W, s).shape == (0, 16)
    assert fgemm.matmul_w4(A, W[:0], s[:0]).shape == (3, 0)


def test_w4_refuses():
    A, W, s, z, _ = w4_inputs(2, 16, 128, "bf16", 128, True, 1)
    for bad in (dict(group=48), dict(epilogue="gelu"), dict(zeros=z[:, :0]), dict(bias=s[0]),
                dict(out=torch.empty(2, 15, device=DEV, dtype=A.dtype))):
        with pytest.raises(fgemm.FgemmError):
            fgemm.matmul_w4(A, W, s, **bad)
    with pytest.raises(fgemm.FgemmError):
        fgemm.matmul_w4(A.float(), W, s)
    with pytest.raises(fgemm.FgemmError):
        fgemm.matmul_w4(A, W, s.half())
    with pytest.raises(fgemm.FgemmError):
        fgemm.matmul_w4(A, W.cpu(), s)
    with pytest.raises(fgemm.FgemmError):
        fgemm.matmul_w4(torch.empty(2, 129, device=DEV, dtype=A.dtype)[:, 1:], W, s)


# ------------------------------------------------------------------- sample


def check_sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    token, prob = fgemm.sample(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    x = ref.f64(logits)
    row = lambda v, i: float(v[i]) if isinstance(v, torch.Tensor) else float(np.float32(v))  # noqa: E731
    for i in range(x.shape[0]):
        want, p, gap = ref.sample_row(x[i], float(u[i]), row(temperature, i), int(row(top_k, i)), row(top_p, i),
                                      row(min_p, i))
        if gap < 1e-10:  # nearer to a border than the sums are exact: either side may be right
            continue
        assert int(token[i]) == want, (i, int(token[i]), want, gap)
        # masses hold 36 bits, the stored probability 24
        assert abs(float(prob[i]) - p) <= p * (2.0 ** -35 + 2 * ref.U32), (i, float(prob[i]), p)
    return token, prob


def settings(g, rows):
    return dict(temperature=0.5 + torch.rand(rows, generator=g, device=DEV),
                top_k=torch.randint(0, 60, (rows,), generator=g, device=DEV, dtype=torch.int32),
                top_p=0.5 + 0.6 * torch.rand(rows, generator=g, device=DEV),
                min_p=0.1 * torch.rand(rows, generator=g, device=DEV) - 0.02)


@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 31), (5, 257), (4, 4096), (9, 4097), (300, 1000), (3, 32000),
                                        (2, 50257), (1, 131072), (2, 200001), (1, 524288)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_sample_sizes(rows, vocab, dtype):
    g = gen(rows + vocab)
    x = (2.5 * rand(g, rows, vocab)).to(TYPES[dtype])
    u = torch.rand(rows, generator=g, device=DEV)
    check_sample(x, u)
    check_sample(x, u, top_k=40, temperature=0.7)
    check_sample(x, u, top_p=0.9)
    check_sample(x, u, min_p=0.05, temperature=1.3)
    check_sample(x, u, temperature=0.0)
    check_sample(x, u, **settings(g, rows))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "two", "narrow", "wide", "near zero", "masked", "one left", "lowest", "steps"])
def test_sample_distributions(kind, dtype):
    t = TYPES[dtype]
    g = gen(11)
    rows, vocab = 24, 9001
    if kind == "equal":
        x = torch.full((rows, vocab), -3.25, device=DEV)
    elif kind == "two":
        x = (rand(g, rows, vocab) > 0.5).float()
    elif kind == "narrow":
        x = 20 + 1e-3 * rand(g, rows, vocab)
    elif kind == "wide":
        x = 300 * rand(g, rows, vocab)
    elif kind == "near zero":
        x = 1e-6 * rand(g, rows, vocab)
    elif kind == "masked":
        x = rand(g, rows, vocab).masked_fill(torch.rand((rows, vocab), generator=g, device=DEV) < 0.9, -math.inf)
    elif kind == "one left":
        x = torch.full((rows, vocab), -math.inf, device=DEV)
        x[torch.arange(rows), torch.arange(rows) * 300 + 5] = -7
    elif kind == "lowest":  # masks of the type's lowest value
        x = rand(g, rows, vocab).masked_fill(torch.rand((rows, vocab), generator=g, device=DEV) < 0.9, torch.finfo(t).min)
        x[3] = torch.finfo(t).min
    else:
        x = torch.floor(4 * rand(g, rows, vocab)) / 4
    x = x.to(t)
    u = torch.rand(rows, generator=g, device=DEV)
    u[0] = 0
    u[1] = 1 - 2.0 ** -24
    u[2] = 1
    for kw in (dict(), dict(top_k=5), dict(top_k=3000), dict(top_p=0.5), dict(top_p=0.999), dict(min_p=0.5),
               dict(top_k=100, top_p=0.7, min_p=0.2), dict(temperature=0.01), dict(temperature=100.0, top_p=0.3),
               dict(temperature=0.01, top_k=7, top_p=0.9)):
        check_sample(x, u, **kw)


def test_sample_rows_with_nothing_left_and_specials():
    inf = math.inf
    x = torch.tensor([[-inf] * 6, [math.nan] * 6, [math.nan, -inf, 2.0, math.nan, -inf, -inf], [0.0, inf, 1.0, inf, 5.0, -inf],
                      [1.0, 1.0, 1.0, 1.0, -0.0, 0.0]], device=DEV)
    u = torch.tensor([0.5, 0.5, 0.99, 0.75, 0.999], device=DEV)
    token, prob = fgemm.sample(x, u)
    assert token.tolist()[:4] == [-1, -1, 2, 3] and token[4] == 5
    assert prob.tolist()[:4] == [0.0, 0.0, 1.0, 0.5]
    token, prob = fgemm.sample(x, u, temperature=0.0)
    assert token.tolist() == [-1, -1, 2, 1, 0]
    # -0 and 0 tie: the lower index is first
    token, _ = fgemm.sample(x[4:, 4:], u[:1], top_k=1)
    assert token.tolist() == [0]


def test_sample_settings_outside_their_ranges_and_odd_u():
    g = gen(12)
    x = rand(g, 6, 300)
    u = torch.tensor([-0.5, 0.0, 1.0, 2.0, math.nan, math.inf], device=DEV)
    token, _ = fgemm.sample(x, u)
    assert token.tolist() == [0, 0, 299, 299, 0, 299]
    u = torch.rand(6, generator=g, device=DEV)
    plain = fgemm.sample(x, u)[0]
    for kw in (dict(top_k=-3), dict(top_k=1000), dict(top_p=1.5), dict(top_p=math.nan), dict(min_p=-1.0),
               dict(min_p=math.nan)):
        assert torch.equal(fgemm.sample(x, u, **kw)[0], plain), kw
    first = x.argmax(1).int()
    for kw in (dict(top_k=1), dict(top_p=0.0), dict(top_p=-1.0), dict(min_p=1.5), dict(temperature=-1.0),
               dict(temperature=math.nan), dict(temperature=1e-38)):
        assert torch.equal(fgemm.sample(x, u, **kw)[0], first), kw


def test_sample_strides_and_frequencies():
    g = gen(13)
    x = rand(g, 40, 700)
    u = torch.rand(40, generator=g, device=DEV)
    for t in (torch.float32, torch.float16):
        y = x.to(t)
        assert torch.equal(fgemm.sample(padded(y, 9, 1), u, top_k=20)[0], fgemm.sample(y, u, top_k=20)[0])
    # u on a grid: every token is taken in proportion to its probability, to one grid step
    n = 4096
    row = rand(g, 1, 50)
    grid = (torch.arange(n, device=DEV) + 0.5) / n
    token, _ = fgemm.sample(row.expand(n, 50).contiguous(), grid)
    share = torch.bincount(token.long(), minlength=50).double() / n
    assert torch.all((share - torch.softmax(row.double()[0], 0)).abs() <= 1.0 / n + 1e-9)


def test_sample_empty_and_refusals():
    token, prob = fgemm.sample(torch.empty(0, 10, device=DEV), torch.empty(0, device=DEV))
    assert token.shape == (0,)
    token, prob = fgemm.sample(torch.empty(3, 0, device=DEV), torch.rand(3, device=DEV))
    assert token.tolist() == [-1, -1, -1]
    x, u = torch.zeros(2, 10, device=DEV), torch.rand(2, device=DEV)
    for args, kw in (((x.double(), u), {}), ((x, u[:1]), {}), ((x[0], u), {}), ((x.cpu(), u), {}), ((x, u.half()), {}),
                     ((x, u), dict(top_k=torch.zeros(2, device=DEV))), ((x, u), dict(temperature=u[:1]))):
        with pytest.raises(fgemm.FgemmError):
            fgemm.sample(*args, **kw)


# ------------------------------------------------------ streams and graphs


def token_step(x, res, gain, A, W, s, u):
    y, total, inv = fgemm.rms_norm(x, gain, residual=res)
    q, sc, _, _ = fgemm.rms_norm_mx(x, gain)
    logits = fgemm.matmul_w4(y, W, s, group=64)
    many = fgemm.matmul_w4(A, W, s, group=64)
    token, prob = fgemm.sample(logits, u, top_k=10, top_p=0.9)
    dx, dgain = fgemm.rms_norm_backward(y, total, gain, inv, dtotal=x)
    return y, total, inv, q, sc, logits, many, token, prob, dx, dgain


@pytest.mark.parametrize("how", ["stream", "graph"])
def test_streams_and_graphs(how):
    g = gen(21)
    x, res = rand(g, 3, 512).bfloat16(), rand(g, 3, 512).bfloat16()
    gain = (1 + 0.1 * rand(g, 512)).bfloat16()
    A, W, s, _, _ = w4_inputs(150, 1000, 512, "bf16", 64, False, 3)
    u = torch.rand(3, generator=g, device=DEV)
    args = (x, res, gain, A, W, s, u)
    want = [v.clone() for v in token_step(*args)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    if how == "stream":
        with torch.cuda.stream(side):
            got = token_step(*args)
        side.synchronize()
    else:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = token_step(*args)
        for v in got:
            if v.data_ptr() != x.data_ptr():
                v.zero_()
        graph.replay()
        torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
