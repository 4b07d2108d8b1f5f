"""Python binding of the fgemm C ABI (include/fgemm.h).

Argument marshalling only: every step of the product runs in the CUDA
library ``_build/libfgemm.so``.  If that library is missing, every call
raises -- there is no fallback of any kind.

``matmul`` takes torch CUDA tensors (fp16 or bf16, row-major, unit column
stride) and enqueues on torch's current stream.  Given CPU tensors it copies
them to the current device first and returns a CPU result (the end-to-end
path: host -> device -> kernel -> host).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfgemm.so")

OK, ERR_INVALID_ARG, ERR_ALIGNMENT, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_NO_DEVICE, \
    ERR_CALIBRATION = range(8)
F16, BF16 = 0, 1
ALGOS = {"auto": 0, "classical": 1, "strassen1": 2, "strassen2": 3, "winograd1": 4}
ALGO_NAMES = {v: k for k, v in ALGOS.items()}
EPILOGUES = {"none": 0, "scale_bias": 1, "silu": 2, "swiglu": 3}


class Rms(ctypes.Structure):
    _fields_ = [("sumsq_out", ctypes.c_void_p), ("sumsq_in", ctypes.c_void_p),
                ("sumsq_parts", ctypes.c_int32), ("norm_width", ctypes.c_int64),
                ("eps", ctypes.c_float)]


class Sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("temperatures", ctypes.c_void_p), ("top_ks", ctypes.c_void_p),
                ("top_ps", ctypes.c_void_p), ("min_ps", ctypes.c_void_p)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("k_page", ctypes.c_int64), ("k_token", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_page", ctypes.c_int64), ("v_token", ctypes.c_int64),
                ("v_head", ctypes.c_int64)]


class FgemmError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(message)


class Epilogue(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("alpha", ctypes.c_float), ("bias", ctypes.c_void_p)]


class DeviceModel(ctypes.Structure):
    _fields_ = [("num_sms", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("peak_tflops", ctypes.c_double), ("hbm_gbs", ctypes.c_double),
                ("eff_classical", ctypes.c_double * 3),
                ("eff_pair", ctypes.c_double * 2),
                ("eff_strassen", (ctypes.c_double * 2) * 2),
                ("eff_strassen_pair", ctypes.c_double * 2),
                ("launch_us", ctypes.c_double), ("tile_fill_us", ctypes.c_double),
                ("l2_bytes", ctypes.c_double), ("l2_gbs", ctypes.c_double),
                ("split_fix_us", ctypes.c_double),
                ("eff_winograd", ctypes.c_double * 2),
                ("eff_small_m", ctypes.c_double * 3), ("hbm_stream_eff", ctypes.c_double),
                ("small_m_stream_eff", ctypes.c_double), ("small_m_fix_us", ctypes.c_double),
                ("small_m_aligned_eff", ctypes.c_double),
                ("form_in_kernel_eff", ctypes.c_double),
                ("form_in_kernel_drag", ctypes.c_double),
                ("lcma_margin", ctypes.c_double),
                ("dram_miss_slope", ctypes.c_double),
                ("dram_exposed", ctypes.c_double),
                ("eff_strassen2_pair", ctypes.c_double * 2),
                ("fold2_unit_us", ctypes.c_double)]


_lib = None
_lib_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise FgemmError(ERR_CUDA, f"fgemm CUDA library not built: {LIB_PATH} is missing "
                                       "(run python -m complexity_matmul_tcgen05_gb300.build)")
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, vp, st = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int
        epi_p = ctypes.POINTER(Epilogue)
        model_p = ctypes.POINTER(DeviceModel)
        L.fgemm_create.argtypes = [ctypes.POINTER(vp)]
        L.fgemm_destroy.argtypes = [vp]
        L.fgemm_set_stream.argtypes = [vp, vp]
        mm = [vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, st, epi_p, st]
        L.fgemm_matmul.argtypes = mm
        L.fgemm_matmul_ex.argtypes = mm + [i32, i32]
        L.fgemm_matmul_rms.argtypes = mm + [i32, i32, ctypes.POINTER(Rms)]
        L.fgemm_matmul_mx.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, i32, vp, i64, vp, i64,
                                      i32, vp, i64, epi_p, st, i32, i32]
        L.fgemm_mx_to_bf16.argtypes = [vp, i64, i64, vp, i64, vp, i64, i32, i32, vp, i64]
        f32, size = ctypes.c_float, ctypes.c_size_t
        norm = [vp, i64, i64, vp, i64, vp, i64, vp, f32, st, vp, i64]
        L.fgemm_rms_norm.argtypes = norm + [vp, i64, vp]
        L.fgemm_rms_norm_mx.argtypes = norm + [i32, vp, i64, vp, i64, vp]
        L.fgemm_rms_norm_backward.argtypes = [vp, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, st, vp, i64, vp, vp,
                                              size]
        L.fgemm_rms_norm_backward_workspace.argtypes = [vp, i64, i64]
        L.fgemm_rms_norm_backward_workspace.restype = size
        L.fgemm_matmul_w4.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, i64, st, epi_p,
                                      vp, size]
        L.fgemm_matmul_w4_workspace.argtypes = [i64, i64, i32]
        L.fgemm_matmul_w4_workspace.restype = size
        L.fgemm_sample.argtypes = [vp, i64, i64, vp, i64, i32, vp, ctypes.POINTER(Sampling), vp, vp]
        heads = [vp, i64, i64]
        cache_p = ctypes.POINTER(KvCache)
        L.fgemm_rotary_cache.argtypes = [vp, i64, i32, i32, i32] + 3 * heads + [vp, vp, vp, i32, i32, st] + heads + \
            [cache_p]
        L.fgemm_attention_paged_workspace.argtypes = [vp, i64, i32, i32, i32]
        L.fgemm_attention_paged_workspace.restype = size
        L.fgemm_attention_paged.argtypes = [vp, i64, i32, i32, i32] + heads + [cache_p, vp, i64, i64, vp, f32, i32,
                                                                               st] + heads + [vp, vp, size]
        L.fgemm_attention.argtypes = [vp, i64, i64, i64, i32, i32, i32] + 3 * heads + [vp, vp, i32, i32, f32, st] + \
            heads + [vp]
        L.fgemm_logprobs.argtypes = [vp, i64, i64, vp, i64, i32, vp, i32, vp, vp, vp, vp]
        L.fgemm_plan.argtypes = [vp, i64, i64, i64, st, epi_p, ctypes.POINTER(st),
                                 ctypes.POINTER(i32), ctypes.POINTER(i32),
                                 ctypes.POINTER(ctypes.c_double)]
        L.fgemm_plan_ex.argtypes = [vp, i64, i64, i64, st, epi_p, st, i32, i32, ctypes.POINTER(st),
                                    ctypes.POINTER(i32), ctypes.POINTER(i32),
                                    ctypes.POINTER(ctypes.c_double)]
        L.fgemm_get_error.argtypes = [vp]
        L.fgemm_matmul_host.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, st, epi_p, st, i32, i32]
        L.fgemm_matmul_host_ex.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, st, epi_p, st, i32,
                                           i32, i32]
        L.fgemm_call_launches.argtypes = [vp, i64, i64, i64, epi_p, st, i32, i32, ctypes.POINTER(i32)]
        L.fgemm_selftest_wait_timeout.argtypes = [vp, i32]
        L.fgemm_calibrate.argtypes = [vp, ctypes.c_char_p]
        L.fgemm_calibrate_ex.argtypes = [vp, i64, ctypes.c_char_p]
        L.fgemm_model_load_json.argtypes = [ctypes.c_char_p, model_p]
        L.fgemm_model_save_json.argtypes = [model_p, ctypes.c_char_p]
        L.fgemm_status_string.argtypes = [st]
        L.fgemm_status_string.restype = ctypes.c_char_p
        L.fgemm_last_message.argtypes = [vp]
        L.fgemm_last_message.restype = ctypes.c_char_p
        L.fgemm_validate.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, st, epi_p, st, i32,
                                     i32]
        L.fgemm_model_default.argtypes = [model_p, i32, ctypes.c_double, ctypes.c_double]
        L.fgemm_model_default.restype = None
        L.fgemm_model_tiles.argtypes = [i64, i64, i32, i32]
        L.fgemm_model_tiles.restype = i64
        L.fgemm_model_waves.argtypes = [i64, i32, ctypes.POINTER(ctypes.c_double)]
        L.fgemm_model_waves.restype = i64
        L.fgemm_model_tiled_reads.argtypes = [i64, i64, i64, i32, i32]
        L.fgemm_model_tiled_reads.restype = ctypes.c_double
        L.fgemm_model_roofline.argtypes = [ctypes.c_double] * 4
        L.fgemm_model_roofline.restype = ctypes.c_double
        L.fgemm_model_predict.argtypes = [model_p, i64, i64, i64, i32, st, i32, i32,
                                          ctypes.POINTER(ctypes.c_double)]
        L.fgemm_model_plan.argtypes = [model_p, i64, i64, i64, i32, ctypes.POINTER(st),
                                       ctypes.POINTER(i32), ctypes.POINTER(i32),
                                       ctypes.POINTER(ctypes.c_double)]
        L.fgemm_strassen_matmul_static.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, st,
                                                   epi_p, i32, i32, vp]
        L.fgemm_strassen_static_get_error.argtypes = [vp]
        L.fgemm_strassen_static_selftest_timeout.argtypes = [i32, vp]
        L.fgemm_model_split_tail.argtypes = [model_p, i64, i32, i32, i32, i32, ctypes.POINTER(i32)]
        L.fgemm_model_split_tail.restype = i32
        L.fgemm_split_work_item.argtypes = [i64, i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32)]
        L.fgemm_split_work_item.restype = i32
        L.fgemm_set_split_mode.argtypes = [vp, i32]
        L.fgemm_set_lcma_formation.argtypes = [vp, i32]
        L.fgemm_stream_k_work_item.argtypes = [i64, i32, i32, i32, i32, ctypes.POINTER(i64)]
        L.fgemm_stream_k_work_item.restype = i32
        L.fgemm_small_m_grid.argtypes = [i64, i32, i32, ctypes.POINTER(i32)]
        L.fgemm_small_m_grid.restype = i32
        L.fgemm_lcma_pair_clusters.argtypes = [i64, i32, i32]
        L.fgemm_lcma_pair_clusters.restype = i64
        L.fgemm_get_device_model.argtypes = [vp, model_p]
        L.fgemm_set_device_model.argtypes = [vp, model_p]
        for name in ("fgemm_create", "fgemm_destroy", "fgemm_set_stream", "fgemm_matmul",
                     "fgemm_matmul_ex", "fgemm_plan", "fgemm_plan_ex", "fgemm_get_error", "fgemm_calibrate",
                     "fgemm_calibrate_ex", "fgemm_model_load_json", "fgemm_model_save_json",
                     "fgemm_validate", "fgemm_model_predict", "fgemm_model_plan",
                     "fgemm_get_device_model", "fgemm_set_device_model",
                     "fgemm_strassen_matmul_static", "fgemm_selftest_wait_timeout",
                     "fgemm_set_split_mode", "fgemm_set_lcma_formation", "fgemm_call_launches", "fgemm_matmul_host", "fgemm_matmul_host_ex", "fgemm_matmul_rms", "fgemm_matmul_mx",
                     "fgemm_mx_to_bf16", "fgemm_strassen_static_get_error",
                     "fgemm_strassen_static_selftest_timeout", "fgemm_rms_norm", "fgemm_rms_norm_mx",
                     "fgemm_rms_norm_backward", "fgemm_matmul_w4", "fgemm_sample", "fgemm_rotary_cache",
                     "fgemm_attention_paged", "fgemm_attention", "fgemm_logprobs"):
            getattr(L, name).restype = st
        _lib = L
        return L


SPLIT_MODES = {"off": 0, "auto": 1, "force": 2}
FORMATION_MODES = {"auto": 0, "prepass": 1, "in_kernel": 2}


def split_work_items(tiles: int, split_tiles: int, split_pieces: int, clusters: int,
                     k_blocks: int, cluster: int):
    """The work list of one pair in the K-split schedule, as (unit, k0, k1,
    piece, npieces) tuples (host-side copy of what the kernel runs)."""
    out = (ctypes.c_int32 * 5)()
    items = []
    n = 0
    while lib().fgemm_split_work_item(tiles, split_tiles, split_pieces, clusters, k_blocks,
                                      cluster, n, out):
        items.append(tuple(out))
        n += 1
    return items


def stream_k_work_items(tiles: int, k_blocks: int, ctas: int, cta: int):
    """The work list of one CTA of the small-M kernel, as (unit, k0, k1,
    piece, npieces, slot) tuples (host-side copy of what the kernel runs)."""
    out = (ctypes.c_int64 * 6)()
    items = []
    n = 0
    while lib().fgemm_stream_k_work_item(tiles, k_blocks, ctas, cta, n, out):
        items.append(tuple(out))
        n += 1
    return items


def small_m_grid(tiles: int, k_blocks: int, num_sms: int):
    """(CTA count, phases) of the small-M kernel's grid (fgemm_small_m_grid)."""
    ph = ctypes.c_int32()
    return lib().fgemm_small_m_grid(tiles, k_blocks, num_sms, ctypes.byref(ph)), ph.value


def status_string(status: int) -> str:
    return lib().fgemm_status_string(status).decode()


def _check(status: int, handle_ptr=None):
    if status != OK:
        msg = lib().fgemm_last_message(handle_ptr).decode()
        raise FgemmError(status, f"{status_string(status)}: {msg}")


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float16:
        return F16
    if t == torch.bfloat16:
        return BF16
    raise FgemmError(ERR_INVALID_ARG, f"fgemm supports float16 and bfloat16, not {t}")


def make_epilogue(kind: str = "none", alpha: float = 1.0, bias_ptr: int | None = None) -> Epilogue:
    return Epilogue(EPILOGUES[kind], float(alpha), bias_ptr)


def validate(M, N, K, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, dtype: int, epilogue: Epilogue | None,
             algo: str = "auto", tile_n: int = 0, tile_m: int = 0) -> int:
    """Host-only argument check (no device): the status fgemm_matmul_ex would return."""
    return lib().fgemm_validate(M, N, K, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, dtype,
                                ctypes.byref(epilogue) if epilogue is not None else None,
                                ALGOS[algo], tile_m, tile_n)


class Handle:
    """An fgemm handle on the current CUDA device.

    The C library wants a handle used by one host thread at a time: the functions of this
    module hold `lock` from setting their thread's current stream to the end of the C
    call, so threads may share one (the default handle).  A product's workspace is the
    handle's, though: products on two streams need a handle each, as do threads that
    call the methods."""

    def __init__(self):
        self.lock = threading.Lock()
        h = ctypes.c_void_p()
        _check(lib().fgemm_create(ctypes.byref(h)))
        self._h = h
        self.device = torch.cuda.current_device()

    @property
    def ptr(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().fgemm_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):  # pragma: no cover - interpreter teardown order
        try:
            self.close()
        except Exception:
            pass

    def set_stream(self, stream_ptr: int):
        _check(lib().fgemm_set_stream(self._h, ctypes.c_void_p(stream_ptr)), self._h)

    def set_split_mode(self, mode):
        """K split of the last wave of CTA-pair tiles: "off" (0), "auto" (1,
        the default) or "force" (2, whenever possible)."""
        code = SPLIT_MODES[mode] if isinstance(mode, str) else int(mode)
        _check(lib().fgemm_set_split_mode(self._h, code), self._h)

    def set_lcma_formation(self, mode):
        """Where one-level Strassen-like launches on CTA pairs form their
        summed operands: "auto" (0, the default), "prepass" (1, a separate
        launch) or "in_kernel" (2, inside the product kernel while the
        scheme's leading products that read only blocks of A and B run)."""
        code = FORMATION_MODES[mode] if isinstance(mode, str) else int(mode)
        _check(lib().fgemm_set_lcma_formation(self._h, code), self._h)

    def matmul_raw(self, M, N, K, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, dtype: int,
                   epilogue: Epilogue | None = None, algo: str = "auto", tile_n: int = 0,
                   tile_m: int = 0) -> int:
        """Direct C-ABI call on raw device pointers; returns the status."""
        return lib().fgemm_matmul_ex(self._h, M, N, K, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, dtype,
                                     ctypes.byref(epilogue) if epilogue is not None else None,
                                     ALGOS[algo], tile_m, tile_n)

    def matmul_rms_raw(self, M, N, K, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, dtype: int,
                       epilogue: Epilogue | None, algo: str, tile_n: int, tile_m: int,
                       rms: Rms) -> int:
        """fgemm_matmul_rms on raw device pointers; returns the status."""
        return lib().fgemm_matmul_rms(self._h, M, N, K, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, dtype,
                                      ctypes.byref(epilogue) if epilogue is not None else None,
                                      ALGOS[algo], tile_m, tile_n, ctypes.byref(rms))

    def plan(self, M, N, K, dtype: int = BF16, epilogue: Epilogue | None = None,
             algo: str = "auto", tile_m: int = 0, tile_n: int = 0):
        """(algorithm, tile_m, tile_n, predicted us) of the model's choice,
        restricted to a form / tile when those are given."""
        a = ctypes.c_int()
        tm = ctypes.c_int32()
        tn = ctypes.c_int32()
        us = ctypes.c_double()
        _check(lib().fgemm_plan_ex(self._h, M, N, K, dtype,
                                   ctypes.byref(epilogue) if epilogue is not None else None,
                                   ALGOS[algo], tile_m, tile_n, ctypes.byref(a), ctypes.byref(tm),
                                   ctypes.byref(tn), ctypes.byref(us)), self._h)
        return ALGO_NAMES[a.value], tm.value, tn.value, us.value

    def call_launches(self, M, N, K, epilogue: Epilogue | None = None, algo: str = "auto",
                      tile_m: int = 0, tile_n: int = 0) -> int:
        """Kernels of this library one matmul call with these arguments
        launches on this handle (host only)."""
        n = ctypes.c_int32()
        _check(lib().fgemm_call_launches(self._h, M, N, K,
                                         ctypes.byref(epilogue) if epilogue is not None else None,
                                         ALGOS[algo], tile_m, tile_n, ctypes.byref(n)), self._h)
        return n.value

    def get_error(self) -> int:
        return lib().fgemm_get_error(self._h)

    def last_message(self) -> str:
        return lib().fgemm_last_message(self._h).decode()

    def calibrate(self, json_path: str | None = None, n: int = 8192):
        _check(lib().fgemm_calibrate_ex(self._h, n, json_path.encode() if json_path else None),
               self._h)

    def device_model(self) -> DeviceModel:
        m = DeviceModel()
        _check(lib().fgemm_get_device_model(self._h, ctypes.byref(m)), self._h)
        return m

    def set_device_model(self, m: DeviceModel):
        _check(lib().fgemm_set_device_model(self._h, ctypes.byref(m)), self._h)


_handles: dict[int, Handle] = {}
_handles_lock = threading.Lock()


def default_handle() -> Handle:
    dev = torch.cuda.current_device()
    h = _handles.get(dev)
    if h is None:
        with _handles_lock:  # one for all threads
            h = _handles.get(dev)
            if h is None:
                h = Handle()
                _handles[dev] = h
    return h


def _check_matrix(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise FgemmError(ERR_INVALID_ARG, f"{name} must be 2-D")
    if t.size(1) > 1 and t.stride(1) != 1:
        raise FgemmError(ERR_INVALID_ARG, f"{name} must be row-major with unit column stride")


def matmul(A: torch.Tensor, B: torch.Tensor, *, out: torch.Tensor | None = None,
           epilogue: str = "none", alpha: float = 1.0, bias: torch.Tensor | None = None,
           algo: str = "auto", tile_n: int = 0, tile_m: int = 0,
           handle: Handle | None = None, sumsq_out: torch.Tensor | None = None,
           sumsq_in: torch.Tensor | None = None, norm_width: int = 0,
           rms_eps: float = 1e-6, blocking: bool = True) -> torch.Tensor:
    """C = epi(alpha * A @ B + bias) through fgemm_matmul_ex.

    A is M x K, B is K x N (row-major), bias has N entries; for
    epilogue="swiglu" the output is M x N/2 (gate | up halves of B's columns).

    RMSNorm statistics (fgemm_matmul_rms): ``sumsq_out`` (fp32, shape
    [ceil(N_out/64), M]) receives each row's sums of squares of the stored
    outputs per 64-column block; ``sumsq_in`` (fp32 [parts, M], from an earlier
    call) scales accumulator row i by 1/sqrt(sum / norm_width + rms_eps).

    A and B on the host (CPU tensors, pinned for overlapped copies): the
    product goes through fgemm_matmul_host and ``out`` (or the returned
    tensor) is on the host.  With ``blocking=False`` the call returns once it
    is enqueued (fgemm_matmul_host_ex with FGEMM_HOST_OVERLAP: its uploads may
    run under the previous host call's products); C is written once the
    current CUDA stream has reached the call, and the inputs must not be
    written by other work still pending on that stream.
    """
    if A.device.type == "cpu" and B.device.type == "cpu":
        return _matmul_host(A, B, out, epilogue, alpha, bias, algo, tile_n, tile_m, handle, blocking)
    _check_matrix(A, "A")
    _check_matrix(B, "B")
    if not (A.is_cuda and B.is_cuda):
        raise FgemmError(ERR_INVALID_ARG, "A and B must both be CUDA tensors (or both CPU)")
    if A.dtype != B.dtype:
        raise FgemmError(ERR_INVALID_ARG, "A and B must have the same dtype")
    dt = _dtype_code(A.dtype)
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise FgemmError(ERR_INVALID_ARG, f"inner dimensions differ: {K} vs {K2}")
    n_out = N // 2 if epilogue == "swiglu" else N
    if out is None:
        out = torch.empty((M, n_out), dtype=A.dtype, device=A.device)
    else:
        _check_matrix(out, "out")
        if out.dtype != A.dtype or tuple(out.shape) != (M, n_out):
            raise FgemmError(ERR_INVALID_ARG, "out has the wrong dtype or shape")
    bias_ptr = None
    if bias is not None:
        if bias.dtype != A.dtype or bias.numel() != N or not bias.is_cuda:
            raise FgemmError(ERR_INVALID_ARG, "bias must be a CUDA vector of N entries, same dtype")
        bias = bias.contiguous()
        bias_ptr = bias.data_ptr()
    h = handle if handle is not None else default_handle()
    stream = torch.cuda.current_stream(A.device).cuda_stream
    epi = make_epilogue(epilogue, alpha, bias_ptr)
    lda = A.stride(0) if M > 1 else max(K, 1)
    ldb = B.stride(0) if K > 1 else max(N, 1)
    ldc = out.stride(0) if M > 1 else max(n_out, 1)
    rms = None
    if sumsq_out is not None or sumsq_in is not None:
        parts = 0
        for t, name in ((sumsq_out, "sumsq_out"), (sumsq_in, "sumsq_in")):
            if t is not None and (t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous()):
                raise FgemmError(ERR_INVALID_ARG, f"{name} must be a contiguous CUDA float32 tensor")
        if sumsq_out is not None and tuple(sumsq_out.shape) != ((n_out + 63) // 64, M):
            raise FgemmError(ERR_INVALID_ARG, "sumsq_out must have shape [ceil(N_out / 64), M]")
        if sumsq_in is not None:
            if sumsq_in.dim() != 2 or sumsq_in.shape[1] != M:
                raise FgemmError(ERR_INVALID_ARG, "sumsq_in must have shape [parts, M]")
            parts = sumsq_in.shape[0]
        rms = Rms(None if sumsq_out is None else sumsq_out.data_ptr(),
                  None if sumsq_in is None else sumsq_in.data_ptr(), parts, int(norm_width),
                  float(rms_eps))
    args = (M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, out.data_ptr(), ldc, dt, epi, algo, tile_n, tile_m)
    with h.lock:
        h.set_stream(stream)
        _check(h.matmul_raw(*args) if rms is None else h.matmul_rms_raw(*args, rms), h.ptr)
    return out


HOST_OVERLAP = 1


def _matmul_host(A, B, out, epilogue, alpha, bias, algo, tile_n, tile_m, handle, blocking=True):
    """Host tensors through fgemm_matmul_host_ex (pipelined copies; they
    overlap when the tensors are pinned); returns once C is written, or
    (blocking=False) once the call is enqueued."""
    for t, name in ((A, "A"), (B, "B")):
        if t.dim() != 2 or t.stride(1) != 1:
            raise FgemmError(ERR_INVALID_ARG, f"{name} must be a 2-D tensor with unit column stride")
    if A.dtype != B.dtype:
        raise FgemmError(ERR_INVALID_ARG, "A and B must have the same dtype")
    dt = _dtype_code(A.dtype)
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise FgemmError(ERR_INVALID_ARG, f"inner dimensions differ: {K} vs {K2}")
    n_out = N // 2 if epilogue == "swiglu" else N
    if out is None:
        out = torch.empty((M, n_out), dtype=A.dtype, pin_memory=A.is_pinned())
    elif (out.device.type != "cpu" or out.dtype != A.dtype or tuple(out.shape) != (M, n_out)
          or out.stride(1) != 1):
        raise FgemmError(ERR_INVALID_ARG, "out must be a host tensor of the right dtype and shape")
    bias_ptr = None
    if bias is not None:
        if bias.device.type != "cpu" or bias.dtype != A.dtype or bias.numel() != N:
            raise FgemmError(ERR_INVALID_ARG, "bias must be a host vector of N entries, same dtype")
        if not blocking and not bias.is_contiguous():
            raise FgemmError(ERR_INVALID_ARG, "a non-blocking call needs a contiguous bias")
        bias = bias.contiguous()
        bias_ptr = bias.data_ptr()
    h = handle if handle is not None else default_handle()
    stream = torch.cuda.current_stream().cuda_stream
    epi = make_epilogue(epilogue, alpha, bias_ptr)
    with h.lock:
        h.set_stream(stream)
        s = lib().fgemm_matmul_host_ex(h.ptr, M, N, K, A.data_ptr(), A.stride(0) if M > 1 else max(K, 1),
                                       B.data_ptr(), B.stride(0) if K > 1 else max(N, 1), out.data_ptr(),
                                       out.stride(0) if M > 1 else max(n_out, 1), dt, ctypes.byref(epi),
                                       ALGOS[algo], tile_m, tile_n, 0 if blocking else HOST_OVERLAP)
        _check(s, h.ptr)
    if blocking:
        torch.cuda.current_stream().synchronize()
        with h.lock:
            h.set_stream(stream)
            _check(h.get_error(), h.ptr)
    return out


FP8_FORMATS = {"e4m3": 0, "e5m2": 1}


def matmul_mx(A: torch.Tensor, scale_a: torch.Tensor, B: torch.Tensor, scale_b: torch.Tensor, *,
              a_format: str = "e4m3", b_format: str = "e4m3", out: torch.Tensor | None = None,
              epilogue: str = "none", alpha: float = 1.0, bias: torch.Tensor | None = None,
              algo: str = "auto", tile_n: int = 0, tile_m: int = 0,
              handle: Handle | None = None) -> torch.Tensor:
    """C = epi(alpha * A @ B + bias) for block-scaled 8-bit A (M x K) and B
    (K x N), given as uint8 (or float8) CUDA tensors, with E8M0 scales
    scale_a (M x ceil(K/32)) and scale_b (ceil(K/32) x N) as uint8; C is bf16."""
    for t, name in ((A, "A"), (B, "B"), (scale_a, "scale_a"), (scale_b, "scale_b")):
        if not t.is_cuda or t.dim() != 2 or t.element_size() != 1 or t.stride(1) != 1:
            raise FgemmError(ERR_INVALID_ARG, f"{name} must be a 2-D CUDA byte tensor with unit column stride")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise FgemmError(ERR_INVALID_ARG, f"inner dimensions differ: {K} vs {K2}")
    kb = (K + 31) // 32
    if tuple(scale_a.shape) != (M, kb) or tuple(scale_b.shape) != (kb, N):
        raise FgemmError(ERR_INVALID_ARG, "scales must be M x ceil(K/32) and ceil(K/32) x N")
    n_out = N // 2 if epilogue == "swiglu" else N
    if out is None:
        out = torch.empty((M, n_out), dtype=torch.bfloat16, device=A.device)
    bias_ptr = None
    if bias is not None:
        if bias.dtype != torch.bfloat16 or bias.numel() != N or not bias.is_cuda:
            raise FgemmError(ERR_INVALID_ARG, "bias must be a CUDA bf16 vector of N entries")
        bias = bias.contiguous()
        bias_ptr = bias.data_ptr()
    h = handle if handle is not None else default_handle()
    stream = torch.cuda.current_stream(A.device).cuda_stream
    epi = make_epilogue(epilogue, alpha, bias_ptr)
    with h.lock:
        h.set_stream(stream)
        s = lib().fgemm_matmul_mx(h.ptr, M, N, K, A.data_ptr(), A.stride(0) if M > 1 else max(K, 1),
                                  scale_a.data_ptr(), scale_a.stride(0) if M > 1 else max(kb, 1),
                                  FP8_FORMATS[a_format], B.data_ptr(), B.stride(0) if K > 1 else max(N, 1),
                                  scale_b.data_ptr(), scale_b.stride(0) if kb > 1 else max(N, 1),
                                  FP8_FORMATS[b_format], out.data_ptr(),
                                  out.stride(0) if M > 1 else max(n_out, 1), ctypes.byref(epi),
                                  ALGOS[algo], tile_m, tile_n)
        _check(s, h.ptr)
    return out


def mx_to_bf16(X: torch.Tensor, S: torch.Tensor, fmt: str = "e4m3", along: str = "row",
               handle: Handle | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 values of a block-scaled 8-bit matrix X (uint8, rows x cols) with
    E8M0 scales S: blocks of 32 along each row (S rows x ceil(cols/32)) or
    down each column (S ceil(rows/32) x cols).  `out`, if given, is a bf16
    rows x cols tensor on X's device with unit column stride."""
    rows, cols = X.shape
    if out is not None and (out.dtype != torch.bfloat16 or tuple(out.shape) != (rows, cols)
                            or out.device != X.device or (cols > 1 and out.stride(1) != 1)):
        raise ValueError("out must be a bf16 tensor of X's shape and device with unit column stride")
    Y = out if out is not None else torch.empty((rows, cols), dtype=torch.bfloat16, device=X.device)
    h = handle if handle is not None else default_handle()
    stream = torch.cuda.current_stream(X.device).cuda_stream
    with h.lock:
        h.set_stream(stream)
        s = lib().fgemm_mx_to_bf16(h.ptr, rows, cols, X.data_ptr(), X.stride(0) if rows > 1 else max(cols, 1),
                                   S.data_ptr(), S.stride(0) if S.shape[0] > 1 else max(S.shape[1], 1),
                                   FP8_FORMATS[fmt], 0 if along == "row" else 1, Y.data_ptr(),
                                   Y.stride(0) if rows > 1 else max(cols, 1))
        _check(s, h.ptr)
    return Y


def plan(M: int, N: int, K: int, dtype: torch.dtype = torch.bfloat16, epilogue: str = "none"):
    """(algorithm, tile_m, tile_n, predicted microseconds) the decision model picks."""
    h = default_handle()
    return h.plan(M, N, K, _dtype_code(dtype), make_epilogue(epilogue))


# ------------------------------------------- operators of a token step


# The raw handle of a device's current stream: torch.cuda.current_stream builds
# an object around it, which costs as much as one of these kernels.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _rows(t: torch.Tensor | None, name: str, shape, dtype, dev: int) -> tuple[int | None, int]:
    """(address, leading dimension) of a 2-D operand on device dev, checked;
    (None, 0) for None."""
    if t is None:
        return None, 0
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise FgemmError(ERR_INVALID_ARG, f"{name} must be a {tuple(shape)} {dtype} tensor on cuda:{dev}")
    ld, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        raise FgemmError(ERR_INVALID_ARG, f"{name} must be row-major with unit column stride")
    return t.data_ptr(), ld if shape[0] > 1 else max(shape[1], 1)


def _vector(t: torch.Tensor | None, name: str, n: int, dtype, dev: int) -> int | None:
    """Address of a contiguous vector of n entries on device dev, checked; None for None."""
    if t is None:
        return None
    if t.shape != (n,) or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        raise FgemmError(ERR_INVALID_ARG, f"{name} must be a contiguous vector of {n} {dtype} entries on cuda:{dev}")
    return t.data_ptr()


def _on(t: torch.Tensor, name: str, handle: Handle | None, dims: int = 2):
    """(library, handle, device index) of a call whose main operand is t."""
    dev = t.get_device()
    if dev < 0:
        raise FgemmError(ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise FgemmError(ERR_INVALID_ARG, f"{name} must be {dims}-D")
    h = handle if handle is not None else _handles.get(_current_device()) or default_handle()
    if dev != h.device:
        raise FgemmError(ERR_INVALID_ARG, f"{name} is on cuda:{dev}, the handle on cuda:{h.device}")
    return _lib or lib(), h, dev


def _run(h: Handle, dev: int, f, *args):
    """The C call f on h and args, on the current stream of device dev.  (ctypes lets other
    threads run during each call: without the lock another's stream could be set
    between the two.)"""
    with h.lock:
        _lib.fgemm_set_stream(h._h, _raw_stream(dev))
        s = f(h._h, *args)
        if s != OK:
            _check(s, h._h)


def _like(x: torch.Tensor) -> torch.Tensor:
    """New memory of x's shape and type whose rows lie behind 16-byte boundaries
    as x's do, so that the kernel takes the same sums."""
    m, n = x.shape
    ld = n + (x.stride(0) - n) % 8 if m > 1 else max(n, 1)
    shift = x.data_ptr() % 16 // x.element_size()
    return torch.empty(m * ld + shift, dtype=x.dtype, device=x.device).as_strided((m, n), (ld, 1), shift)


def _norm_operands(x, gain, residual, total, inv_rms, eps, handle, out=None):
    """The arguments both forms of the norm share, in the order of the C calls
    (through total's leading dimension), with the outputs they return."""
    L, h, dev = _on(x, "x", handle)
    t, shape = x.dtype, x.shape
    m, n = shape
    dt = _dtype_code(t)
    xp, ldx = _rows(x, "x", shape, t, dev)
    gp = _vector(gain, "gain", n, t, dev)
    if residual is None and total is None and (out is None or out.data_ptr() != xp):
        total, rp, ldr, tp, ldt = x, None, 0, None, 0
    else:
        rp, ldr = _rows(residual, "residual", shape, t, dev)
        if total is None:
            total = torch.empty_like(x) if residual is not None else _like(x)
        tp, ldt = _rows(total, "total", shape, t, dev)
    if inv_rms is None:
        inv_rms = torch.empty(m, dtype=torch.float32, device=x.device)
        ip = inv_rms.data_ptr()
    else:
        ip = _vector(inv_rms, "inv_rms", m, torch.float32, dev)
    return L, h, dev, (m, n, xp, ldx, rp, ldr, gp, eps, dt, tp, ldt), total, inv_rms, ip


def rms_norm(x: torch.Tensor, gain: torch.Tensor, *, residual: torch.Tensor | None = None, eps: float = 1e-6,
             out: torch.Tensor | None = None, total: torch.Tensor | None = None,
             inv_rms: torch.Tensor | None = None, handle: Handle | None = None):
    """(y, total, inv_rms) of fgemm_rms_norm: total = x + residual rounded to
    x's type (without a residual x itself, or a copy where out takes its place),
    y = total * inv_rms * gain with inv_rms = 1 / sqrt(mean(total^2) + eps) per
    row (fp32).

    x and residual are M x N fp16 or bf16, gain has N entries.  out, total and
    inv_rms, if given, are written (out or total may be x, total may be the
    residual)."""
    L, h, dev, args, total, inv_rms, ip = _norm_operands(x, gain, residual, total, inv_rms, eps, handle, out)
    if out is None:
        out = torch.empty_like(x)
    yp, ldy = _rows(out, "out", x.shape, x.dtype, dev)
    _run(h, dev, L.fgemm_rms_norm, *args, yp, ldy, ip)
    return out, total, inv_rms


def rms_norm_mx(x: torch.Tensor, gain: torch.Tensor, *, residual: torch.Tensor | None = None, eps: float = 1e-6,
                fmt: str = "e4m3", total: torch.Tensor | None = None, inv_rms: torch.Tensor | None = None,
                handle: Handle | None = None):
    """(q, scales, total, inv_rms) of fgemm_rms_norm_mx: rms_norm with its
    output in block-scaled 8 bits, q (M x N uint8) and E8M0 scales (M x
    ceil(N / 32) uint8) as matmul_mx takes its A and scale_a."""
    L, h, dev, args, total, inv_rms, ip = _norm_operands(x, gain, residual, total, inv_rms, eps, handle)
    if fmt not in FP8_FORMATS:
        raise FgemmError(ERR_INVALID_ARG, f"fmt must be one of {sorted(FP8_FORMATS)}")
    m, n = x.shape
    blocks = (n + 31) // 32
    q = torch.empty((m, n), dtype=torch.uint8, device=x.device)
    scales = torch.empty((m, blocks), dtype=torch.uint8, device=x.device)
    _run(h, dev, L.fgemm_rms_norm_mx, *args, FP8_FORMATS[fmt], q.data_ptr(), max(n, 1), scales.data_ptr(),
         max(blocks, 1), ip)
    return q, scales, total, inv_rms


def rms_norm_backward(dy: torch.Tensor, total: torch.Tensor, gain: torch.Tensor, inv_rms: torch.Tensor, *,
                      dtotal: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      dgain: torch.Tensor | None = None, handle: Handle | None = None):
    """(dx, dgain) of fgemm_rms_norm_backward, from dy and what rms_norm
    returned.  dx (dy's type) is the gradient of x and of the residual alike
    and includes dtotal, the gradient that reaches total by other ways; dgain
    (N fp32 entries) is summed over the rows.  out and dgain, if given, are
    written (out may be dy or dtotal)."""
    L, h, dev = _on(dy, "dy", handle)
    t, shape = dy.dtype, dy.shape
    m, n = shape
    dt = _dtype_code(t)
    dyp, lddy = _rows(dy, "dy", shape, t, dev)
    tp, ldt = _rows(total, "total", shape, t, dev)
    gp = _vector(gain, "gain", n, t, dev)
    ip = _vector(inv_rms, "inv_rms", m, torch.float32, dev)
    dtp, lddt = _rows(dtotal, "dtotal", shape, t, dev)
    if out is None:
        out = torch.empty_like(dy)
    op, ldo = _rows(out, "out", shape, t, dev)
    if dgain is None:
        dgain = torch.empty(n, dtype=torch.float32, device=dy.device)
    dgp = _vector(dgain, "dgain", n, torch.float32, dev)
    size = L.fgemm_rms_norm_backward_workspace(h._h, m, n)
    work = torch.empty(size, dtype=torch.uint8, device=dy.device)
    _run(h, dev, L.fgemm_rms_norm_backward, m, n, dyp, lddy, tp, ldt, gp, ip, dtp, lddt, dt, op, ldo, dgp,
         work.data_ptr(), size)
    return out, dgain


def matmul_w4(A: torch.Tensor, W: torch.Tensor, scales: torch.Tensor, *, zeros: torch.Tensor | None = None,
              group: int = 128, out: torch.Tensor | None = None, epilogue: str = "none", alpha: float = 1.0,
              bias: torch.Tensor | None = None, handle: Handle | None = None) -> torch.Tensor:
    """C = epi(alpha * A @ Wv.T + bias) through fgemm_matmul_w4, with 4-bit
    weights Wv[j, k] = (code[j, k] - zero[j, k // group]) * scale[j, k // group].

    A is M x K (fp16 or bf16), W is N x ceil(K / 2) uint8 (two codes to a byte
    along K, the even k in the low half), scales N x ceil(K / group) of A's
    type, zeros the same shape in uint8 (None: 8 everywhere), group 32, 64 or
    128.  Epilogues and bias as in matmul (swiglu: rows [0, N / 2) of W are
    the gate, the output is M x N / 2)."""
    L, h, dev = _on(A, "A", handle)
    t = A.dtype
    dt = _dtype_code(t)
    m, k = A.shape
    n = W.shape[0]
    if epilogue not in EPILOGUES:
        raise FgemmError(ERR_INVALID_ARG, f"epilogue must be one of {sorted(EPILOGUES)}")
    if group not in (32, 64, 128):
        raise FgemmError(ERR_INVALID_ARG, "group must be 32, 64 or 128")
    n_out = n // 2 if epilogue == "swiglu" else n
    groups = (n, (k + group - 1) // group)
    ap, lda = _rows(A, "A", (m, k), t, dev)
    wp, ldw = _rows(W, "W", (n, (k + 1) // 2), torch.uint8, dev)
    sp, lds = _rows(scales, "scales", groups, t, dev)
    zp, ldz = _rows(zeros, "zeros", groups, torch.uint8, dev)
    bp = _vector(bias, "bias", n, t, dev)
    if out is None:
        out = torch.empty((m, n_out), dtype=t, device=A.device)
    cp, ldc = _rows(out, "out", (m, n_out), t, dev)
    size = L.fgemm_matmul_w4_workspace(m, k, group)
    work = torch.empty(size, dtype=torch.uint8, device=A.device) if size else None
    _run(h, dev, L.fgemm_matmul_w4, m, n, k, ap, lda, wp, ldw, sp, lds, zp, ldz, group, cp, ldc, dt,
         ctypes.byref(Epilogue(EPILOGUES[epilogue], alpha, bp)), None if work is None else work.data_ptr(), size)
    return out


LOGIT_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def sample(logits: torch.Tensor, u: torch.Tensor, *, temperature: float | torch.Tensor = 1.0,
           top_k: int | torch.Tensor = 0, top_p: float | torch.Tensor = 1.0, min_p: float | torch.Tensor = 0.0,
           handle: Handle | None = None):
    """(token, prob) of fgemm_sample: one token (int32) from each row of
    logits (rows x vocab, fp16, bf16 or fp32) by the uniform numbers u (fp32,
    one a row), and its probability among the tokens that were kept (fp32).

    temperature (0: the largest logit), top_k (0: off), top_p (1: off) and
    min_p (0: off) are one number for all rows, or vectors with an entry for
    each (fp32; top_k int32).  A row with nothing above -inf gives token -1
    and prob 0."""
    L, h, dev = _on(logits, "logits", handle)
    rows, vocab = logits.shape
    code = LOGIT_TYPES.get(logits.dtype)
    if code is None:
        raise FgemmError(ERR_INVALID_ARG, f"logits must be float16, bfloat16 or float32, not {logits.dtype}")
    one, each = [], []
    for name, value, off, dtype in (("temperature", temperature, 1.0, torch.float32), ("top_k", top_k, 0, torch.int32),
                                    ("top_p", top_p, 1.0, torch.float32), ("min_p", min_p, 0.0, torch.float32)):
        if isinstance(value, torch.Tensor):
            one.append(off)
            each.append(_vector(value, name, rows, dtype, dev))
        else:
            # (ctypes would take the lower 32 bits of a top_k beyond them)
            one.append(min(max(value, -1), 0x7FFFFFFF) if name == "top_k" else value)
            each.append(None)
    lp, ld = _rows(logits, "logits", (rows, vocab), logits.dtype, dev)
    up = _vector(u, "u", rows, torch.float32, dev)
    token = torch.empty(rows, dtype=torch.int32, device=logits.device)
    prob = torch.empty(rows, dtype=torch.float32, device=logits.device)
    _run(h, dev, L.fgemm_sample, rows, vocab, lp, ld, code, up, ctypes.byref(Sampling(*one, *each)), token.data_ptr(),
         prob.data_ptr())
    return token, prob


# ---------------------------------- operators around a key-value cache


# The C calls take heads, page sizes and windows in 32 bits, and ctypes drops what is
# above them.
_INT32_MAX = 2 ** 31 - 1


def _softmax(scale: float | None, window: int, dim: int) -> tuple[float, int]:
    """scale (None: 1 / sqrt(dim)) and window for a C call; a window beyond 32 bits is
    the largest there is."""
    return (max(dim, 1) ** -0.5 if scale is None else scale), max(-1, min(window, _INT32_MAX))


def _heads(t: torch.Tensor, name: str, shape, dtype, dev: int) -> tuple[int, int, int]:
    """(address, token stride, head stride) of a tokens x heads x dim operand on
    device dev, checked."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise FgemmError(ERR_INVALID_ARG, f"{name} must be a {tuple(shape)} {dtype} tensor on cuda:{dev}")
    if shape[1] > _INT32_MAX or shape[2] > _INT32_MAX:
        raise FgemmError(ERR_INVALID_ARG, f"{name} has more heads, or values of a head, than 32 bits count")
    ld, hs, unit = t.stride()
    if unit != 1 and shape[2] > 1:
        raise FgemmError(ERR_INVALID_ARG, f"the values of a head of {name} must be adjacent")
    return t.data_ptr(), ld, hs


def _cache(k: torch.Tensor, v: torch.Tensor, kv_heads: int | None, dim: int, dtype, dev: int) -> KvCache:
    """The C view of a paged cache, checked; kv_heads None: any number."""
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or shape[3] != dim or kv_heads not in (None, shape[2]) or \
            k.dtype != dtype or v.dtype != dtype or k.get_device() != dev or v.get_device() != dev:
        raise FgemmError(ERR_INVALID_ARG, f"k_cache and v_cache must be pages x page size x key heads x {dim} {dtype} "
                                          f"tensors of one shape on cuda:{dev}")
    if shape[1] > _INT32_MAX or shape[2] > _INT32_MAX:
        raise FgemmError(ERR_INVALID_ARG, "a page of the cache has more tokens, or heads, than 32 bits count")
    k_page, k_token, k_head, k_unit = k.stride()
    v_page, v_token, v_head, v_unit = v.stride()
    if (k_unit != 1 or v_unit != 1) and dim > 1:
        raise FgemmError(ERR_INVALID_ARG, "the values of a head of k_cache and v_cache must be adjacent")
    return KvCache(k.data_ptr(), v.data_ptr(), shape[0], shape[1], k_page, k_token, k_head, v_page, v_token, v_head)


def rotary_cache(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                 inv_freq: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, *, interleaved: bool = False,
                 out: torch.Tensor | None = None, handle: Handle | None = None) -> torch.Tensor:
    """The queries with rotary positions (fgemm_rotary_cache); the keys with
    theirs and the values go into the cache.

    q is T x heads x dim, k and v T x key heads x dim (fp16 or bf16; parts of one
    projection's output do), positions and slots T int32 entries, inv_freq rot / 2
    fp32 entries (radians a position).  The first rot values of a head turn in
    pairs (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved.  k_cache and v_cache are
    pages x page size x key heads x dim; slot = page * page size + token in the
    page, tokens with a slot outside the cache (-1) are not written.  out, if
    given, is written (it may be q).  The outputs carry no gradients."""
    L, h, dev = _on(q, "q", handle, 3)
    t = q.dtype
    dt = _dtype_code(t)
    n, heads, dim = q.shape
    kv = (n, k.shape[1] if k.dim() == 3 else 1, dim)
    qa = _heads(q, "q", q.shape, t, dev)
    ka = _heads(k, "k", kv, t, dev)
    va = _heads(v, "v", kv, t, dev)
    pp = _vector(positions, "positions", n, torch.int32, dev)
    sp = _vector(slots, "slots", n, torch.int32, dev)
    half = inv_freq.shape[0] if inv_freq.dim() == 1 else 0
    if 2 * half > dim:
        raise FgemmError(ERR_INVALID_ARG, "inv_freq has more entries than a head has pairs")
    fp = _vector(inv_freq, "inv_freq", half, torch.float32, dev)
    cache = _cache(k_cache, v_cache, kv[1], dim, t, dev)
    if out is None:
        out = torch.empty_like(q)
    oa = _heads(out, "out", q.shape, t, dev)
    _run(h, dev, L.fgemm_rotary_cache, n, heads, kv[1], dim, *qa, *ka, *va, pp, sp, fp, 2 * half,
         1 if interleaved else 0, dt, *oa, ctypes.byref(cache))
    return out


def attention_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                    lengths: torch.Tensor, *, scale: float | None = None, window: int = 0,
                    out: torch.Tensor | None = None, handle: Handle | None = None):
    """(out, lse) of fgemm_attention_paged: attention of one new token of each
    sequence, q (sequences x heads x dim), over the lengths[s] tokens (int32,
    the new one among them) that the pages page_table[s] (int32) of the cache
    hold (k_cache and v_cache: pages x page size x key heads x dim).

    scale None: 1 / sqrt(dim); window 0: every token, else the last `window`.
    lse is the natural logarithm of each row's sum (sequences x heads, fp32); a
    sequence of length 0 gives zeros and -inf.  out, if given, is written (it
    may be q).  The outputs carry no gradients."""
    L, h, dev = _on(q, "q", handle, 3)
    t = q.dtype
    dt = _dtype_code(t)
    n, heads, dim = q.shape
    cache = _cache(k_cache, v_cache, None, dim, t, dev)
    kv_heads = k_cache.shape[2]
    qa = _heads(q, "q", q.shape, t, dev)
    pages = page_table.shape[1] if page_table.dim() == 2 else 0
    tp, ldt = _rows(page_table, "page_table", (n, pages), torch.int32, dev)
    lp = _vector(lengths, "lengths", n, torch.int32, dev)
    if out is None:
        out = torch.empty_like(q)
    oa = _heads(out, "out", q.shape, t, dev)
    lse = torch.empty((n, heads), dtype=torch.float32, device=q.device)
    scale, window = _softmax(scale, window, dim)
    size = L.fgemm_attention_paged_workspace(h._h, n, heads, kv_heads, dim)
    work = torch.empty(size, dtype=torch.uint8, device=q.device) if size else None
    _run(h, dev, L.fgemm_attention_paged, n, heads, kv_heads, dim, *qa, ctypes.byref(cache), tp, ldt, pages, lp,
         scale, window, dt, *oa, lse.data_ptr(), None if work is None else work.data_ptr(), size)
    return out, lse


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor, *,
              k_starts: torch.Tensor | None = None, causal: bool = True, window: int = 0, scale: float | None = None,
              out: torch.Tensor | None = None, lse: torch.Tensor | None = None, handle: Handle | None = None):
    """(out, lse) of fgemm_attention over packed prompts: sequence s has the
    queries starts[s] .. starts[s + 1] - 1 of q (T x heads x dim) and the keys and
    values k_starts[s] .. k_starts[s + 1] - 1 of k and v (T_k x key heads x dim);
    its queries are the last of its keys' positions.  starts and k_starts (None:
    starts) are ascending int32 vectors of sequences + 1 entries.

    causal: keys up to a query's own position, the last `window` of them if
    window > 0.  scale None: 1 / sqrt(dim).  lse is the natural logarithm of each
    row's sum (T x heads, fp32).  A query that sees no key gives zeros and -inf;
    rows of no sequence are left as they are.  out and lse, if given, are
    written.  The outputs carry no gradients."""
    L, h, dev = _on(q, "q", handle, 3)
    t = q.dtype
    dt = _dtype_code(t)
    n, heads, dim = q.shape
    kv = (k.shape[0], k.shape[1], dim) if k.dim() == 3 else (0, 1, dim)
    qa = _heads(q, "q", q.shape, t, dev)
    ka = _heads(k, "k", kv, t, dev)
    va = _heads(v, "v", kv, t, dev)
    seqs = starts.shape[0] - 1 if starts.dim() == 1 else -1
    if seqs < 0:
        raise FgemmError(ERR_INVALID_ARG, "starts must be a vector of sequences + 1 entries")
    sp = _vector(starts, "starts", seqs + 1, torch.int32, dev)
    kp = _vector(k_starts, "k_starts", seqs + 1, torch.int32, dev)
    if out is None:
        out = torch.empty_like(q)
    oa = _heads(out, "out", q.shape, t, dev)
    if lse is None:
        lse = torch.empty((n, heads), dtype=torch.float32, device=q.device)
    elif lse.shape != (n, heads) or lse.dtype != torch.float32 or lse.get_device() != dev or not lse.is_contiguous():
        raise FgemmError(ERR_INVALID_ARG, f"lse must be a contiguous {(n, heads)} float32 tensor on cuda:{dev}")
    scale, window = _softmax(scale, window, dim)
    _run(h, dev, L.fgemm_attention, seqs, n, kv[0], heads, kv[1], dim, *qa, *ka, *va, sp, kp, 1 if causal else 0,
         window, scale, dt, *oa, lse.data_ptr())
    return out, lse


def logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, top: int = 0, handle: Handle | None = None):
    """(logprob, entropy, top_tokens, top_logprobs) of fgemm_logprobs: for each
    row of logits (rows x vocab, fp16, bf16 or fp32) the log probability of the
    given token (int32), the entropy (both fp32, natural logarithms), and the
    `top` (0 to 32) most probable tokens (rows x top, int32, ties by the lower
    index) with their log probabilities (fp32).

    A token outside the vocabulary has -inf; where fewer than `top` logits are
    above -inf the rest is token -1 with -inf.  The outputs carry no gradients."""
    L, h, dev = _on(logits, "logits", handle)
    rows, vocab = logits.shape
    code = LOGIT_TYPES.get(logits.dtype)
    if code is None:
        raise FgemmError(ERR_INVALID_ARG, f"logits must be float16, bfloat16 or float32, not {logits.dtype}")
    if not 0 <= top <= 32:
        raise FgemmError(ERR_INVALID_ARG, "top must be in 0 .. 32")
    lp, ld = _rows(logits, "logits", (rows, vocab), logits.dtype, dev)
    tp = _vector(tokens, "tokens", rows, torch.int32, dev)
    logprob = torch.empty(rows, dtype=torch.float32, device=logits.device)
    entropy = torch.empty(rows, dtype=torch.float32, device=logits.device)
    top_tokens = torch.empty((rows, top), dtype=torch.int32, device=logits.device)
    top_logprobs = torch.empty((rows, top), dtype=torch.float32, device=logits.device)
    _run(h, dev, L.fgemm_logprobs, rows, vocab, lp, ld, code, tp, top, logprob.data_ptr(), entropy.data_ptr(),
         top_tokens.data_ptr() if top else None, top_logprobs.data_ptr() if top else None)
    return logprob, entropy, top_tokens, top_logprobs
