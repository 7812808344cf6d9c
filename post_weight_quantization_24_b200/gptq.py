"""Python binding of ``libgptq_b200.so`` (ctypes; argument marshalling only).

Every computation runs in the library's sm_100a kernels; torch supplies device memory and the
current CUDA stream. If the library is not built, calls raise immediately — there is no CPU or
torch fallback.

Functions (names follow the C ABI in ``include/gptq.h``):
  Hessian(d_in)                    handle: .accumulate(X), .get(), .data_ptr, .tokens, .reset()
  hessian_accumulate_into(H, X)    H += 2·XᵀX on a caller tensor (upper triangle)
  quantize_layer(W, H, ...)        GPTQ one linear layer -> codes, scales, zeros, g_idx, perm, loss
  quantize_layer_workspace(...)    workspace bytes for quantize_layer
  inverse_factor(H, ...)           processing order and U with UᵀU = H_d⁻¹ (stage 2 alone)
  rtn_minmax_quantize(W, ...)      group min-max RTN -> packed codes, scales, zeros
  fp8_quantize_act(X)              e4m3 codes, a scale per token and 128 channels
  fp8_quantize_weight(W)           e4m3 codes, a scale per 128 x 128 block
  fp8_linear(X8, sx, W8, sw, ...)  Y = X̂·Ŵᵀ (+ R) from those codes and scales
  kv_cache_alloc / _write / _read  paged key/value cache of 4- or 8-bit codes
  profile_enable(on), profile_read()  per-stage milliseconds of the last quantize_layer call
"""

from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgptq_b200.so")

STATUS = {0: "GPTQ_OK", -1: "GPTQ_ERR_ARG", -2: "GPTQ_ERR_NOT_PD", -3: "GPTQ_ERR_NONFINITE",
          -4: "GPTQ_ERR_CUDA", -5: "GPTQ_ERR_OOM", -6: "GPTQ_ERR_TIMEOUT",
          -7: "GPTQ_ERR_WORKSPACE", -8: "GPTQ_ERR_UNSUPPORTED"}
DTYPE_F16, DTYPE_F32, DTYPE_BF16 = 0, 1, 2
STAGES = ("prepare", "factor", "images", "column_loop", "lazy_update", "assemble", "loss")


class GPTQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{where}: {self.name}")


_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "gptq_status_string": ([_I], ctypes.c_char_p),
    "gptq_hessian_create": ([_I, ctypes.POINTER(_P)], _I),
    "gptq_hessian_accumulate": ([_P, _P, _I64, _P], _I),
    "gptq_hessian_get": ([_P, _P, _P], _I),
    "gptq_hessian_data": ([_P], _P),
    "gptq_hessian_tokens": ([_P], _I64),
    "gptq_hessian_dim": ([_P], _I),
    "gptq_hessian_reset": ([_P, _P], _I),
    "gptq_hessian_destroy": ([_P], _I),
    "gptq_hessian_accumulate_into": ([_P, _I, _P, _I64, _I, _P, _P], _I),
    "gptq_quantize_layer_workspace": ([_I, _I, _I], _SZ),
    "gptq_quantize_layer": ([_P, _I, _I, _I, _P, _I, _I, _I, _F, _I, _P, _P, _P, _P, _P,
                             ctypes.POINTER(_F), _P, _SZ, _P], _I),
    "gptq_inverse_factor_workspace": ([_I], _SZ),
    "gptq_inverse_factor": ([_P, _I, _F, _I, _P, _P, _P, _SZ, _P], _I),
    "rtn_minmax_quantize": ([_P, _I, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "gptq_quantize_layer_ex": ([_P, _I, _I, _I, _P, _I, _I, _I, _F, _I, _I, _I, _P, _P, _P, _P,
                                _P, ctypes.POINTER(_F), _P, _SZ, _P], _I),
    "rtn_quantize_ex": ([_P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "rtn_clip_search": ([_P, _I, _I, _I, _I, _I, _I, _P, ctypes.c_double, ctypes.c_double, _P,
                         _P, _P, _P, _P], _I),
    "rtn_range_clip": ([_P, _I, _I, _I, _I, _I, _I, ctypes.c_double, ctypes.c_double, _P, _P,
                        _P, _P], _I),
    "w4a16_pack": ([_P, _I, _I, _P, _P, _P], _I),
    "w4a16_linear_workspace": ([_I64, _I, _I], _SZ),
    "w4a16_linear": ([_P, _I64, _I, _P, _P, _P, _I, _I, _P, _P, _P, _P, _SZ, _P, _P], _I),
    "gptq_silu_mul": ([_P, _I64, _I, _P, _P], _I),
    "gptq_rms_norm": ([_P, _I64, _I, _F, _P, _P], _I),
    "gptq_channel_abs_sum": ([_P, _I, _I64, _I, _P, _P], _I),
    "awq_lite_workspace": ([_I, _I, ctypes.c_double], _SZ),
    "awq_lite_search": ([_P, _I, _I, _I, _P, _I64, _P, _I, _I, _I, ctypes.c_double, _P, _P, _P,
                         _P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_I), _P, _SZ, _P],
                        _I),
    "fp8_quantize_act": ([_P, _I, _I64, _I, _P, _P, _P], _I),
    "fp8_quantize_weight": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "fp8_linear": ([_P, _P, _I64, _I, _P, _P, _I, _P, _P, _I, _P, _P], _I),
    "kv_cache_write": ([_P, _P, _I, _I64, _I64, _I64, _I, _I, _P, _I64, _I, _I, _P, _P, _P, _P,
                        _P], _I),
    "kv_cache_read": ([_P, _P, _P, _I64, _I, _I, _I, _I, _I, _P, _I, _I, _P, _I64, _P, _P, _I,
                       _P, _P], _I),
    "gptq_quantize_layer_noalloc": ([_P, _I, _I, _I, _P, _I, _I, _I, _F, _I, _P, _P, _P, _P, _P,
                                     ctypes.POINTER(_F), _P], _I),
    "gptq_profile_enable": ([_I], None),
    "gptq_profile_read": ([ctypes.POINTER(_F), _I], _I),
    "gptq_launch_count": ([], ctypes.c_ulonglong),
    "gptq_test_stall_factor": ([_I], _I),
    "gptq_test_stall_fp8": ([_I], _I),
    "gptq_test_fp8_no_pair": ([_I], _I),
}


def lib() -> ctypes.CDLL:
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m post_weight_quantization_24_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise GPTQError(status, where)


def _stream() -> int:
    # the current stream's handle without building a Stream object (3 us less per call)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return DTYPE_F16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"W must be float16 or float32, got {t.dtype}")


def _require_cuda(t: torch.Tensor, name: str) -> None:
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


# ------------------------------------------------------------------------------------------
# Hessian
# ------------------------------------------------------------------------------------------
class Hessian:
    """H = 2·XᵀX accumulated over calls (fp32, d_in x d_in) on the current device."""

    def __init__(self, d_in: int):
        h = _P()
        _check(lib().gptq_hessian_create(d_in, ctypes.byref(h)), "gptq_hessian_create")
        self._h = h
        self.d_in = d_in

    def accumulate(self, X: torch.Tensor) -> None:
        _require_cuda(X, "X")
        if X.dtype != torch.float16 or X.dim() != 2 or X.shape[1] != self.d_in:
            raise ValueError("X must be fp16 [n_tokens, d_in]")
        _check(lib().gptq_hessian_accumulate(self._h, X.data_ptr(), X.shape[0], _stream()),
               "gptq_hessian_accumulate")

    def get(self, out: torch.Tensor | None = None) -> torch.Tensor:
        if out is None:
            out = torch.empty(self.d_in, self.d_in, dtype=torch.float32, device="cuda")
        _check(lib().gptq_hessian_get(self._h, out.data_ptr(), _stream()), "gptq_hessian_get")
        return out

    @property
    def data_ptr(self) -> int:
        return lib().gptq_hessian_data(self._h)

    def raw(self) -> torch.Tensor:
        """The handle's storage viewed as a tensor (upper triangle valid); no copy."""
        return _wrap_device_ptr(self.data_ptr, (self.d_in, self.d_in), owner=self)

    @property
    def tokens(self) -> int:
        return lib().gptq_hessian_tokens(self._h)

    def reset(self) -> None:
        _check(lib().gptq_hessian_reset(self._h, _stream()), "gptq_hessian_reset")

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().gptq_hessian_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _wrap_device_ptr(ptr: int, shape, owner):
    """Zero-copy fp32 tensor over device memory owned by ``owner`` (kept alive by the tensor)."""
    class _CAI:
        def __init__(self):
            self.__cuda_array_interface__ = {
                "shape": tuple(shape), "typestr": "<f4", "data": (ptr, False), "version": 3,
                "strides": None}
            self._owner = owner
    return torch.as_tensor(_CAI(), device="cuda")


def hessian_accumulate_into(H: torch.Tensor, X: torch.Tensor, unit_tokens: int = 0,
                            status: torch.Tensor | None = None) -> None:
    """H (fp32 [d, d], upper triangle) += 2·XᵀX for X fp16 [n, d]."""
    _require_cuda(H, "H")
    _require_cuda(X, "X")
    if H.dtype != torch.float32 or X.dtype != torch.float16:
        raise TypeError("H must be fp32 and X fp16")
    d = H.shape[0]
    if H.shape != (d, d) or X.dim() != 2 or X.shape[1] != d:
        raise ValueError("shape mismatch")
    _check(lib().gptq_hessian_accumulate_into(H.data_ptr(), d, X.data_ptr(), X.shape[0],
                                              unit_tokens, _ptr(status), _stream()),
           "gptq_hessian_accumulate_into")


# ------------------------------------------------------------------------------------------
# GPTQ layer
# ------------------------------------------------------------------------------------------
def quantize_layer_workspace(d_out: int, d_in: int, block_size: int = 128) -> int:
    return int(lib().gptq_quantize_layer_workspace(d_out, d_in, block_size))


def quantize_layer(W: torch.Tensor, H: torch.Tensor, bits: int = 4, group_size: int = 128,
                   block_size: int = 128, percdamp: float = 0.01, act_order: bool = False,
                   compute_loss: bool = False, workspace: torch.Tensor | None = None,
                   out: dict | None = None, sym: bool = False,
                   static_groups: bool = False) -> dict:
    """GPTQ-quantize W [d_out, d_in] (fp16/fp32) with Hessian H [d_in, d_in] (upper read).

    Returns dict(codes uint8 [d_out, d_in] original order, scales/zeros fp16 [d_out, d_in/g],
    g_idx int32 [d_in], perm int32 [d_in], loss float | None). ``sym``, ``static_groups`` and
    group_size == d_in (per-channel) select the quantizer variants of gptq_quantize_layer_ex.
    """
    _require_cuda(W, "W")
    _require_cuda(H, "H")
    d_out, d_in = W.shape
    if H.dtype != torch.float32 or H.shape != (d_in, d_in):
        raise ValueError("H must be fp32 [d_in, d_in]")
    dev = W.device
    if out is None:
        ng = d_in // group_size if group_size > 0 and d_in % group_size == 0 else 1
        out = dict(codes=torch.empty(d_out, d_in, dtype=torch.uint8, device=dev),
                   scales=torch.empty(d_out, ng, dtype=torch.float16, device=dev),
                   zeros=torch.empty(d_out, ng, dtype=torch.float16, device=dev),
                   g_idx=torch.empty(d_in, dtype=torch.int32, device=dev),
                   perm=torch.empty(d_in, dtype=torch.int32, device=dev))
    if workspace is None:
        nbytes = quantize_layer_workspace(d_out, d_in, block_size)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    loss = ctypes.c_float(float("nan"))
    st = lib().gptq_quantize_layer_ex(
        W.data_ptr(), _dtype_code(W), d_out, d_in, H.data_ptr(), bits, group_size, block_size,
        float(percdamp), int(bool(act_order)), int(bool(sym)), int(bool(static_groups)),
        out["codes"].data_ptr(), out["scales"].data_ptr(), out["zeros"].data_ptr(),
        out["g_idx"].data_ptr(), _ptr(out.get("perm")),
        ctypes.byref(loss) if compute_loss else None, workspace.data_ptr(),
        workspace.numel(), _stream())
    _check(st, "gptq_quantize_layer_ex")
    res = dict(out)
    res["loss"] = float(loss.value) if compute_loss else None
    return res


def quantize_layer_noalloc(W: torch.Tensor, H: torch.Tensor, bits: int = 4,
                           group_size: int = 128, block_size: int = 128,
                           percdamp: float = 0.01, act_order: bool = False,
                           compute_loss: bool = False, out: dict | None = None) -> dict:
    """quantize_layer without a workspace: the library uses its fixed 32 MiB device scratch.

    For callers that may not allocate device memory while quantizing. Only ``out`` (the
    caller's output tensors) is allocated here when it is not given. Layers whose workspace
    would exceed 32 MiB raise GPTQError(GPTQ_ERR_WORKSPACE). Calls share the scratch, so they
    must not overlap on the GPU.
    """
    _require_cuda(W, "W")
    _require_cuda(H, "H")
    d_out, d_in = W.shape
    dev = W.device
    if out is None:
        ng = d_in // group_size if group_size > 0 and d_in % group_size == 0 else 1
        out = dict(codes=torch.empty(d_out, d_in, dtype=torch.uint8, device=dev),
                   scales=torch.empty(d_out, ng, dtype=torch.float16, device=dev),
                   zeros=torch.empty(d_out, ng, dtype=torch.float16, device=dev),
                   g_idx=torch.empty(d_in, dtype=torch.int32, device=dev),
                   perm=torch.empty(d_in, dtype=torch.int32, device=dev))
    loss = ctypes.c_float(float("nan"))
    st = lib().gptq_quantize_layer_noalloc(
        W.data_ptr(), _dtype_code(W), d_out, d_in, H.data_ptr(), bits, group_size, block_size,
        float(percdamp), int(bool(act_order)), out["codes"].data_ptr(), out["scales"].data_ptr(),
        out["zeros"].data_ptr(), out["g_idx"].data_ptr(), _ptr(out.get("perm")),
        ctypes.byref(loss) if compute_loss else None, _stream())
    _check(st, "gptq_quantize_layer_noalloc")
    res = dict(out)
    res["loss"] = float(loss.value) if compute_loss else None
    return res


def inverse_factor(H: torch.Tensor, percdamp: float = 0.01, act_order: bool = False):
    """(U, perm): U upper with UᵀU = (P H P + λI)⁻¹ in processing order; perm int32."""
    _require_cuda(H, "H")
    d = H.shape[0]
    U = torch.empty(d, d, dtype=torch.float32, device=H.device)
    perm = torch.empty(d, dtype=torch.int32, device=H.device)
    ws = torch.empty(int(lib().gptq_inverse_factor_workspace(d)), dtype=torch.uint8,
                     device=H.device)
    _check(lib().gptq_inverse_factor(H.data_ptr(), d, float(percdamp), int(bool(act_order)),
                                     U.data_ptr(), perm.data_ptr(), ws.data_ptr(), ws.numel(),
                                     _stream()), "gptq_inverse_factor")
    return U, perm


# ------------------------------------------------------------------------------------------
# RTN
# ------------------------------------------------------------------------------------------
def rtn_minmax_quantize(W: torch.Tensor, bits: int = 4, group_size: int = 128,
                        out: tuple | None = None, sym: bool = False):
    """Group min-max RTN of W [d_out, d_in] -> (packed uint8, scales fp16, zeros fp16).

    bits == 4: packed is [d_out, d_in/2] (even column in the low nibble); else [d_out, d_in].
    ``sym`` takes the symmetric quantizer (rtn_quantize_ex).
    """
    _require_cuda(W, "W")
    d_out, d_in = W.shape
    dev = W.device
    if out is None:
        ng = d_in // group_size if group_size > 0 and d_in % group_size == 0 else 1
        packed = torch.empty(d_out, d_in // 2 if bits == 4 else d_in, dtype=torch.uint8, device=dev)
        out = (packed, torch.empty(d_out, ng, dtype=torch.float16, device=dev),
               torch.empty(d_out, ng, dtype=torch.float16, device=dev))
    packed, scales, zeros = out
    st = lib().rtn_quantize_ex(W.data_ptr(), _dtype_code(W), d_out, d_in, bits, group_size,
                               int(bool(sym)), packed.data_ptr(), scales.data_ptr(),
                               zeros.data_ptr(), _stream())
    _check(st, "rtn_quantize_ex")
    return packed, scales, zeros


def rtn_clip_search(W: torch.Tensor, bits: int = 4, group_size: int = 128,
                    H: torch.Tensor | None = None, sym: bool = False, min_ratio: float = 0.5,
                    step: float = 0.05):
    """Group RTN with a clip search per group (criterion d·H_gg·d, or d·d without H) ->
    (packed uint8, scales fp16, zeros fp16, ratio index uint8 [d_out, d_in/g])."""
    _require_cuda(W, "W")
    d_out, d_in = W.shape
    dev = W.device
    ng = d_in // group_size if group_size > 0 and d_in % group_size == 0 else 1
    packed = torch.empty(d_out, d_in // 2 if bits == 4 else d_in, dtype=torch.uint8, device=dev)
    scales = torch.empty(d_out, ng, dtype=torch.float16, device=dev)
    zeros = torch.empty(d_out, ng, dtype=torch.float16, device=dev)
    ridx = torch.empty(d_out, ng, dtype=torch.uint8, device=dev)
    if H is not None:
        _require_cuda(H, "H")
        if H.dtype != torch.float32 or H.shape != (d_in, d_in):
            raise ValueError("H must be fp32 [d_in, d_in]")
    st = lib().rtn_clip_search(W.data_ptr(), _dtype_code(W), d_out, d_in, bits, group_size,
                               int(bool(sym)), _ptr(H), float(min_ratio), float(step),
                               packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                               ridx.data_ptr(), _stream())
    _check(st, "rtn_clip_search")
    return packed, scales, zeros, ridx


def rtn_range_clip(W: torch.Tensor, bits: int = 4, group_size: int = 128,
                   percentile: float = 99.99, abs_range: float = 0.0, sym: bool = False):
    """Group RTN of the weights clipped to each group's (100 - percentile)/percentile
    quantiles, limited to [-abs_range, abs_range] when abs_range > 0 ->
    (packed uint8, scales fp16, zeros fp16)."""
    _require_cuda(W, "W")
    d_out, d_in = W.shape
    dev = W.device
    ng = d_in // group_size if group_size > 0 and d_in % group_size == 0 else 1
    packed = torch.empty(d_out, d_in // 2 if bits == 4 else d_in, dtype=torch.uint8, device=dev)
    scales = torch.empty(d_out, ng, dtype=torch.float16, device=dev)
    zeros = torch.empty(d_out, ng, dtype=torch.float16, device=dev)
    st = lib().rtn_range_clip(W.data_ptr(), _dtype_code(W), d_out, d_in, bits, group_size,
                              int(bool(sym)), float(percentile), float(abs_range),
                              packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(), _stream())
    _check(st, "rtn_range_clip")
    return packed, scales, zeros


# ------------------------------------------------------------------------------------------
# W4A16 layer
# ------------------------------------------------------------------------------------------
def w4a16_pack(codes: torch.Tensor, perm: torch.Tensor | None = None) -> torch.Tensor:
    """INT4 codes [d_out, d_in] (original order) -> packed [d_out, d_in/2] in perm's order."""
    _require_cuda(codes, "codes")
    d_out, d_in = codes.shape
    packed = torch.empty(d_out, d_in // 2, dtype=torch.uint8, device=codes.device)
    _check(lib().w4a16_pack(codes.data_ptr(), d_out, d_in, _ptr(perm), packed.data_ptr(),
                            _stream()), "w4a16_pack")
    return packed


def w4a16_linear(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                 zeros: torch.Tensor, group_size: int = 128, perm: torch.Tensor | None = None,
                 R: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None,
                 status: torch.Tensor | None = None) -> torch.Tensor:
    """Y = fp16(X·Ŵᵀ + R) for fp16 X [n, d_in] and packed INT4 weights [d_out, d_in/2]."""
    _require_cuda(X, "X")
    n, d_in = X.shape
    d_out = packed.shape[0]
    if out is None:
        out = torch.empty(n, d_out, dtype=torch.float16, device=X.device)
    nb = int(lib().w4a16_linear_workspace(n, d_in, int(perm is not None)))
    if perm is not None and (workspace is None or workspace.numel() < nb):
        workspace = torch.empty(nb, dtype=torch.uint8, device=X.device)
    st = lib().w4a16_linear(X.data_ptr(), n, d_in, packed.data_ptr(), scales.data_ptr(),
                            zeros.data_ptr(), group_size, d_out, _ptr(perm), _ptr(R),
                            out.data_ptr(), _ptr(workspace),
                            0 if workspace is None else workspace.numel(), _ptr(status),
                            _stream())
    _check(st, "w4a16_linear")
    return out


def channel_abs_sum(X: torch.Tensor, sums: torch.Tensor | None = None) -> torch.Tensor:
    """sums[c] += Σ_t |X[t, c]| (fp64 [d]); a new zeroed buffer when `sums` is None."""
    _require_cuda(X, "X")
    n, d = X.shape
    if sums is None:
        sums = torch.zeros(d, dtype=torch.float64, device=X.device)
    _check(lib().gptq_channel_abs_sum(X.data_ptr(), _dtype_code(X), n, d, sums.data_ptr(),
                                      _stream()), "gptq_channel_abs_sum")
    return sums


def awq_lite_search(W: torch.Tensor, x_abs_sum: torch.Tensor, n_tokens: int, H: torch.Tensor,
                    bits: int = 4, group_size: int = 128, sym: bool = False,
                    alpha_step: float = 0.1) -> dict:
    """AWQ-lite grid search (H full symmetric). Returns dict(packed, scales, zeros, s (fp16
    [d_in]), losses (list), best (index), alpha)."""
    _require_cuda(W, "W")
    _require_cuda(H, "H")
    d_out, d_in = W.shape
    dev = W.device
    ng = d_in // group_size
    n_alpha = int(round(1.0 / alpha_step)) + 1
    packed = torch.empty(d_out, d_in // 2 if bits == 4 else d_in, dtype=torch.uint8, device=dev)
    scales = torch.empty(d_out, ng, dtype=torch.float16, device=dev)
    zeros = torch.empty(d_out, ng, dtype=torch.float16, device=dev)
    s_out = torch.empty(d_in, dtype=torch.float16, device=dev)
    ws = torch.empty(max(1, int(lib().awq_lite_workspace(d_out, d_in, float(alpha_step)))),
                     dtype=torch.uint8, device=dev)
    losses = (ctypes.c_double * n_alpha)()
    best = ctypes.c_int(-1)
    st = lib().awq_lite_search(W.data_ptr(), _dtype_code(W), d_out, d_in, x_abs_sum.data_ptr(),
                               int(n_tokens), H.data_ptr(), bits, group_size, int(bool(sym)),
                               float(alpha_step), packed.data_ptr(), scales.data_ptr(),
                               zeros.data_ptr(), s_out.data_ptr(), losses, ctypes.byref(best),
                               ws.data_ptr(), ws.numel(), _stream())
    _check(st, "awq_lite_search")
    return dict(packed=packed, scales=scales, zeros=zeros, s=s_out, losses=list(losses),
                best=int(best.value), alpha=int(best.value) * alpha_step)


def rms_norm(X: torch.Tensor, eps: float = 1e-6, out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = fp16(x / sqrt(mean(x²) + eps)) per row of fp16 X [n, d] (unit-weight RMS norm)."""
    _require_cuda(X, "X")
    n, d = X.shape
    if out is None:
        out = torch.empty_like(X)
    _check(lib().gptq_rms_norm(X.data_ptr(), n, d, float(eps), out.data_ptr(), _stream()),
           "gptq_rms_norm")
    return out


def silu_mul(GU: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """A = fp16(silu(gate)·up) for GU fp16 [n, 2·d_ff] (gate outputs, then up outputs)."""
    _require_cuda(GU, "GU")
    n, two = GU.shape
    if out is None:
        out = torch.empty(n, two // 2, dtype=torch.float16, device=GU.device)
    _check(lib().gptq_silu_mul(GU.data_ptr(), n, two // 2, out.data_ptr(), _stream()),
           "gptq_silu_mul")
    return out


# ------------------------------------------------------------------------------------------
# 8-bit floating-point layer
# ------------------------------------------------------------------------------------------
_FLOAT_CODES = {torch.float16: DTYPE_F16, torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_E4M3 = torch.float8_e4m3fn


def _float_code(dtype: torch.dtype, name: str) -> int:
    code = _FLOAT_CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float16, float32 or bfloat16, got {dtype}")
    return code


def _device() -> int:
    """The current CUDA device; no tensor's (-2) before CUDA is in use, when all are the host's."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2


def _require(t: torch.Tensor, name: str, dtype: torch.dtype | None = None, shape=None,
             dev: int | None = None) -> None:
    """A contiguous tensor on the current CUDA device (``dev``), of this type and shape."""
    if dev is None:
        dev = _device()
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on the current device")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _require_status(status: torch.Tensor | None) -> None:
    if status is not None:
        _require(status, "status", torch.int32)
        if status.numel() < 1:
            raise ValueError("status must hold an int32")


def fp8_quantize_act(X: torch.Tensor, out: tuple | None = None):
    """Activations X [n, d] (fp16/fp32/bf16, d a multiple of 16) -> (codes float8_e4m3fn [n, d],
    scales fp32 [ceil(d/128), n]): one scale per token and 128 channels (see fp8_quantize_act in
    include/gptq.h). ``out``: the two tensors to write."""
    _require(X, "X")
    if X.dim() != 2:
        raise ValueError("X must be [n, d]")
    n, d = X.shape
    code = _float_code(X.dtype, "X")
    nb = (d + 127) // 128
    if out is None:
        codes = torch.empty_like(X, dtype=_E4M3)
        scales = torch.empty(nb, n, dtype=torch.float32, device=X.device)
    else:
        codes, scales = out
        _require(codes, "codes", _E4M3, (n, d))
        _require(scales, "scales", torch.float32, (nb, n))
    _check(lib().fp8_quantize_act(X.data_ptr(), code, n, d, codes.data_ptr(), scales.data_ptr(),
                                  _stream()), "fp8_quantize_act")
    return codes, scales


def fp8_quantize_weight(W: torch.Tensor, out: tuple | None = None):
    """Weights W [d_out, d_in] (fp16/fp32/bf16, d_in a multiple of 16) -> (codes float8_e4m3fn
    [d_out, d_in], scales fp32 [ceil(d_out/128), ceil(d_in/128)]): one scale per 128 x 128
    block."""
    _require(W, "W")
    if W.dim() != 2:
        raise ValueError("W must be [d_out, d_in]")
    d_out, d_in = W.shape
    code = _float_code(W.dtype, "W")
    ns = ((d_out + 127) // 128, (d_in + 127) // 128)
    if out is None:
        codes = torch.empty_like(W, dtype=_E4M3)
        scales = torch.empty(ns, dtype=torch.float32, device=W.device)
    else:
        codes, scales = out
        _require(codes, "codes", _E4M3, (d_out, d_in))
        _require(scales, "scales", torch.float32, ns)
    _check(lib().fp8_quantize_weight(W.data_ptr(), code, d_out, d_in, codes.data_ptr(),
                                     scales.data_ptr(), _stream()), "fp8_quantize_weight")
    return codes, scales


def fp8_linear(X8: torch.Tensor, x_scales: torch.Tensor, W8: torch.Tensor,
               w_scales: torch.Tensor, R: torch.Tensor | None = None,
               out: torch.Tensor | None = None, dtype: torch.dtype = torch.float16,
               status: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X̂·Ŵᵀ + R [n, d_out] (fp16/fp32/bf16) from fp8_quantize_act's and
    fp8_quantize_weight's codes and scales; R has Y's type and may be ``out``. Products of two
    scales are fp32 numbers (include/gptq.h says what that bounds). ``status`` (int32, zeroed by the
    caller): GPTQ_ERR_TIMEOUT if a device-side wait gave up; Y is unspecified then."""
    dev = _device()
    _require(X8, "X8", _E4M3, None, dev)
    _require(W8, "W8", _E4M3, None, dev)
    if X8.dim() != 2 or W8.dim() != 2 or X8.shape[1] != W8.shape[1]:
        raise ValueError("X8 must be [n, d_in] and W8 [d_out, d_in]")
    n, d_in = X8.shape
    d_out = W8.shape[0]
    nb = (d_in + 127) // 128
    _require(x_scales, "x_scales", torch.float32, (nb, n), dev)
    _require(w_scales, "w_scales", torch.float32, ((d_out + 127) // 128, nb), dev)
    if out is None:
        code = _float_code(dtype, "dtype")
        out = torch.empty(n, d_out, dtype=dtype, device=X8.device)
    else:
        _require(out, "out", None, (n, d_out), dev)
        code = _float_code(out.dtype, "out")
    if R is not None:
        _require(R, "R", out.dtype, (n, d_out), dev)
    _require_status(status)
    _check(lib().fp8_linear(X8.data_ptr(), x_scales.data_ptr(), n, d_in, W8.data_ptr(),
                            w_scales.data_ptr(), d_out, _ptr(R), out.data_ptr(), code,
                            _ptr(status), _stream()), "fp8_linear")
    return out


# ------------------------------------------------------------------------------------------
# quantised key/value cache
# ------------------------------------------------------------------------------------------
def kv_cache_alloc(n_pages: int, page_size: int, n_heads: int, head_dim: int, bits: int = 8,
                   group_size: int = 64, device="cuda"):
    """The three arrays of an empty cache: codes uint8 [2, n_pages, page_size, n_heads,
    head_dim*bits/8], scales and zeros fp16 [2, n_pages, page_size, n_heads,
    head_dim/group_size] (keys, then values). A slot that was never written reads as zeros."""
    if bits not in (4, 8) or group_size < 1 or head_dim % group_size:
        raise ValueError("bits must be 4 or 8 and group_size divide head_dim")
    shape = (2, n_pages, page_size, n_heads)
    codes = torch.zeros(*shape, head_dim * bits // 8, dtype=torch.uint8, device=device)
    scales = torch.zeros(*shape, head_dim // group_size, dtype=torch.float16, device=device)
    return codes, scales, torch.zeros_like(scales)


def _cache_dims(codes, scales, zeros, bits, dev):
    """(n_pages, page_size, n_heads, head_dim, group_size) of a cache's arrays, checked."""
    cs, ss = codes.shape, scales.shape
    if len(cs) != 5 or cs[0] != 2 or bits not in (4, 8) or cs[4] < 1:
        raise ValueError("codes must be [2, n_pages, page_size, n_heads, head_dim*bits/8], bits 4 or 8")
    _, n_pages, page_size, n_heads, row = cs
    head_dim = row * 8 // bits
    if len(ss) != 5 or ss[4] < 1 or head_dim % ss[4] or ss[:4] != cs[:4]:
        raise ValueError("scales must be [2, n_pages, page_size, n_heads, head_dim/group_size]")
    _require(codes, "codes", torch.uint8, None, dev)
    _require(scales, "scales", torch.float16, None, dev)
    _require(zeros, "zeros", torch.float16, ss, dev)
    return n_pages, page_size, n_heads, head_dim, head_dim // ss[4]


def _token_stride(t: torch.Tensor, name: str, n_heads: int, head_dim: int, dev: int) -> int:
    """Elements from a token's row to the next; the row itself is contiguous."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if t.dim() != 3 or t.shape[1:] != (n_heads, head_dim):
        raise ValueError(f"{name} must be [n, {n_heads}, {head_dim}]")
    st = t.stride()
    if (st[2] != 1 or (n_heads > 1 and st[1] != head_dim)) and t.numel():
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return st[0] if t.shape[0] > 1 else n_heads * head_dim


def kv_cache_write(K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, codes: torch.Tensor,
                   scales: torch.Tensor, zeros: torch.Tensor, bits: int = 8,
                   status: torch.Tensor | None = None) -> None:
    """Quantise K, V [n, n_heads, head_dim] (fp16/fp32/bf16; rows may lie apart, as in a fused
    projection's output) into the cache's slots [n] int64 (page * page_size + place; negative:
    skipped; distinct). A slot behind the cache is skipped and sets ``status`` to
    GPTQ_ERR_ARG."""
    dev = _device()
    n_pages, page_size, H, D, g = _cache_dims(codes, scales, zeros, bits, dev)
    ks, vs = _token_stride(K, "K", H, D, dev), _token_stride(V, "V", H, D, dev)
    code = _float_code(K.dtype, "K")
    n = K.shape[0]
    if V.dtype is not K.dtype or V.shape[0] != n:
        raise ValueError("V must have K's type and shape")
    _require(slots, "slots", torch.int64, (n,), dev)
    _require_status(status)
    _check(lib().kv_cache_write(K.data_ptr(), V.data_ptr(), code, n, ks, vs, H, D,
                                slots.data_ptr(), n_pages * page_size, bits, g, codes.data_ptr(),
                                scales.data_ptr(), zeros.data_ptr(), _ptr(status), _stream()),
           "kv_cache_write")


def kv_cache_read(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                  page_table: torch.Tensor, cu_lens: torch.Tensor, total: int, bits: int = 8,
                  dtype: torch.dtype = torch.float16, out: tuple | None = None,
                  status: torch.Tensor | None = None):
    """The context of every sequence, packed: (K, V) [total, n_heads, head_dim] of positions
    0 .. len-1 of each sequence in turn. page_table int32 [n_seqs, max_pages], cu_lens int32
    [n_seqs + 1] (running sums of the lengths). Rows behind cu_lens[-1] are left as they were;
    positions without a page of the cache come as zeros and set ``status`` to GPTQ_ERR_ARG. In
    float16, values that come to 65520 or more are infinite (keys near 65504, whose scale was
    rounded up)."""
    dev = _device()
    n_pages, page_size, H, D, g = _cache_dims(codes, scales, zeros, bits, dev)
    _require(page_table, "page_table", torch.int32, None, dev)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_seqs, max_pages]")
    n_seqs, max_pages = page_table.shape
    _require(cu_lens, "cu_lens", torch.int32, (n_seqs + 1,), dev)
    if out is None:
        code = _float_code(dtype, "dtype")
        K = torch.empty(total, H, D, dtype=dtype, device=codes.device)
        V = torch.empty_like(K)
    else:
        K, V = out
        code = _float_code(K.dtype, "K")
        _require(K, "K", None, (total, H, D))
        _require(V, "V", K.dtype, (total, H, D))
    _require_status(status)
    _check(lib().kv_cache_read(codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(), n_pages,
                               page_size, H, D, bits, g, page_table.data_ptr(), n_seqs, max_pages,
                               cu_lens.data_ptr(), total, K.data_ptr(), V.data_ptr(), code,
                               _ptr(status), _stream()), "kv_cache_read")
    return K, V


# ------------------------------------------------------------------------------------------
# stage timing
# ------------------------------------------------------------------------------------------
def profile_enable(on: bool = True) -> None:
    lib().gptq_profile_enable(int(bool(on)))


def profile_read() -> dict:
    buf = (ctypes.c_float * len(STAGES))()
    n = lib().gptq_profile_read(buf, len(STAGES))
    return {STAGES[i]: float(buf[i]) for i in range(n)}


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(lib().gptq_launch_count())


def test_stall_factor(on: bool) -> None:
    """Test hook: make the factorisation's bounded wait run out (see include/gptq.h)."""
    _check(lib().gptq_test_stall_factor(int(bool(on))), "gptq_test_stall_factor")


def test_stall_fp8(rank: int | None) -> None:
    """Test hook: in fp8_linear the producer of each cluster's CTA ``rank`` gives up (None: off; see
    include/gptq.h)."""
    _check(lib().gptq_test_stall_fp8(-1 if rank is None else int(rank)), "gptq_test_stall_fp8")


def test_fp8_no_pair(on: bool) -> None:
    """Test hook: fp8_linear without its kernel for pairs of CTAs (see include/gptq.h)."""
    _check(lib().gptq_test_fp8_no_pair(int(bool(on))), "gptq_test_fp8_no_pair")


def status_string(status: int) -> str:
    return lib().gptq_status_string(status).decode()
