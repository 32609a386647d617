"""Python binding of libkq, the gfx950 KroQuant online activation quantizer.

Thin ctypes layer over the C ABI declared in ``include/kq.h``: each function
has the C entry point's name and only marshals arguments (tensor -> device
pointer, current torch stream -> hipStream_t) and turns a status code into an
exception.  All computation happens in the HIP kernels.  PyTorch supplies
device memory and streams.  There is no fallback: if ``libkq.so`` is missing
or a tensor is not on the GPU, the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = [
    "KQError", "KQ_AUTO", "KQ_MFMA_DENSE", "KQ_MFMA_OTF", "KQ_BUTTERFLY",
    "KQ_FRONT_KRON", "KQ_FRONT_PLAIN", "KQ_FRONT_SMOOTH", "KQ_FRONT_HADAMARD",
    "lib", "kq_abi_version", "kq_status_str", "kq_build_blocks", "kq_quantize", "kq_quantize_ex",
    "kq_mx_quantize", "kq_smooth_quantize", "kq_hadamard_quantize", "kq_transform_f32",
    "alloc_outputs", "LIB_PATH", "kq_auto_variant", "variant_name", "kq_row_stats", "kq_quantize_adaln",
    "kq_build_blocks_inverse_t", "kq_gemm_mx", "kq_hadamard_quantize_ex", "kq_build_blocks16", "kq_tune",
    "kq_tune_reset", "kq_stream_probe", "KQ_ACT_NONE", "KQ_ACT_GELU_TANH", "KQ_ACT_GELU_ERF", "KQ_ACT_SILU",
    "kq_gemm_mx_ex", "alloc_cache", "kq_cache_write", "kq_cache_read", "kq_attention_mx", "kq_attention_mx_workspace",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkq.so")

KQ_AUTO, KQ_MFMA_DENSE, KQ_MFMA_OTF, KQ_BUTTERFLY = 0, 1, 2, 3
KQ_FRONT_KRON, KQ_FRONT_PLAIN, KQ_FRONT_SMOOTH, KQ_FRONT_HADAMARD = 0, 1, 2, 3
KQ_ACT_NONE, KQ_ACT_GELU_TANH, KQ_ACT_GELU_ERF, KQ_ACT_SILU = 0, 1, 2, 3
VARIANTS = {"auto": KQ_AUTO, "mfma_dense": KQ_MFMA_DENSE, "mfma_otf": KQ_MFMA_OTF, "butterfly": KQ_BUTTERFLY}

_lib = None


class KQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kq_status_str(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Load libkq.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} not found: build the HIP library first (__graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.kq_abi_version.argtypes = []
        L.kq_abi_version.restype = ci
        L.kq_status_str.argtypes = [ci]
        L.kq_status_str.restype = ctypes.c_char_p
        L.kq_build_blocks.argtypes = [vp, i64, vp, vp, ci, vp]
        L.kq_quantize.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        L.kq_quantize_ex.argtypes = [vp, i64, i64, vp, i64, vp, ci, vp, vp, vp]
        L.kq_mx_quantize.argtypes = [vp, i64, i64, vp, vp, vp]
        L.kq_stream_probe.argtypes = [vp, i64, i64, vp, vp, vp]
        L.kq_smooth_quantize.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        L.kq_hadamard_quantize.argtypes = [vp, i64, i64, vp, vp, vp]
        L.kq_transform_f32.argtypes = [ci, vp, i64, i64, vp, i64, vp, ci, vp, vp, vp, vp, vp]
        L.kq_auto_variant.argtypes = [i64, i64, ci, ci]
        L.kq_auto_variant.restype = ci
        L.kq_row_stats.argtypes = [vp, i64, i64, ctypes.c_float, vp, vp]
        L.kq_build_blocks_inverse_t.argtypes = [vp, i64, vp, vp, ci, vp]
        L.kq_gemm_mx.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, vp, vp]
        L.kq_hadamard_quantize_ex.argtypes = [vp, i64, i64, ci, vp, vp, vp]
        L.kq_build_blocks16.argtypes = [vp, i64, vp, vp, ci, vp]
        L.kq_tune.argtypes = [vp, i64, i64, vp, vp, vp, vp, ci, ctypes.POINTER(ci), vp]
        L.kq_tune_reset.argtypes = []
        L.kq_tune_reset.restype = None
        L.kq_quantize_adaln.argtypes = [vp, i64, i64, vp, vp, vp, i64, vp, i64, vp, ci, vp, vp, vp]
        cf = ctypes.c_float
        L.kq_gemm_mx_ex.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, ci, vp, i64, vp, vp, vp, vp]
        L.kq_cache_write.argtypes = [vp, i64, vp, i64, i64, i64, vp, i64, vp, vp, vp, vp, vp]
        L.kq_cache_read.argtypes = [vp, vp, vp, vp, i64, i64, vp, i64, vp, i64, vp, i64, vp]
        L.kq_attention_mx.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, i64, vp, i64, i64, vp, i64, i64, i64,
                                      cf, ci, vp, i64, vp, vp, i64, vp]
        L.kq_attention_mx_workspace.argtypes = [i64] * 7
        L.kq_attention_mx_workspace.restype = i64
        for name in ("kq_gemm_mx_ex", "kq_cache_write", "kq_cache_read", "kq_attention_mx"):
            getattr(L, name).restype = ci
        for name in ("kq_build_blocks", "kq_quantize", "kq_quantize_ex", "kq_mx_quantize", "kq_stream_probe",
                     "kq_smooth_quantize",
                     "kq_hadamard_quantize", "kq_transform_f32", "kq_row_stats", "kq_quantize_adaln",
                     "kq_build_blocks_inverse_t", "kq_gemm_mx", "kq_hadamard_quantize_ex", "kq_build_blocks16", "kq_tune"):
            getattr(L, name).restype = ci
        _lib = L
    return _lib


def kq_abi_version() -> int:
    return int(lib().kq_abi_version())


def kq_auto_variant(tokens: int, d: int, has_params: bool = True, has_split: bool = False) -> int:
    return int(lib().kq_auto_variant(tokens, d, int(has_params), int(has_split)))


def variant_name(v: int) -> str:
    return {v_: k for k, v_ in VARIANTS.items()}[int(v)]


def kq_status_str(status: int) -> str:
    return lib().kq_status_str(int(status)).decode()


def _ptr(t, what: str, dtype=None):
    """Device pointer of a tensor (or None / a raw integer address)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{what}: tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    if dtype is not None and t.dtype not in dtype:
        raise TypeError(f"{what}: dtype {t.dtype} not in {dtype}")
    return t.data_ptr()


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_U8 = (torch.uint8,)
_F32 = (torch.float32,)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str):
    if status != 0:
        raise KQError(status, where)


def _shape(X):
    if X.dim() != 2:
        raise ValueError("X must be 2-D [tokens, d]")
    return X.shape[0], X.shape[1]


def alloc_outputs(X: torch.Tensor):
    """Empty (codes [T, d/2] uint8, scales [T, d/32] uint8) on X's device."""
    T, d = _shape(X)
    return (torch.empty((T, d // 2), dtype=torch.uint8, device=X.device),
            torch.empty((T, d // 32), dtype=torch.uint8, device=X.device))


def kq_build_blocks(K_params, nb: int, K_f32=None, K_bf16=None, n_split: int = 3, stream=None):
    _check(lib().kq_build_blocks(_ptr(K_params, "K_params", _F32), nb, _ptr(K_f32, "K_f32", _F32),
                                 _ptr(K_bf16, "K_bf16", _BF16), n_split, _stream(stream)), "kq_build_blocks")
    return K_f32, K_bf16


def kq_quantize(X, K_params, out_codes, out_scales, stream=None):
    T, d = _shape(X)
    _check(lib().kq_quantize(_ptr(X, "X", _BF16), T, d, _ptr(K_params, "K_params", _F32),
                             _ptr(out_codes, "out_codes", _U8), _ptr(out_scales, "out_scales", _U8),
                             _stream(stream)), "kq_quantize")
    return out_codes, out_scales


def kq_quantize_ex(X, K_params, params_block_stride: int, K_bf16, variant: int, out_codes, out_scales,
                   stream=None):
    T, d = _shape(X)
    _check(lib().kq_quantize_ex(_ptr(X, "X", _BF16), T, d, _ptr(K_params, "K_params", _F32),
                                params_block_stride, _ptr(K_bf16, "K_bf16", _BF16), int(variant),
                                _ptr(out_codes, "out_codes", _U8), _ptr(out_scales, "out_scales", _U8),
                                _stream(stream)), "kq_quantize_ex")
    return out_codes, out_scales


def kq_mx_quantize(X, out_codes, out_scales, stream=None):
    T, d = _shape(X)
    _check(lib().kq_mx_quantize(_ptr(X, "X", _BF16), T, d, _ptr(out_codes, "out_codes", _U8),
                                _ptr(out_scales, "out_scales", _U8), _stream(stream)), "kq_mx_quantize")
    return out_codes, out_scales


def kq_stream_probe(X, out_codes, out_scales, stream=None):
    """Measurement only: the default quantizer's memory traffic with no arithmetic (outputs are a digest)."""
    T, d = _shape(X)
    _check(lib().kq_stream_probe(_ptr(X, "X", _BF16), T, d, _ptr(out_codes, "out_codes", _U8),
                                 _ptr(out_scales, "out_scales", _U8), _stream(stream)), "kq_stream_probe")
    return out_codes, out_scales


def kq_smooth_quantize(X, ch_mult, out_codes, out_scales, stream=None):
    T, d = _shape(X)
    _check(lib().kq_smooth_quantize(_ptr(X, "X", _BF16), T, d, _ptr(ch_mult, "ch_mult", _F32),
                                    _ptr(out_codes, "out_codes", _U8), _ptr(out_scales, "out_scales", _U8),
                                    _stream(stream)), "kq_smooth_quantize")
    return out_codes, out_scales


def kq_hadamard_quantize(X, out_codes, out_scales, stream=None):
    T, d = _shape(X)
    _check(lib().kq_hadamard_quantize(_ptr(X, "X", _BF16), T, d, _ptr(out_codes, "out_codes", _U8),
                                      _ptr(out_scales, "out_scales", _U8), _stream(stream)),
           "kq_hadamard_quantize")
    return out_codes, out_scales


def kq_transform_f32(front: int, X, K_params=None, params_block_stride: int = 15, K_bf16=None,
                     variant: int = KQ_AUTO, ch_mult=None, Y=None, out_codes=None, out_scales=None, stream=None):
    T, d = _shape(X)
    _check(lib().kq_transform_f32(int(front), _ptr(X, "X", _BF16), T, d, _ptr(K_params, "K_params", _F32),
                                  params_block_stride, _ptr(K_bf16, "K_bf16", _BF16), int(variant),
                                  _ptr(ch_mult, "ch_mult", _F32), _ptr(Y, "Y", _F32),
                                  _ptr(out_codes, "out_codes", _U8), _ptr(out_scales, "out_scales", _U8),
                                  _stream(stream)), "kq_transform_f32")
    return Y, out_codes, out_scales


def kq_row_stats(X, eps: float, row_stats, stream=None):
    """LayerNorm (mean, rstd) per row into row_stats (float32 [tokens, 2])."""
    T, d = _shape(X)
    _check(lib().kq_row_stats(_ptr(X, "X", _BF16), T, d, float(eps), _ptr(row_stats, "row_stats", _F32),
                              _stream(stream)), "kq_row_stats")
    return row_stats


def kq_quantize_adaln(X, row_stats, mod_scale, mod_shift, tokens_per_sample: int, K_params, out_codes, out_scales,
                      params_block_stride: int = 15, K_bf16=None, variant: int = KQ_AUTO, stream=None):
    """Fused LayerNorm-normalise + AdaLN-modulate + transform + MXFP4 (any of the first three inputs may be None)."""
    T, d = _shape(X)
    _check(lib().kq_quantize_adaln(_ptr(X, "X", _BF16), T, d, _ptr(row_stats, "row_stats", _F32),
                                   _ptr(mod_scale, "mod_scale", _F32), _ptr(mod_shift, "mod_shift", _F32),
                                   int(tokens_per_sample), _ptr(K_params, "K_params", _F32), params_block_stride,
                                   _ptr(K_bf16, "K_bf16", _BF16), int(variant), _ptr(out_codes, "out_codes", _U8),
                                   _ptr(out_scales, "out_scales", _U8), _stream(stream)), "kq_quantize_adaln")
    return out_codes, out_scales


def kq_build_blocks_inverse_t(K_params, nb: int, K_f32=None, K_bf16=None, n_split: int = 3, stream=None):
    """Blocks K^-T of the weight fold (fp32 [nb,32,32] and/or transposed bf16 split [nb,n_split,32,32])."""
    _check(lib().kq_build_blocks_inverse_t(_ptr(K_params, "K_params", _F32), nb, _ptr(K_f32, "K_f32", _F32),
                                           _ptr(K_bf16, "K_bf16", _BF16), n_split, _stream(stream)),
           "kq_build_blocks_inverse_t")
    return K_f32, K_bf16


def kq_gemm_mx(a_codes, a_scales, b_codes, b_scales, y_f32=None, y_bf16=None, stream=None):
    """Y = deq(A) deq(B)^T: A codes [M, K/2] + scales [M, K/32], B codes [N, K/2] + scales [N, K/32]."""
    M, N = a_codes.shape[0], b_codes.shape[0]
    K = a_codes.shape[1] * 2
    if b_codes.shape[1] * 2 != K:
        raise ValueError("A and B must have the same K")
    _check(lib().kq_gemm_mx(_ptr(a_codes, "a_codes", _U8), _ptr(a_scales, "a_scales", _U8), M,
                            _ptr(b_codes, "b_codes", _U8), _ptr(b_scales, "b_scales", _U8), N, K,
                            _ptr(y_f32, "y_f32", _F32), _ptr(y_bf16, "y_bf16", _BF16), _stream(stream)),
           "kq_gemm_mx")
    return y_f32, y_bf16


def kq_hadamard_quantize_ex(X, block: int, out_codes, out_scales, stream=None):
    """Block-Hadamard (size 32..512) front-end + MXFP4."""
    T, d = _shape(X)
    _check(lib().kq_hadamard_quantize_ex(_ptr(X, "X", _BF16), T, d, int(block), _ptr(out_codes, "out_codes", _U8),
                                         _ptr(out_scales, "out_scales", _U8), _stream(stream)), "kq_hadamard_quantize_ex")
    return out_codes, out_scales


def kq_build_blocks16(K_params16, nb16: int, K_f32=None, K_bf16=None, n_split: int = 3, stream=None):
    """16-wide 4-factor blocks as block-diagonal 32x32 dense blocks (fp32 and/or transposed bf16 split)."""
    _check(lib().kq_build_blocks16(_ptr(K_params16, "K_params16", _F32), nb16, _ptr(K_f32, "K_f32", _F32),
                                   _ptr(K_bf16, "K_bf16", _BF16), n_split, _stream(stream)), "kq_build_blocks16")
    return K_f32, K_bf16


def kq_tune(X, K_params, K_bf16, out_codes, out_scales, reps: int = 10, stream=None) -> int:
    """Time the variants the inputs allow, record the fastest for KQ_AUTO at this shape; returns it."""
    T, d = _shape(X)
    chosen = ctypes.c_int(0)
    _check(lib().kq_tune(_ptr(X, "X", _BF16), T, d, _ptr(K_params, "K_params", _F32), _ptr(K_bf16, "K_bf16", _BF16),
                         _ptr(out_codes, "out_codes", _U8), _ptr(out_scales, "out_scales", _U8), int(reps),
                         ctypes.byref(chosen), _stream(stream)), "kq_tune")
    return chosen.value


def kq_tune_reset() -> None:
    lib().kq_tune_reset()


# The entry points below take strided rows, tables and several optional tensors: their tensors are checked
# against one another here (the C ABI sees only addresses), have to be on one device, and run on that device.

def _wrong_place(t, what: str, dev: int):
    if not t.is_cuda:
        raise ValueError(f"{what}: tensor must be on the GPU")
    raise ValueError(f"{what}: tensor on {t.device}, others on cuda:{dev}")


def _device(t, what: str) -> int:
    """Index of the GPU that a tensor is on."""
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{what}: tensor must be on the GPU")
    return dev


def _rows(t, what: str, width: int, rows: int, dev: int):
    """Address and row stride of a bf16 matrix [rows, width] on GPU `dev` whose rows are contiguous."""
    if t.get_device() != dev:
        _wrong_place(t, what, dev)
    if t.dtype not in _BF16:
        raise TypeError(f"{what}: dtype {t.dtype} not in {_BF16}")
    if t.shape != (rows, width):
        raise ValueError(f"{what}: expected [{rows}, {width}], got {list(t.shape)}")
    stride, step = t.stride()
    if step != 1 and width > 1:
        raise ValueError(f"{what}: rows must be contiguous")
    return t.data_ptr(), stride if rows > 1 else width


def _full(t, what: str, dtype, shape, dev: int):
    """Address of a contiguous tensor of this type and shape on GPU `dev` (None stays None)."""
    if t is None:
        return None
    if t.get_device() != dev:
        _wrong_place(t, what, dev)
    if t.dtype not in dtype:
        raise TypeError(f"{what}: dtype {t.dtype} not in {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous {list(shape)}, got {list(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _call(fn, where: str, dev: int, stream, *args):
    """fn(*args, stream) on GPU `dev` (its tensors are there): that GPU's current stream, or the one given."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _call(fn, where, dev, stream, *args)
    status = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status:
        raise KQError(status, where)


def _stream_object(stream, dev: int):
    """The torch stream of a `stream` argument.  Address 0 is the default stream; an ExternalStream of it would be
    another one, of torch's pool."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), dev) if int(stream) else torch.cuda.default_stream(dev)


_I32 = (torch.int32,)
_PAGE = 1 << 24  # slots of a page at most


def kq_gemm_mx_ex(a_codes, a_scales, b_codes, b_scales, bias=None, act: int = KQ_ACT_NONE, gate=None,
                  rows_per_sample: int | None = None, residual=None, y_f32=None, y_bf16=None, stream=None):
    """Y = residual + gate[m // rows_per_sample] * act(deq(A) deq(B)^T + bias); any of the three may be None.

    bias float32 [N], gate float32 [samples, N] (rows_per_sample defaults to M: one sample), residual bfloat16
    [M, N], which may be y_bf16 itself."""
    M, half = a_codes.shape
    N = b_codes.shape[0]
    K = half * 2
    rps = M if rows_per_sample is None else int(rows_per_sample)
    if gate is not None and rps <= 0 < M:
        raise ValueError("rows_per_sample must be positive")
    dev = _device(a_codes, "a_codes")
    _call(lib().kq_gemm_mx_ex, "kq_gemm_mx_ex", dev, stream,
          _full(a_codes, "a_codes", _U8, (M, half), dev), _full(a_scales, "a_scales", _U8, (M, K // 32), dev), M,
          _full(b_codes, "b_codes", _U8, (N, half), dev), _full(b_scales, "b_scales", _U8, (N, K // 32), dev), N, K,
          _full(bias, "bias", _F32, (N,), dev), act,
          None if gate is None else _full(gate, "gate", _F32, (-(-M // rps) if M else gate.shape[0], N), dev), rps or 1,
          _full(residual, "residual", _BF16, (M, N), dev), _full(y_f32, "y_f32", _F32, (M, N), dev),
          _full(y_bf16, "y_bf16", _BF16, (M, N), dev))
    return y_f32, y_bf16


def alloc_cache(n_slots: int, width: int, device="cuda"):
    """An empty MXFP4 key/value cache: (k_codes, k_scales, v_codes, v_scales), zeros."""
    def zeros(w):
        return torch.zeros((n_slots, w), dtype=torch.uint8, device=device)
    return zeros(width // 2), zeros(width // 32), zeros(width // 2), zeros(width // 32)


def _cache(k_codes, k_scales, v_codes, v_scales, width: int, dev: int, both: bool = True):
    """(n_slots, four addresses) of a cache's pools; the values' are None without `both`."""
    n = k_codes.shape[0]
    codes, scales = (n, width // 2), (n, width // 32)
    k, ks = _full(k_codes, "k_codes", _U8, codes, dev), _full(k_scales, "k_scales", _U8, scales, dev)
    if not both:
        return n, (k, ks, None, None)
    return n, (k, ks, _full(v_codes, "v_codes", _U8, codes, dev), _full(v_scales, "v_scales", _U8, scales, dev))


def _cache_rows(K, V, slots, dev: int):
    T, W = K.shape
    k, ks = _rows(K, "K", W, T, dev)
    v, vs = (None, W) if V is None else _rows(V, "V", W, T, dev)
    return T, W, k, ks, v, vs, _full(slots, "slots", _I32, (T,), dev)


def kq_cache_write(K, V, slots, k_codes, k_scales, v_codes, v_scales, stream=None):
    """Quantize rows of K and V (bfloat16 [tokens, width], V may be None) to MXFP4 and write them to their slots
    (int32 [tokens], outside the cache: not written)."""
    dev = _device(K, "K")
    T, W, k, ks, v, vs, at = _cache_rows(K, V, slots, dev)
    n, pools = _cache(k_codes, k_scales, v_codes, v_scales, W, dev, V is not None)
    _call(lib().kq_cache_write, "kq_cache_write", dev, stream, k, ks, v, vs, T, W, at, n, *pools)
    return k_codes, k_scales, v_codes, v_scales


def kq_cache_read(k_codes, k_scales, v_codes, v_scales, slots, K, V, stream=None):
    """The values of slots (int32 [tokens], outside the cache: zeros) into K and V (bfloat16 [tokens, width], V may
    be None)."""
    dev = _device(K, "K")
    T, W, k, ks, v, vs, at = _cache_rows(K, V, slots, dev)
    n, pools = _cache(k_codes, k_scales, v_codes, v_scales, W, dev, V is not None)
    _call(lib().kq_cache_read, "kq_cache_read", dev, stream, *pools, n, W, at, T, k, ks, v, vs)
    return K, V


@functools.lru_cache(maxsize=1024)
def kq_attention_mx_workspace(q_rows: int, batch: int, max_q: int, q_heads: int, kv_heads: int, head_dim: int,
                              capacity: int) -> int:
    """Bytes of workspace that kq_attention_mx needs (0: none)."""
    return int(lib().kq_attention_mx_workspace(q_rows, batch, max_q, q_heads, kv_heads, head_dim, capacity))


def kq_attention_mx(Q, k_codes, k_scales, v_codes, v_scales, kv_len, out, q_heads: int, kv_heads: int,
                    page_size: int | None = None, pages_per_seq: int | None = None, page_table=None, q_start=None,
                    max_q: int | None = None, scale: float | None = None, causal: bool = False, lse=None,
                    workspace=None, stream=None):
    """Attention of Q (bfloat16 [q_rows, q_heads * head_dim]) over an MXFP4 cache into out (as Q) and lse (float32
    [q_rows, q_heads], or None).

    kv_len int32 [batch]; page_table int32 [batch, pages_per_seq], or None: the sequences' slots in order, of
    pages_per_seq * page_size each (by default an equal share of the cache).  q_start int32 [batch + 1], or None: max_q
    rows each (by default an equal share).  With q_start, max_q bounds its differences: pass it, for the call is divided
    by it (all rows, the default, is right and slow: each sequence then has room for every row).  scale defaults to
    head_dim ** -0.5.  workspace (uint8, kq_attention_mx_workspace bytes) is allocated for the call if None."""
    rows, width = Q.shape
    batch = kv_len.shape[0]
    if q_heads < 1 or width % q_heads:
        raise ValueError(f"Q: {width} columns are not {q_heads} heads")
    dim = width // q_heads
    dev = _device(Q, "Q")
    n, pools = _cache(k_codes, k_scales, v_codes, v_scales, kv_heads * dim, dev)
    if page_table is not None:
        pages_per_seq = page_table.shape[1]
        if page_size is None:
            raise ValueError("page_size is needed with a page_table")
    elif page_size is None:  # one page each, or, of more slots than a page may have, a page a slot; no slots: no pages
        share = n // max(1, batch)
        page_size, pages_per_seq = (share, 1) if 0 < share <= _PAGE else (1, share)
    elif pages_per_seq is None:
        pages_per_seq = n // page_size // max(1, batch)
    if max_q is None:
        max_q = rows // max(1, batch) if q_start is None else rows
    q, qs = _rows(Q, "Q", width, rows, dev)
    o, os_ = _rows(out, "out", width, rows, dev)
    need = kq_attention_mx_workspace(rows, batch, max_q, q_heads, kv_heads, dim, pages_per_seq * page_size)
    if workspace is None and need:
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
        else:  # memory of the stream that uses it, so that its reuse waits for this call
            with torch.cuda.stream(_stream_object(stream, dev)):
                workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    wbytes = 0 if workspace is None else workspace.numel()
    _call(lib().kq_attention_mx, "kq_attention_mx", dev, stream, q, qs, rows,
          _full(q_start, "q_start", _I32, (batch + 1,), dev), batch, max_q, *pools, n,
          _full(page_table, "page_table", _I32, (batch, pages_per_seq), dev), pages_per_seq, page_size,
          _full(kv_len, "kv_len", _I32, (batch,), dev), q_heads, kv_heads, dim, dim ** -0.5 if scale is None else scale,
          causal, o, os_, _full(lse, "lse", _F32, (rows, q_heads), dev),
          _full(workspace, "workspace", _U8, (wbytes,), dev), wbytes)
    return out, lse
