"""Python binding of the sm_100a hybrid dense / 2:4 linear layer (PATCH).

Argument marshalling only: every step of the layer runs in the CUDA kernels of
``libpatch_hybrid.so`` (the C ABI declared in ``include/patch_hybrid.h``).
PyTorch supplies device memory and streams. If the library is missing this
module raises on import, and the 8-bit calls raise without the extension that
marshals them; there is no fallback.

    import hybrid_sparse_gemm_b200 as hsg
    lin = hsg.PackedLinear.pack(W, mask_bits, tile_flags, tile_rows=128, tile_cols=128)
    Y = lin(X)                       # Y = X @ (W * mask).T, bf16

The same tiles in 8-bit integers, one scale per token and per output channel:

    lin = hsg.PackedLinearQ8.pack(W, mask_bits, tile_flags)
    qkv = hsg.LinearGroupQ8([q, k, v])
    (Yq, Yk, Yv), h = qkv.norm(x, gamma, eps, residual=h)   # RMS norm -> codes -> one launch
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("PATCH_HYBRID_LIB") or os.path.join(_HERE, "libpatch_hybrid.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m hybrid_sparse_gemm_b200.build`")

_lib = ctypes.CDLL(LIB_PATH)

PATCH_OK = 0
STATUS_NAMES = {0: "PATCH_OK", 1: "PATCH_ERR_ARG", 2: "PATCH_ERR_SHAPE", 3: "PATCH_ERR_ALIGN",
                4: "PATCH_ERR_MASK", 5: "PATCH_ERR_CUDA", 6: "PATCH_ERR_TIMEOUT",
                7: "PATCH_ERR_NOMEM", 8: "PATCH_ERR_UNSUPPORTED"}
PATH_AUTO, PATH_GEMM, PATH_GEMV, PATH_GEMM_SINGLE, PATH_GEMM_PAIR, PATH_GEMV_SIMT, PATH_GEMM_WIDE = 0, 1, 2, 3, 4, 5, 6
PATH_GEMM_WIDE_24 = 7

EXPORTED = ["patch_pack", "patch_linear", "patch_linear_path", "patch_linear_host", "patch_unpack",
            "patch_info", "patch_copy_packed", "patch_check", "patch_free", "patch_last_error",
            "patch_version", "patch_plan", "patch_linear_noalloc", "patch_group_create",
            "patch_group_linear", "patch_group_path", "patch_group_free", "patch_selftest_wait",
            "patch_partition_rows", "patch_classify_tiles", "patch_group_linear_host", "patch_plan_pairs",
            "patch_pack_q8", "patch_linear_q8", "patch_group_linear_q8", "patch_unpack_q8",
            "patch_quantize_q8", "patch_rmsnorm_q8", "patch_silu_mul_q8", "patch_dequantize_q8"]
TYPE_BF16, TYPE_FP16, TYPE_FP32, TYPE_INT8 = 0, 1, 2, 3


class patch_info_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("tile_rows", ctypes.c_int32), ("tile_cols", ctypes.c_int32),
                ("tiles_total", ctypes.c_int64), ("tiles_sparse", ctypes.c_int64),
                ("slabs_total", ctypes.c_int64), ("slabs_sparse", ctypes.c_int64),
                ("slabs_pair_sparse", ctypes.c_int64), ("meta_blocks", ctypes.c_int64),
                ("dense_images", ctypes.c_int64), ("packed_bytes", ctypes.c_int64), ("pruned", ctypes.c_int64),
                ("stray_zeros", ctypes.c_int64), ("sparsity", ctypes.c_double)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_lib.patch_pack.argtypes = [_P, _I64, _I64, _P, _I, _P, _I, _I, _P, ctypes.POINTER(_P)]
_lib.patch_linear.argtypes = [_P, _P, _I64, _P, _P]
_lib.patch_linear_path.argtypes = [_P, _P, _I64, _P, _I, _P]
_lib.patch_linear_host.argtypes = [_P, _P, _I64, _P, _P]
_lib.patch_linear_noalloc.argtypes = [_P, _P, _I64, _P, _P]
_lib.patch_group_create.argtypes = [_P, _I, ctypes.POINTER(_P)]
_lib.patch_group_linear.argtypes = [_P, _P, _I64, _P, _I, _P]
_lib.patch_group_linear_host.argtypes = [_P, _P, _I64, _P, _I, _P]
_lib.patch_group_path.argtypes = [_P, _I64, _I, ctypes.POINTER(_I)]
_lib.patch_group_free.argtypes = [_P]
_lib.patch_selftest_wait.argtypes = [_P]
_lib.patch_group_free.restype = None
_lib.patch_unpack.argtypes = [_P, _P, _P]
_lib.patch_info.argtypes = [_P, ctypes.POINTER(patch_info_t)]
_lib.patch_copy_packed.argtypes = [_P, _P, _I64, _P, _I64, _P, _I64, _P, _I64]
_lib.patch_check.argtypes = [_P, _P]
_lib.patch_plan.argtypes = [_I64, _I64, _P, _I, _I, _P, _P, _P, ctypes.POINTER(_I64)]
_lib.patch_plan_pairs.argtypes = [_I64, _I64, _P, _I, _I, _P]
_lib.patch_partition_rows.argtypes = [_I64, _I64, _P, _I, _I, _I, _I64, _P]
_lib.patch_classify_tiles.argtypes = [_P, _I64, _I64, _I, _I, _P, ctypes.POINTER(_I64)]
_F = ctypes.c_float
_lib.patch_pack_q8.argtypes = [_P, _I, _P, _I64, _I64, _P, _I, _P, _I, _I, _P, ctypes.POINTER(_P)]
_lib.patch_linear_q8.argtypes = [_P, _P, _I64, _P, _I64, _P, _I64, _I, _I, _P]
_lib.patch_group_linear_q8.argtypes = [_P, _P, _P, _P, _I64, _P, _P, _I, _I, _P]
_lib.patch_unpack_q8.argtypes = [_P, _P, _P, _P]
_lib.patch_quantize_q8.argtypes = [_P, _I64, _I, _I64, _I64, _P, _I64, _P, _P]
_lib.patch_rmsnorm_q8.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _I, _F, _I64, _I64, _P, _I64, _P, _P]
_lib.patch_silu_mul_q8.argtypes = [_P, _I64, _P, _I64, _I, _I64, _I64, _P, _I64, _P, _P]
_lib.patch_dequantize_q8.argtypes = [_P, _I64, _P, _I64, _I64, _P, _I64, _I, _P]
_lib.patch_free.argtypes = [_P]
_lib.patch_free.restype = None
_lib.patch_last_error.restype = ctypes.c_char_p
_lib.patch_version.restype = ctypes.c_int
for _n in ["patch_pack", "patch_linear", "patch_linear_path", "patch_linear_host", "patch_unpack",
           "patch_info", "patch_copy_packed", "patch_check", "patch_plan", "patch_linear_noalloc",
           "patch_group_create", "patch_group_linear", "patch_partition_rows", "patch_classify_tiles",
           "patch_group_linear_host", "patch_plan_pairs", "patch_pack_q8", "patch_linear_q8",
           "patch_group_linear_q8", "patch_unpack_q8", "patch_quantize_q8", "patch_rmsnorm_q8",
           "patch_silu_mul_q8", "patch_dequantize_q8"]:
    getattr(_lib, _n).restype = ctypes.c_int


class _NoBinding:
    """In the place of the extension that marshals the 8-bit calls, where it is not
    built for this interpreter: those calls raise, the others do not need it."""

    def __init__(self, why: ImportError):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{_HERE}/_binding.*.so is missing or does not load: build it with "
                          "`python hybrid_sparse_gemm_b200/build.py`") from self._why


try:
    from . import _binding
    _binding.init((torch.bfloat16, torch.float16, torch.float32, torch.int8), torch.cuda.current_device,
                  getattr(torch._C, "_cuda_getCurrentRawStream", None),
                  tuple(ctypes.cast(getattr(_lib, n), _P).value for n in
                        ("patch_linear_q8", "patch_quantize_q8", "patch_rmsnorm_q8", "patch_silu_mul_q8",
                         "patch_dequantize_q8", "patch_group_linear_q8")))
except ImportError as e:
    _binding = _NoBinding(e)


class PatchError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(status: int):
    if status != PATCH_OK:
        raise PatchError(status, _lib.patch_last_error().decode())


def _stream(stream) -> int:
    if stream is None:
        # the current stream's handle, without building a Stream object (3 us of a 5 us call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def library() -> ctypes.CDLL:
    return _lib


def version() -> int:
    return _lib.patch_version()


# ---- thin functions with the C ABI's names -----------------------------------

def _table_sizes(N: int, K: int):
    S, KB = N // 128, K // 64
    return S * KB, S * ((KB + 1) // 2), S * KB


def patch_plan(N: int, K: int, tile_flags, tile_rows: int = 128, tile_cols: int = 128):
    """Host-only: ((slab, meta, gemm) tables as uint32 numpy arrays, packed byte count)."""
    import numpy as np
    flags = np.ascontiguousarray(np.asarray(tile_flags, dtype=np.uint8).reshape(-1))
    ok = N > 0 and K > 0 and N % 128 == 0 and K % 64 == 0
    ns, nm, ng = _table_sizes(N, K) if ok else (0, 0, 0)
    slab, meta, gemm = (np.zeros(max(n, 1), np.uint32) for n in (ns, nm, ng))
    nbytes = _I64(0)
    _check(_lib.patch_plan(N, K, flags.ctypes.data, tile_rows, tile_cols, slab.ctypes.data,
                           meta.ctypes.data, gemm.ctypes.data, ctypes.byref(nbytes)))
    return (slab[:ns], meta[:nm], gemm[:ng]), int(nbytes.value)


def patch_plan_pairs(N: int, K: int, tile_flags, tile_rows: int = 128, tile_cols: int = 128):
    """Host-only: the strip order of the CTA-pair kernels as an int32 numpy
    array of N/128 entries (pair i = strips order[2i], order[2i+1])."""
    import numpy as np
    flags = np.ascontiguousarray(np.asarray(tile_flags, dtype=np.uint8).reshape(-1))
    S = N // 128 if N > 0 and N % 128 == 0 else 0
    order = np.zeros(max(S, 1), np.int32)
    _check(_lib.patch_plan_pairs(N, K, flags.ctypes.data, tile_rows, tile_cols, order.ctypes.data))
    return order[:S]


def patch_classify_tiles(mask_bits, N: int, K: int, tile_rows: int = 128, tile_cols: int = 128):
    """Host-only: (tile flags as a uint8 numpy array [N/tile_rows, K/tile_cols],
    number of dense tiles that prune some weight) for a bit-packed mask."""
    import numpy as np
    bits = mask_bits.cpu().numpy() if isinstance(mask_bits, torch.Tensor) else np.asarray(mask_bits)
    bits = np.ascontiguousarray(bits.reshape(-1), dtype=np.uint8)
    if bits.size != (N * K + 7) // 8:
        raise ValueError(f"mask_bits has {bits.size} bytes, a {N}x{K} mask needs {(N * K + 7) // 8}")
    ok = tile_rows > 0 and tile_cols > 0 and N > 0 and K > 0 and N % tile_rows == 0 and K % tile_cols == 0
    flags = np.zeros(max((N // tile_rows) * (K // tile_cols) if ok else 1, 1), np.uint8)
    stray = _I64(0)
    _check(_lib.patch_classify_tiles(bits.ctypes.data, N, K, tile_rows, tile_cols, flags.ctypes.data,
                                     ctypes.byref(stray)))
    return flags.reshape(N // tile_rows, K // tile_cols), int(stray.value)


def patch_partition_rows(N: int, K: int, tile_flags, parts: int, tile_rows: int = 128, tile_cols: int = 128,
                         align_rows: int = 256) -> list[int]:
    """Host-only: parts + 1 row bounds of a cost-balanced contiguous split of W."""
    import numpy as np
    flags = np.ascontiguousarray(np.asarray(tile_flags, dtype=np.uint8).reshape(-1))
    if tile_rows > 0 and tile_cols > 0 and N % tile_rows == 0 and K % tile_cols == 0 and N > 0 and K > 0:
        if flags.size != (N // tile_rows) * (K // tile_cols):
            raise ValueError(f"tile_flags has {flags.size} entries, the {N}x{K} weight has "
                             f"{(N // tile_rows) * (K // tile_cols)} tiles")
    bounds = np.zeros(max(parts, 0) + 1, np.int64)
    _check(_lib.patch_partition_rows(N, K, flags.ctypes.data, tile_rows, tile_cols, parts, align_rows,
                                     bounds.ctypes.data))
    return [int(b) for b in bounds]


def patch_pack(W: torch.Tensor, mask_bits: torch.Tensor, tile_flags, tile_rows: int = 128,
               tile_cols: int = 128, bitorder: int = 0, stream=None) -> int:
    """Returns an opaque handle (int). W bf16 [N,K] and mask_bits uint8 on the
    device; tile_flags uint8 on the host (any array-like)."""
    assert W.is_cuda and W.dtype == torch.bfloat16 and W.dim() == 2 and W.is_contiguous()
    assert mask_bits.is_cuda and mask_bits.dtype == torch.uint8 and mask_bits.is_contiguous()
    flags = torch.as_tensor(tile_flags, dtype=torch.uint8).reshape(-1).contiguous().cpu()
    N, K = W.shape
    h = _P()
    _check(_lib.patch_pack(W.data_ptr(), N, K, mask_bits.data_ptr(), bitorder, flags.data_ptr(),
                           tile_rows, tile_cols, _stream(stream), ctypes.byref(h)))
    return h.value


def patch_linear_path(h: int, X: torch.Tensor, Y: torch.Tensor, path: int = PATH_AUTO, stream=None):
    _check(_lib.patch_linear_path(h, X.data_ptr(), X.shape[0], Y.data_ptr(), path, _stream(stream)))


def patch_linear(h: int, X: torch.Tensor, Y: torch.Tensor, stream=None):
    _check(_lib.patch_linear(h, X.data_ptr(), X.shape[0], Y.data_ptr(), _stream(stream)))


def patch_linear_noalloc(h: int, X: torch.Tensor, Y: torch.Tensor, stream=None):
    """patch_linear that allocates no device memory (see the header)."""
    _check(_lib.patch_linear_noalloc(h, X.data_ptr(), X.shape[0], Y.data_ptr(), _stream(stream)))


def patch_linear_host(h: int, X: torch.Tensor, Y: torch.Tensor, stream=None):
    """X, Y are CPU tensors (pinned for speed); synchronous."""
    assert not X.is_cuda and not Y.is_cuda
    _check(_lib.patch_linear_host(h, X.data_ptr(), X.shape[0], Y.data_ptr(), _stream(stream)))


def patch_unpack(h: int, out: torch.Tensor, stream=None):
    _check(_lib.patch_unpack(h, out.data_ptr(), _stream(stream)))


def patch_info(h: int) -> patch_info_t:
    info = patch_info_t()
    _check(_lib.patch_info(h, ctypes.byref(info)))
    return info


def patch_copy_packed(h: int):
    """(packed bytes as a uint8 numpy array, (slab, meta, gemm) uint32 tables)."""
    import numpy as np
    info = patch_info(h)
    ns = ng = int(info.slabs_total)
    nm = int(info.N) // 128 * ((int(info.K) + 127) // 128)  # 128 columns a block, of bf16 weights and of 8-bit codes
    packed = np.empty(int(info.packed_bytes), np.uint8)
    slab, meta, gemm = np.empty(ns, np.uint32), np.empty(nm, np.uint32), np.empty(ng, np.uint32)
    _check(_lib.patch_copy_packed(h, packed.ctypes.data, packed.size, slab.ctypes.data, ns,
                                  meta.ctypes.data, nm, gemm.ctypes.data, ng))
    return packed, (slab, meta, gemm)


def patch_check(h: int, stream=None):
    _check(_lib.patch_check(h, _stream(stream)))


def patch_free(h: int):
    _lib.patch_free(h)


# ---- 8-bit integers ----------------------------------------------------------

def _on_device(*tensors):
    """Every tensor on the current CUDA device, where the calls launch."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensor on {t.device}, the current device is cuda:{dev}")


def _scales(name: str, t: torch.Tensor, n: int):
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} is {t.dtype}, not torch.float32")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be {n} contiguous scales")


def patch_pack_q8(W: torch.Tensor, mask_bits: torch.Tensor, tile_flags, tile_rows: int = 128, tile_cols: int = 128,
                  bitorder: int = 0, w_scale: torch.Tensor | None = None, stream=None) -> int:
    """Returns an opaque handle (int). W [N,K] on the device: bf16, quantised per
    output channel, or int8 codes with their fp32 scales w_scale [N]."""
    if W.dim() != 2 or not W.is_contiguous() or W.dtype not in (torch.bfloat16, torch.int8):
        raise TypeError("W must be a contiguous 2-D bf16 or int8 tensor")
    if mask_bits.dtype != torch.uint8 or not mask_bits.is_contiguous():
        raise TypeError("mask_bits must be a contiguous uint8 tensor")
    N, K = W.shape
    if mask_bits.numel() != (N * K + 7) // 8:
        raise ValueError(f"mask_bits has {mask_bits.numel()} bytes, a {N}x{K} mask needs {(N * K + 7) // 8}")
    if w_scale is not None:
        _scales("w_scale", w_scale, N)
    _on_device(W, mask_bits, w_scale)
    flags = torch.as_tensor(tile_flags, dtype=torch.uint8).reshape(-1).contiguous().cpu()
    if tile_rows > 0 and tile_cols > 0 and N % tile_rows == 0 and K % tile_cols == 0 and \
            flags.numel() != (N // tile_rows) * (K // tile_cols):
        raise ValueError(f"tile_flags has {flags.numel()} entries, the {N}x{K} weight has "
                         f"{(N // tile_rows) * (K // tile_cols)} tiles")
    h = _P()
    _check(_lib.patch_pack_q8(W.data_ptr(), TYPE_BF16 if W.dtype == torch.bfloat16 else TYPE_INT8,
                              None if w_scale is None else w_scale.data_ptr(), N, K, mask_bits.data_ptr(), bitorder,
                              flags.data_ptr(), tile_rows, tile_cols, _stream(stream), ctypes.byref(h)))
    return h.value


def patch_linear_q8(h: int, X: torch.Tensor, x_scale: torch.Tensor, Y: torch.Tensor, path: int = PATH_AUTO, stream=None):
    """Y [M,N] (bf16, fp16 or fp32) from the codes X [M,K] and their scales [M]."""
    for t in (X, x_scale, Y):
        if not t.is_cuda:
            raise ValueError(f"tensor on {t.device}, not on the current CUDA device")
    info = patch_info(h)
    if X.dim() == 2 and Y.dim() == 2 and (X.shape[1] != info.K or Y.shape[1] != info.N):
        raise PatchError(2, f"X has {X.shape[1]} columns and Y {Y.shape[1]}, the weight is {info.N}x{info.K}")
    _check(_binding.linear_q8(h, info.N, info.K, X, x_scale, Y, path, stream))


def patch_unpack_q8(h: int, W: torch.Tensor, w_scale: torch.Tensor, stream=None):
    """The masked codes W [N,K] (int8) and the channel scales w_scale [N] (fp32) of a handle."""
    _check(_lib.patch_linear_q8(h, None, 0, None, 0, None, 0, TYPE_BF16, PATH_AUTO, None))  # no tokens: is it an 8-bit handle
    info = patch_info(h)
    if W.dtype is not torch.int8:
        raise TypeError(f"W is {W.dtype}, not torch.int8")
    if W.shape != (info.N, info.K) or not W.is_contiguous():
        raise ValueError(f"W must be contiguous {info.N}x{info.K} codes")
    _scales("w_scale", w_scale, info.N)
    _on_device(W, w_scale)
    _check(_lib.patch_unpack_q8(h, W.data_ptr(), w_scale.data_ptr(), _stream(stream)))


def patch_quantize_q8(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, stream=None):
    """Codes q [M,K] (int8) and scales [M] (fp32) of the rows of x."""
    _check(_binding.quantize_q8(x, q, scale, stream))


def patch_rmsnorm_q8(x: torch.Tensor, gamma: torch.Tensor, eps: float, q: torch.Tensor, scale: torch.Tensor,
                     residual: torch.Tensor | None = None, residual_out: torch.Tensor | None = None, stream=None):
    """Codes and scales of the RMS norm of x, or of x + residual, which is then
    written to residual_out (which may be x or residual itself)."""
    _check(_binding.rmsnorm_q8(x, gamma, eps, q, scale, residual, residual_out, stream))


def patch_silu_mul_q8(gate: torch.Tensor, up: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, stream=None):
    """Codes and scales of silu(gate) * up."""
    _check(_binding.silu_mul_q8(gate, up, q, scale, stream))


def patch_dequantize_q8(q: torch.Tensor, scale: torch.Tensor, out: torch.Tensor, stream=None):
    """out = q * scale, row by row (bf16, fp16 or fp32)."""
    _check(_binding.dequantize_q8(q, scale, out, stream))


def _empty(shape, dtype, device, stream):
    """Memory for a call on `stream`: from that stream's pool, so that no earlier or
    later owner of the same memory on another stream overlaps the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    raw = _stream(stream)
    with torch.cuda.stream(torch.cuda.ExternalStream(raw) if raw else torch.cuda.default_stream()):
        return torch.empty(shape, dtype=dtype, device=device)


def _codes_like(x: torch.Tensor, stream):
    """Fresh (codes, scales) for the rows of x; the codes' pitch suits the products."""
    M, K = x.shape
    pitch = (K + 15) // 16 * 16
    q = _empty((M, pitch), torch.int8, x.device, stream)
    return q if pitch == K else q[:, :K], _empty(M, torch.float32, x.device, stream)


class LinearGroup:
    """Several packed linears run with one launch (they share M)."""

    def __init__(self, linears):
        self.linears = list(linears)
        arr = (_P * len(self.linears))(*[l.handle for l in self.linears])
        g = _P()
        _check(_lib.patch_group_create(arr, len(self.linears), ctypes.byref(g)))
        self.handle = g.value

    def __call__(self, Xs, outs=None, path: int = PATH_AUTO, stream=None):
        n = len(self.linears)
        assert len(Xs) == n
        M = Xs[0].shape[0]
        if outs is None:
            outs = [torch.empty((M, l.N), dtype=torch.bfloat16, device=Xs[0].device) for l in self.linears]
        xs = (_P * n)(*[x.data_ptr() for x in Xs])
        ys = (_P * n)(*[y.data_ptr() for y in outs])
        _check(_lib.patch_group_linear(self.handle, xs, M, ys, path, _stream(stream)))
        return outs

    def host(self, Xs, outs=None, path: int = PATH_AUTO, stream=None, sync: bool = True):
        """Host tensors in and out (pinned for overlapped copies). With
        sync=False the call only enqueues: the outputs are complete once
        `stream` is."""
        n = len(self.linears)
        assert len(Xs) == n and all(not x.is_cuda for x in Xs)
        M = Xs[0].shape[0]
        if outs is None:
            outs = [torch.empty((M, l.N), dtype=torch.bfloat16, pin_memory=True) for l in self.linears]
        xs = (_P * n)(*[x.data_ptr() for x in Xs])
        ys = (_P * n)(*[y.data_ptr() for y in outs])
        _check(_lib.patch_group_linear_host(self.handle, xs, M, ys, path, _stream(stream)))
        if sync:
            torch.cuda.synchronize()
        return outs

    def path(self, M: int, path: int = PATH_AUTO) -> int:
        """The explicit path a call with this M and requested path would run."""
        out = _I()
        _check(_lib.patch_group_path(self.handle, M, path, ctypes.byref(out)))
        return out.value

    def free(self):
        if self.handle:
            _lib.patch_group_free(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


# ---- object wrapper -----------------------------------------------------------

class PackedLinear:
    """A frozen weight packed as dense / 2:4 slabs; calling it runs the layer."""

    def __init__(self, handle: int, N: int, K: int):
        self.handle = handle
        self.N = N
        self.K = K

    @classmethod
    def pack(cls, W, mask_bits, tile_flags, tile_rows=128, tile_cols=128, bitorder=0, stream=None):
        h = patch_pack(W, mask_bits, tile_flags, tile_rows, tile_cols, bitorder, stream)
        return cls(h, W.shape[0], W.shape[1])

    def __call__(self, X: torch.Tensor, out: torch.Tensor | None = None, path: int = PATH_AUTO,
                 stream=None) -> torch.Tensor:
        assert X.is_cuda and X.dtype == torch.bfloat16 and X.dim() == 2 and X.shape[1] == self.K
        assert X.is_contiguous()
        if out is None:
            out = torch.empty((X.shape[0], self.N), dtype=torch.bfloat16, device=X.device)
        patch_linear_path(self.handle, X, out, path, stream)
        return out

    def host(self, X: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if out is None:
            out = torch.empty((X.shape[0], self.N), dtype=torch.bfloat16, pin_memory=True)
        patch_linear_host(self.handle, X, out, stream)
        return out

    def unpack(self, stream=None) -> torch.Tensor:
        out = torch.empty((self.N, self.K), dtype=torch.bfloat16, device="cuda")
        patch_unpack(self.handle, out, stream)
        return out

    def info(self) -> patch_info_t:
        return patch_info(self.handle)

    def packed(self):
        return patch_copy_packed(self.handle)

    def check(self, stream=None):
        patch_check(self.handle, stream)

    def free(self):
        if self.handle:
            patch_free(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class PackedLinearQ8:
    """A frozen weight packed as dense / 2:4 slabs of 8-bit codes with one scale
    per output channel; calling it runs the layer in 8-bit integers."""

    def __init__(self, handle: int, N: int, K: int):
        self.handle = handle
        self.N = N
        self.K = K

    @classmethod
    def pack(cls, W, mask_bits, tile_flags, tile_rows=128, tile_cols=128, bitorder=0, w_scale=None, stream=None):
        """W [N,K]: bf16, or int8 codes with their channel scales w_scale [N]."""
        h = patch_pack_q8(W, mask_bits, tile_flags, tile_rows, tile_cols, bitorder, w_scale, stream)
        return cls(h, W.shape[0], W.shape[1])

    def __call__(self, X: torch.Tensor, x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype | None = None, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
        """X [M,K]: codes with their scales x_scale [M], or bf16 / fp16 / fp32
        activations, which are quantised first. out_dtype: bf16 unless given (for
        activations, their own type)."""
        if x_scale is None:
            x = X
            out_dtype = out_dtype or X.dtype
            X, x_scale = _codes_like(x, stream)
            patch_quantize_q8(x, X, x_scale, stream)
        if out is None:
            out = _empty((X.shape[0], self.N), out_dtype or torch.bfloat16, X.device, stream)
        _check(_binding.linear_q8(self.handle, self.N, self.K, X, x_scale, out, path, stream))
        return out

    def unpack(self, stream=None):
        """(masked codes int8 [N,K], channel scales fp32 [N])."""
        W = _empty((self.N, self.K), torch.int8, "cuda", stream)
        w_scale = _empty(self.N, torch.float32, "cuda", stream)
        patch_unpack_q8(self.handle, W, w_scale, stream)
        return W, w_scale

    def info(self) -> patch_info_t:
        return patch_info(self.handle)

    def check(self, stream=None):
        patch_check(self.handle, stream)

    def free(self):
        if self.handle:
            patch_free(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class LinearGroupQ8:
    """Several 8-bit packed linears run with one launch (they share M). The
    inputs are codes, or come from one of the operators that end in codes:
    `quantize`, `norm` and `silu_mul` run it and then the group on its output."""

    def __init__(self, linears):
        self.linears = list(linears)
        arr = (_P * len(self.linears))(*[l.handle for l in self.linears])
        g = _P()
        _check(_lib.patch_group_create(arr, len(self.linears), ctypes.byref(g)))
        self.handle = g.value
        self._shapes = tuple(d for l in self.linears for d in (l.N, l.K))

    def __call__(self, Xs, x_scales, outs=None, out_dtype: torch.dtype = torch.bfloat16, path: int = PATH_AUTO,
                 stream=None):
        """Xs, x_scales: one tensor of codes (and its scales) for all members, or
        a list with one per member."""
        n = len(self.linears)
        if isinstance(Xs, torch.Tensor):
            Xs, x_scales = (Xs,) * n, (x_scales,) * n
        if len(Xs) != n or len(x_scales) != n or (outs is not None and len(outs) != n):
            raise ValueError(f"the group has {n} members")
        if outs is None:
            M, device = Xs[0].shape[0], Xs[0].device
            outs = [_empty((M, N), out_dtype, device, stream) for N in self._shapes[::2]]
        _check(_binding.group_linear_q8(self.handle, self._shapes, tuple(Xs), tuple(x_scales), tuple(outs), path, stream))
        return outs

    def quantize(self, x, outs=None, path: int = PATH_AUTO, stream=None):
        """The products of the rows of x, quantised once for all members."""
        q, scale = _codes_like(x, stream)
        patch_quantize_q8(x, q, scale, stream)
        return self(q, scale, outs, x.dtype, path, stream)

    def norm(self, x, gamma, eps: float, residual=None, residual_out=None, outs=None, path: int = PATH_AUTO, stream=None):
        """(products of the RMS norm of x + residual, x + residual); without a
        residual, (products of the norm of x, x)."""
        if residual is not None and residual_out is None:
            residual_out = _empty(x.shape, x.dtype, x.device, stream)
        q, scale = _codes_like(x, stream)
        patch_rmsnorm_q8(x, gamma, eps, q, scale, residual, residual_out, stream)
        return self(q, scale, outs, x.dtype, path, stream), x if residual is None else residual_out

    def silu_mul(self, gate, up, outs=None, path: int = PATH_AUTO, stream=None):
        """The products of silu(gate) * up."""
        q, scale = _codes_like(gate, stream)
        patch_silu_mul_q8(gate, up, q, scale, stream)
        return self(q, scale, outs, gate.dtype, path, stream)

    def path(self, M: int, path: int = PATH_AUTO) -> int:
        """The explicit path a call with this M and requested path would run."""
        out = _I()
        _check(_lib.patch_group_path(self.handle, M, path, ctypes.byref(out)))
        return out.value

    def free(self):
        if self.handle:
            _lib.patch_group_free(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
