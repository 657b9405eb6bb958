"""Refusals of the 8-bit integer calls that need no GPU: every argument is
checked before a device is touched."""
import ctypes

import numpy as np
import pytest

ARG, SHAPE, ALIGN = 1, 2, 3
P = 0x1000  # stands for an aligned device pointer; no call below gets as far as using it
BF16, FP16, FP32, INT8 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    import hybrid_sparse_gemm_b200 as m
    return m.library()


def pack(lib, W=P, w_type=BF16, w_scale=None, N=256, K=256, bits=P, bitorder=0, flags=None, R=128, C=128):
    if flags is None:
        flags = np.zeros(max(1, (N // max(R, 1)) * (K // max(C, 1))), np.uint8)
    h = ctypes.c_void_p(1)
    st = lib.patch_pack_q8(W, w_type, w_scale, N, K, bits, bitorder, flags.ctypes.data, R, C, None, ctypes.byref(h))
    assert h.value is None
    return st


@pytest.mark.parametrize("want,bad", [
    (ARG, dict(W=None)), (ARG, dict(bits=None)), (ARG, dict(bitorder=2)), (ARG, dict(w_type=FP16)),
    (ARG, dict(w_type=FP32)), (ARG, dict(w_type=9)), (ARG, dict(w_type=INT8)), (ARG, dict(w_scale=P)),
    (ALIGN, dict(w_type=INT8, w_scale=P + 2)), (ALIGN, dict(W=P + 8)), (SHAPE, dict(R=96)), (SHAPE, dict(N=200)),
    (SHAPE, dict(K=96, C=64)), (SHAPE, dict(K=192)), (SHAPE, dict(N=0)), (SHAPE, dict(K=131072)),
    (ARG, dict(flags=np.full(4, 2, np.uint8))),
])
def test_pack_q8_refuses(lib, want, bad):
    assert pack(lib, **bad) == want
    assert lib.patch_last_error()


def test_null_handles(lib):
    assert lib.patch_linear_q8(None, P, 256, P, 4, P, 256, BF16, 0, None) == ARG
    assert lib.patch_group_linear_q8(None, None, None, None, 4, None, None, BF16, 0, None) == ARG
    assert lib.patch_unpack_q8(None, P, P, None) == ARG


ROWS = {
    "quantize": (lambda lib, x=P, ldx=64, type=BF16, M=4, K=64, q=P, ldq=64, scale=P:
                 lib.patch_quantize_q8(x, ldx, type, M, K, q, ldq, scale, None)),
    "rmsnorm": (lambda lib, x=P, ldx=64, type=BF16, M=4, K=64, q=P, ldq=64, scale=P, residual=P, ldr=64, out=P, ldo=64,
                gamma=P, eps=1e-5:
                lib.patch_rmsnorm_q8(x, ldx, residual, ldr, out, ldo, gamma, type, eps, M, K, q, ldq, scale, None)),
    "silu_mul": (lambda lib, x=P, ldx=64, type=BF16, M=4, K=64, q=P, ldq=64, scale=P, up=P, ldu=64:
                 lib.patch_silu_mul_q8(x, ldx, up, ldu, type, M, K, q, ldq, scale, None)),
    "dequantize": (lambda lib, x=P, ldx=64, type=BF16, M=4, K=64, q=P, ldq=64, scale=P:
                   lib.patch_dequantize_q8(q, ldq, scale, M, K, x, ldx, type, None)),
}
COMMON = [(ARG, dict(x=None)), (ARG, dict(q=None)), (ARG, dict(scale=None)), (ARG, dict(type=INT8)), (ARG, dict(type=-1)),
          (ARG, dict(M=-1)), (SHAPE, dict(K=0)), (SHAPE, dict(K=-5)), (SHAPE, dict(K=1 << 25)), (SHAPE, dict(M=1 << 31)),
          (SHAPE, dict(ldx=63)), (SHAPE, dict(ldq=63)), (ALIGN, dict(x=P + 1)), (ALIGN, dict(x=P + 2, type=FP32)),
          (ALIGN, dict(scale=P + 2))]


@pytest.mark.parametrize("op", sorted(ROWS))
@pytest.mark.parametrize("want,bad", COMMON)
def test_row_operators_refuse(lib, op, want, bad):
    assert ROWS[op](lib, **bad) == want
    assert lib.patch_last_error()


@pytest.mark.parametrize("op,want,bad", [
    ("rmsnorm", ARG, dict(residual=None)), ("rmsnorm", ARG, dict(out=None)), ("rmsnorm", ARG, dict(gamma=None)),
    ("rmsnorm", ARG, dict(eps=-1e-5)), ("rmsnorm", ARG, dict(eps=float("nan"))), ("rmsnorm", ARG, dict(eps=float("inf"))),
    ("rmsnorm", SHAPE, dict(ldr=63)), ("rmsnorm", SHAPE, dict(ldo=63)), ("rmsnorm", ALIGN, dict(gamma=P + 1)),
    ("silu_mul", ARG, dict(up=None)), ("silu_mul", SHAPE, dict(ldu=63)), ("silu_mul", ALIGN, dict(up=P + 1)),
])
def test_row_operators_refuse_their_own(lib, op, want, bad):
    assert ROWS[op](lib, **bad) == want


@pytest.mark.parametrize("op", sorted(ROWS))
def test_no_rows_is_a_no_op(lib, op):
    assert ROWS[op](lib, M=0, x=None, q=None, scale=None) == 0


def test_cpu_tensors(lib):
    import torch
    import hybrid_sparse_gemm_b200 as hsg
    x, q, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: hsg.patch_quantize_q8(x, q, s), lambda: hsg.patch_silu_mul_q8(x, x, q, s),
                 lambda: hsg.patch_rmsnorm_q8(x, x[0], 1e-5, q, s), lambda: hsg.patch_dequantize_q8(q, s, x),
                 lambda: hsg.patch_linear_q8(1, q, s, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        hsg.patch_pack_q8(x, None, None)
    for bad in (lambda: hsg._binding.quantize_q8(x, q, s), lambda: hsg.patch_rmsnorm_q8(x, x[0], "eps", q, s)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(AttributeError):
        hsg.patch_quantize_q8(3, q, s)
