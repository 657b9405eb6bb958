"""The 8-bit integer path on a B200 against plain 64-bit arithmetic.

Tolerances, fixed before the first run. u = 2^-24 is half a step of fp32, h =
finfo.eps / 2 half a step of the output type (bf16 2^-8, fp16 2^-11, fp32 2^-24).
  * The product's int32 sum is exact; its conversion to fp32 and the two scales
    round three times, the output once: |err| <= |y| (3.01 u + h), and half the
    smallest fp16 subnormal, 2^-25, where the output is fp16.
  * A code is the nearest whole number to the computed y / scale, so it is off
    the exact quotient by at most 1/2 + 127 d, d being the quotient's relative
    error, derived at each operator.
"""
import math
import threading

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-5


@pytest.fixture(scope="module")
def hsg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import hybrid_sparse_gemm_b200 as m
    return m


def gen(*parts):
    return synth.generator("cuda", "q8", *parts)


def codes(g, m, k, pad=0):
    return torch.randint(-128, 128, (m, k + pad), generator=g, device="cuda", dtype=torch.int8)[:, :k]


def scales(g, n):
    return torch.rand(n, generator=g, device="cuda") * 0.02 + 0.001


class Weight:
    """Random codes under a hybrid mask, packed, and what they stand for."""

    def __init__(self, hsg, N, K, R=128, C=128, frac=0.5, seed=0, bitorder=0):
        g = gen(N, K, R, C, frac, seed)
        p = synth.make_problem(N, K, 0, R=R, C=C, frac=frac, seed=seed, device="cuda", bitorder=bitorder)
        self.all = codes(g, N, K).contiguous()
        self.masked = self.all * p.keep
        self.scale = scales(g, N)
        self.bits, self.flags, self.keep = p.bits, p.flags.cpu(), p.keep
        self.lin = hsg.PackedLinearQ8.pack(self.all, p.bits, self.flags, R, C, bitorder, w_scale=self.scale)

    def product(self, x, sx):
        return (x.double() @ self.masked.double().t()) * sx.double()[:, None] * self.scale.double()


def assert_product(y, want):
    h = torch.finfo(y.dtype).eps / 2
    tol = want.abs() * (3.01 * U + h) + (2.0 ** -25 if y.dtype == torch.float16 else 0.0)
    bad = (y.double() - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


def paths(hsg, M):
    return [hsg.PATH_AUTO, hsg.PATH_GEMM_SINGLE, hsg.PATH_GEMM_WIDE] + ([hsg.PATH_GEMV] if M <= 64 else [])


# --------------------------------------------------------------- packing ---

@pytest.mark.parametrize("N,K,R,C", [(256, 384, 128, 128), (384, 448, 128, 64), (256, 512, 64, 128), (384, 320, 64, 64),
                                     (128, 64, 64, 64)])
@pytest.mark.parametrize("frac", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("bitorder", [0, 1])
def test_codes_round_trip(hsg, N, K, R, C, frac, bitorder):
    w = Weight(hsg, N, K, R, C, frac, seed=3, bitorder=bitorder)
    got, scale = w.lin.unpack()
    assert torch.equal(got, w.masked) and torch.equal(scale, w.scale)
    info = w.lin.info()
    assert info.pruned == int((~w.keep).sum()) and info.stray_zeros == 0 and info.tiles_sparse == int(w.flags.sum())


def test_bf16_weights_are_quantised_over_kept_weights(hsg):
    N, K = 256, 448
    p = synth.make_problem(N, K, 0, C=64, frac=0.6, seed=5, device="cuda")
    W = p.W.clone()
    W[3] = 0
    W[p.keep.logical_not()] *= 50  # pruned weights are larger than any kept one
    lin = hsg.PackedLinearQ8.pack(W, p.bits, p.flags.cpu(), 128, 64)
    got, scale = lin.unpack()
    kept = W.double() * p.keep
    want = (kept.abs().amax(1) / 127).clamp_min(2.0 ** -126)
    assert ((scale.double() - want).abs() <= want * 1.01 * U).all()
    # y / scale: the scale's rounding and the quotient's
    assert ((got.double() - kept / want[:, None]).abs() <= 0.5 + 127 * 2.02 * U).all()
    assert not got[3].any() and not got[~p.keep].any()


def test_pack_refusals(hsg):
    p = synth.make_problem(256, 256, 0, frac=1.0, seed=1, device="cuda")
    keep = p.keep.clone()
    keep[5, 8:12] = True  # four kept in one group of a 2:4 tile
    with pytest.raises(hsg.PatchError) as e:
        hsg.PackedLinearQ8.pack(p.W, synth.pack_bits(keep), p.flags.cpu())
    assert e.value.status == 4
    for bad in (float("nan"), float("inf")):
        W = p.W.clone()
        W[7, int(p.keep[7].nonzero()[0])] = bad
        with pytest.raises(hsg.PatchError) as e:
            hsg.PackedLinearQ8.pack(W, p.bits, p.flags.cpu())
        assert e.value.status == 1
    W = p.W.clone()
    W[~p.keep] = float("nan")  # pruned weights may hold anything
    hsg.PackedLinearQ8.pack(W, p.bits, p.flags.cpu()).unpack()
    with pytest.raises(ValueError):
        hsg.PackedLinearQ8.pack(p.W, p.bits[:-1], p.flags.cpu())
    with pytest.raises(ValueError):
        hsg.PackedLinearQ8.pack(p.W, p.bits, p.flags.cpu()[:-1])
    with pytest.raises(hsg.PatchError):
        hsg.PackedLinearQ8.pack(p.W.to(torch.int8), p.bits, p.flags.cpu())
    with pytest.raises(ValueError):
        hsg.PackedLinearQ8.pack(p.W.to(torch.int8), p.bits, p.flags.cpu(), w_scale=torch.ones(255, device="cuda"))


# --------------------------------------------------------------- product ---

SHAPES = [(256, 384, 128, 128), (384, 448, 128, 64), (256, 512, 64, 128), (640, 320, 64, 64), (128, 128, 128, 128),
          (128, 64, 128, 64), (1152, 1088, 128, 64)]


@pytest.mark.parametrize("N,K,R,C", SHAPES)
@pytest.mark.parametrize("frac", [0.0, 0.6, 1.0])
def test_product(hsg, N, K, R, C, frac):
    w = Weight(hsg, N, K, R, C, frac, seed=1)
    for i, M in enumerate((1, 2, 15, 16, 17, 33, 64, 65, 128, 129, 225, 300, 513)):
        g = gen("x", M, K)
        x, sx = codes(g, M, K).contiguous(), scales(g, M)
        want = w.product(x, sx)
        for path in paths(hsg, M):
            y = w.lin(x, sx, out_dtype=TYPES[i % 3], path=path)
            w.lin.check()
            assert_product(y, want)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M", [3, 70, 300, 1000])
def test_pitches_and_what_lies_beside(hsg, t, M):
    w = Weight(hsg, 384, 448, 128, 64, 0.5, seed=2)
    g = gen("pitch", M)
    x, sx = codes(g, M, 448, pad=64), scales(g, M)
    for path in paths(hsg, M):
        frame = torch.full((M + 3, 384 + 24), 7.0, dtype=t, device="cuda")
        w.lin(x, sx, out=frame[:M, :384], path=path)
        assert_product(frame[:M, :384], w.product(x, sx))
        assert (frame[M:] == 7).all() and (frame[:, 384:] == 7).all()


@pytest.mark.parametrize("M", [1, 16, 40, 100, 300])
def test_long_rows(hsg, M):
    """More slabs per row than a warp holds records of (32), and than the wide
    kernel's tables hold (256)."""
    K = 40000
    w = Weight(hsg, 256, K, C=64, frac=0.5, seed=3)
    x, sx = codes(gen("long", M), M, K).contiguous(), scales(gen("long", M), M)
    want = w.product(x, sx)
    for path in paths(hsg, M):
        y = w.lin(x, sx, out_dtype=torch.float32, path=path)
        w.lin.check()
        assert_product(y, want)


def test_kernels_agree_to_the_bit(hsg):
    w = Weight(hsg, 640, 1152, frac=0.6, seed=12)
    for M in (5, 64, 300):
        x, sx = codes(gen("bits", M), M, 1152).contiguous(), scales(gen("bits", M), M)
        for t in TYPES:
            ys = [w.lin(x, sx, out_dtype=t, path=p) for p in paths(hsg, M)]
            assert all(torch.equal(y, ys[0]) for y in ys)


def test_largest_sums(hsg):
    """Every code -128 at the largest K: 128 * 128 * K = 2^31 - 2^20."""
    K = 131008
    lin = hsg.PackedLinearQ8.pack(torch.full((128, K), -128, dtype=torch.int8, device="cuda"),
                                  torch.full((128 * K // 8,), 255, dtype=torch.uint8, device="cuda"),
                                  [0] * (K // 64), 128, 64, w_scale=torch.ones(128, device="cuda"))
    for M in (1, 40, 100, 300):
        x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        for path in paths(hsg, M):
            y = lin(x, torch.ones(M, device="cuda"), out_dtype=torch.float32, path=path)
            lin.check()
            assert (y == 2.0 ** 14 * K).all()


def test_scales_reach_their_rows_only(hsg):
    w = Weight(hsg, 256, 256, seed=4)
    x, sx = codes(gen("nan"), 40, 256).contiguous(), scales(gen("nan"), 40)
    sx[7], sx[39] = float("nan"), float("inf")
    x[39, 0] = 0
    y = w.lin(x, sx)
    assert y[7].isnan().all() and not y[39].isfinite().any()
    rest = [i for i in range(40) if i not in (7, 39)]
    assert_product(y[rest], w.product(x, sx)[rest])


def test_no_tokens(hsg):
    w = Weight(hsg, 128, 128)
    assert w.lin(codes(gen(0), 0, 128), scales(gen(0), 0)).shape == (0, 128)


@pytest.mark.parametrize("M", [1, 16, 40, 100, 600])
def test_group(hsg, M):
    ws = [Weight(hsg, 512, 448, 64, 64, 0.7, 1), Weight(hsg, 128, 448, 128, 64, 0.0, 2), Weight(hsg, 384, 256, 128, 128, 1.0, 3)]
    group = hsg.LinearGroupQ8([w.lin for w in ws])
    g = gen("group", M)
    x, sx = codes(g, M, 448).contiguous(), scales(g, M)
    x2, sx2 = codes(g, M, 256, pad=16), scales(g, M)
    for path in paths(hsg, M):
        for t in TYPES:
            ys = group([x, x, x2], [sx, sx, sx2], out_dtype=t, path=path)
            ws[0].lin.check()
            for w, y, xi, si in zip(ws, ys, (x, x, x2), (sx, sx, sx2)):
                assert_product(y, w.product(xi, si))
    assert group.path(M) == hsg.LinearGroupQ8([ws[0].lin]).path(M) or M > 64


def test_repeats_give_the_same_bits(hsg):
    w = Weight(hsg, 1024, 2048, frac=0.7, seed=9)
    for M in (1, 16, 50, 100, 500):
        x, sx = codes(gen("again", M), M, 2048).contiguous(), scales(gen("again", M), M)
        first = w.lin(x, sx, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(w.lin(x, sx, out_dtype=torch.float32), first)


def test_linear_refusals(hsg):
    w = Weight(hsg, 256, 320, C=64, seed=6)
    bf = synth.make_problem(256, 320, 4, C=64, seed=6, device="cuda")
    plain = hsg.PackedLinear.pack(bf.W, bf.bits, bf.flags.cpu(), 128, 64)
    x, sx = codes(gen(1), 4, 320).contiguous(), scales(gen(1), 4)
    y = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")

    def status(f, *a, **k):
        with pytest.raises(hsg.PatchError) as e:
            f(*a, **k)
        return e.value.status

    assert status(plain, x.new_zeros(4, 320, dtype=torch.bfloat16)[:, :320], path=99) == 1
    assert status(hsg.patch_linear_q8, plain.handle, x, sx, y) == 1        # bf16 weights in the 8-bit call
    for call in (hsg.patch_linear, hsg.patch_linear_path, hsg.patch_linear_noalloc):
        assert status(call, w.lin.handle, bf.X, y) == 1                    # 8-bit weights in the bf16 calls
    assert status(hsg.patch_linear_host, w.lin.handle, bf.X.cpu(), y.cpu()) == 1
    assert status(hsg.patch_unpack, w.lin.handle, torch.empty(256, 320, dtype=torch.bfloat16, device="cuda")) == 1
    assert status(hsg.patch_unpack_q8, plain.handle, torch.empty(256, 320, dtype=torch.int8, device="cuda"), sx) == 1
    assert status(hsg.LinearGroup, [plain, w.lin]) == 1
    assert status(hsg.LinearGroupQ8, [w.lin, plain]) == 1
    group = hsg.LinearGroup([w.lin])
    assert status(group, [bf.X]) == 1
    assert status(group.host, [bf.X.cpu()]) == 1
    assert status(w.lin, x, sx, path=99) == 1
    assert status(w.lin, x, sx, path=hsg.PATH_GEMV_SIMT) == 8
    off = torch.empty(4 * 320 + 16, dtype=torch.int8, device="cuda")
    assert status(w.lin, off[8:8 + 1280].view(4, 320), sx) == 3            # base not on 16 bytes
    assert status(w.lin, torch.empty(4, 321, dtype=torch.int8, device="cuda")[:, :320], sx) == 3
    assert status(w.lin, x, sx, out=torch.empty(4, 257, dtype=torch.float32, device="cuda")[:, :256]) == 3
    assert status(hsg.patch_linear_q8, w.lin.handle, torch.empty(4, 256, dtype=torch.int8, device="cuda"), sx, y) == 2
    for bad in (lambda: w.lin(x[:, :256], sx), lambda: w.lin(x, sx[:3]), lambda: w.lin(x, sx, out=y[:3]),
                lambda: w.lin(x.t().contiguous().t(), sx), lambda: w.lin(x.cpu(), sx),
                lambda: hsg.LinearGroupQ8([w.lin])([x, x], [sx, sx])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: w.lin(x.to(torch.uint8), sx), lambda: w.lin(x, sx.double())):
        with pytest.raises(TypeError):
            bad()


# --------------------------------------------------------- row operators ---

LENGTHS = [(1, 1), (1, 64), (2, 7), (3, 4096), (9, 100), (5, 4097), (300, 1000), (40, 11008), (200, 2048), (3, 13824),
           (2, 16384), (2, 20000), (2, 40000), (500, 256), (150, 5120)]


def rows(g, m, k, t, pad=0):
    x = torch.randn(m, k, generator=g, device="cuda") * torch.exp(torch.randn(m, 1, generator=g, device="cuda"))
    wide = torch.full((m, k + pad), 9.0, device="cuda").to(t)
    wide[:, :k] = x.to(t)
    return wide[:, :k]


def assert_codes(q, scale, y, d_quotient, d_scale):
    want = (y.abs().amax(1) / 127).clamp_min(2.0 ** -126)
    assert ((scale.double() - want).abs() <= want * d_scale).all()
    off = (q.double() - y / want[:, None]).abs()
    assert (off <= 0.5 + 127 * d_quotient).all(), float(off.max())


def sum_error(K):
    """Relative error of the fp32 sum of K squares: each thread adds at most
    32 + K / 1024 terms in a chain, then ten partial sums."""
    return (32 + K / 1024 + 10 + 1) * U


def silu(g):
    return g / (1 + torch.exp(-g))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", LENGTHS)
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_row_operators(hsg, t, M, K, pad):
    g = gen("rows", M, K, str(t), pad)
    x, r, gamma = rows(g, M, K, t, pad), rows(g, M, K, t, pad), rows(g, 1, K, t)[0]
    frame = torch.full((M + 1, K + 5), 99, dtype=torch.int8, device="cuda")
    q, scale = frame[:M, :K], torch.full((M + 1,), 5.0, device="cuda")
    s = scale[:M]
    # the scale's division, its reciprocal; the rounding to a code is the half
    hsg.patch_quantize_q8(x, q, s)
    assert_codes(q, s, x.double(), 2.02 * U, 1.01 * U)
    out = rows(g, M, K, t, pad)
    hsg.patch_dequantize_q8(q, s, out)
    want = q.double() * s.double()[:, None]
    # (two roundings: the fp32 product and the type's)
    assert ((out.double() - want).abs() <= want.abs() * (1.01 * U + torch.finfo(t).eps / 2) + 2.0 ** -25).all()
    # __expf is off by 2 + 1.173 |g| units of 2^-23 (damped by e^-g for g > 0), __fdividef by 2 units, and five
    # roundings; the row's largest value and the code both carry it
    xd = x.double()
    d = (2 + 1.173 * float((-xd).clamp_min(0).max()) + 1 + 2) * 2 * U + 5 * U
    hsg.patch_silu_mul_q8(x, r, q, s)
    assert_codes(q, s, silu(xd) * r.double(), 2 * d + 3 * U, d + 2 * U)
    # h * gamma, the factor, /127, the reciprocal, code's factor: six roundings (the norm's own error is common to
    # code and scale); the scale: rsqrtf two units, half the mean's error, four roundings
    d_scale = 4 * U + 0.5 * (sum_error(K) + 3 * U) + 4 * U
    hsg.patch_rmsnorm_q8(x, gamma, EPS, q, s)
    assert_codes(q, s, xd * torch.rsqrt(xd.square().mean(1, keepdim=True) + EPS) * gamma.double(), 6.1 * U, d_scale)
    total = torch.empty_like(x)
    hsg.patch_rmsnorm_q8(x, gamma, EPS, q, s, residual=r, residual_out=total)
    h = (x.float() + r.float()).to(t)
    hd = h.double()
    y = hd * torch.rsqrt(hd.square().mean(1, keepdim=True) + EPS) * gamma.double()
    assert torch.equal(total, h)
    assert_codes(q, s, y, 6.1 * U, d_scale)
    first = q.clone()
    for where in (x.clone(), r.clone()):  # the sum in the place of either input
        a, b = (where, r) if torch.equal(where, x) else (x, where)
        hsg.patch_rmsnorm_q8(a, gamma, EPS, q, s, residual=b, residual_out=where)
        assert torch.equal(where, h) and torch.equal(q, first)
    assert (frame[M:] == 99).all() and (frame[:, K:] == 99).all() and scale[M] == 5


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("K", [64, 100, 4096, 20000])
def test_rows_without_numbers(hsg, t, K):
    M = 12
    g = gen("odd", K, str(t))
    x, ones = rows(g, M, K, t), torch.ones(M, K, dtype=t, device="cuda")
    x[0] = 0
    x[1, K // 2] = float("nan")
    x[2, K - 1] = float("inf")
    x[3, 0] = float("-inf")
    x[4] = 0
    x[4, K // 3] = 2.0 ** -130 if t != torch.float16 else 2.0 ** -24
    x[5] = 0
    x[5, 1] = torch.finfo(t).max
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    calls = {"quantize": lambda: hsg.patch_quantize_q8(x, q, s),
             "norm": lambda: hsg.patch_rmsnorm_q8(x, ones[0], EPS, q, s),
             "residual": lambda: hsg.patch_rmsnorm_q8(x, ones[0], EPS, q, s, residual=torch.zeros_like(x),
                                                      residual_out=torch.empty_like(x)),
             "silu": lambda: hsg.patch_silu_mul_q8(ones, x, q, s)}
    for name, call in calls.items():
        call()
        assert s[1:4].isnan().all() and not q[1:4].any(), name
        assert s[0] == 2.0 ** -126 and not q[0].any(), name
        assert s[4] > 0 and s[6:].isfinite().all(), name
        if name == "quantize":
            assert abs(int(q[4, K // 3])) == (127 if t == torch.float16 else round(2.0 ** -130 / 2.0 ** -126)), name
        overflows = t != torch.float16 and name in ("norm", "residual")  # the square of the largest bf16 or fp32 value
        assert (s[5].isnan() and not q[5].any()) if overflows else q[5, 1] == 127, name
    hsg.patch_rmsnorm_q8(x, ones[0], 0.0, q, s)  # 0 / 0
    assert s[0].isnan() and not q[0].any()


def test_row_refusals(hsg):
    x = torch.zeros(4, 64, device="cuda")
    q, s = torch.empty(4, 64, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    gamma = torch.ones(64, device="cuda")
    for bad in (lambda: hsg.patch_quantize_q8(x.t(), q, s), lambda: hsg.patch_quantize_q8(x, q[:, :63], s),
                lambda: hsg.patch_quantize_q8(x, q, s[:3]), lambda: hsg.patch_quantize_q8(x, q.cpu(), s),
                lambda: hsg.patch_quantize_q8(x.expand(4, 64)[:, :1].expand(4, 64), q, s),
                lambda: hsg.patch_silu_mul_q8(x, x[:3], q, s), lambda: hsg.patch_rmsnorm_q8(x, gamma[:63], EPS, q, s),
                lambda: hsg.patch_rmsnorm_q8(x, gamma, EPS, q, s, residual=x),
                lambda: hsg.patch_dequantize_q8(q, s[:3], x)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: hsg.patch_quantize_q8(x, q.view(torch.uint8), s), lambda: hsg.patch_quantize_q8(x, q, s.half()),
                lambda: hsg.patch_silu_mul_q8(x, x.half(), q, s),
                lambda: hsg.patch_rmsnorm_q8(x, gamma.half(), EPS, q, s), lambda: hsg.patch_dequantize_q8(q, s, x.double())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(hsg.PatchError):
        hsg.patch_rmsnorm_q8(x, gamma, -1.0, q, s)


# ------------------------------------------------------- used together -----

def layer(hsg, hidden, ffn, seed):
    shapes = dict(q=(hidden, hidden), k=(hidden // 4, hidden), v=(hidden // 4, hidden), o=(hidden, hidden),
                  gate=(ffn, hidden), up=(ffn, hidden), down=(hidden, ffn))
    ws = {n: Weight(hsg, *nk, frac=0.7, seed=seed) for n, nk in shapes.items()}
    for w in ws.values():
        w.value = w.masked.double() * w.scale.double()[:, None]
    return ws


def coded(y):
    s = (y.abs().amax(1, keepdim=True) / 127).clamp_min(2.0 ** -126)
    return torch.round(y / s) * s


@pytest.mark.parametrize("M", [1, 20, 80, 400])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
def test_layer(hsg, M, t):
    """A layer's linears with the operators between them (v stands in for the
    attention's output), against the same steps in 64 bits. Each step is fed
    the framework's own input, so that the bound of one step applies: a code
    may land one step off where the quotient is at a border, which moves an
    output by one code times a weight, and the output's rounding."""
    hidden, ffn = 512, 1408
    ws = layer(hsg, hidden, ffn, 11)
    g = gen("layer", M, str(t))
    x, h0 = rows(g, M, hidden, t), rows(g, M, hidden, t)
    g1, g2 = (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).to(t), torch.ones(hidden, dtype=t, device="cuda")
    qkv = hsg.LinearGroupQ8([ws[n].lin for n in ("q", "k", "v")])
    gate_up = hsg.LinearGroupQ8([ws[n].lin for n in ("gate", "up")])

    def norm(h, gamma):
        hd = h.double()
        return hd * torch.rsqrt(hd.square().mean(1, keepdim=True) + EPS) * gamma.double()

    def close(got, y, name):
        s = y.abs().amax(1, keepdim=True) / 127
        want = coded(y) @ ws[name].value.t()
        flips = ((y / s).frac().abs() - 0.5).abs() < 1e-3  # values at a border may go either way
        tol = (flips.double() * s) @ ws[name].value.abs().t() + want.abs() * (torch.finfo(t).eps / 2 + 1e-5)
        tol += 1e-5 * (coded(y).abs() @ ws[name].value.abs().t()) + 2.0 ** -24
        assert ((got.double() - want).abs() <= tol).all(), name

    (yq, yk, yv), h = qkv.norm(x, g1, EPS, residual=h0)
    assert torch.equal(h, (x.float() + h0.float()).to(t))
    for got, name in ((yq, "q"), (yk, "k"), (yv, "v")):
        close(got, norm(h, g1), name)
    att = yq.clone().clamp(-100, 100)
    o = ws["o"].lin(att)
    close(o, att.double(), "o")
    (yg, yu), h2 = gate_up.norm(o, g2, EPS, residual=h, residual_out=h)
    for got, name in ((yg, "gate"), (yu, "up")):
        close(got, norm(h2, g2), name)
    yg = (yg.float() / yg.float().abs().amax(1, keepdim=True).clamp_min(1e-3) * 4).to(t)
    down = hsg.LinearGroupQ8([ws["down"].lin])
    yu = (yu.float() / 64).to(t)
    (d,) = down.silu_mul(yg, yu)
    close(d, silu(yg.double()) * yu.double(), "down")
    (dq,) = down.quantize(yu)
    close(dq, yu.double(), "down")
    torch.cuda.synchronize()
    for w in ws.values():
        w.lin.check()


@pytest.mark.parametrize("M", [1, 40, 100, 400])
def test_capture_and_replay(hsg, M):
    """Norm and group captured together; replays follow new inputs, two graphs
    of one group run in turn."""
    ws = [Weight(hsg, 512, 1024, frac=0.7, seed=s) for s in (1, 2)]
    group = hsg.LinearGroupQ8([w.lin for w in ws])
    K = 1024
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    x = [rows(gen("cap", M, i), M, K, torch.bfloat16).contiguous() for i in range(2)]
    q = [torch.empty(M, K, dtype=torch.int8, device="cuda") for _ in x]
    s = [torch.empty(M, device="cuda") for _ in x]
    ys = [[torch.empty(M, 512, dtype=torch.float32, device="cuda") for _ in ws] for _ in x]

    def step(i):
        hsg.patch_rmsnorm_q8(x[i], gamma, EPS, q[i], s[i])
        group(q[i], s[i], outs=ys[i])

    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        step(0)
        side.synchronize()
        for i in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step(i)
            graphs.append(graph)
    for turn in range(3):
        for i in range(2):
            x[i].copy_(rows(gen("new", M, turn, i), M, K, torch.bfloat16))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for w, y in zip(ws, ys[i]):
                assert_product(y, w.product(q[i], s[i]))
            again = torch.empty_like(q[i])
            hsg.patch_rmsnorm_q8(x[i], gamma, EPS, again, s[i])
            assert torch.equal(again, q[i])


@pytest.mark.parametrize("M", [1, 30, 100, 600])
def test_first_call_captured_and_graphs_side_by_side(hsg, M):
    """No call needs a warm-up; two graphs of one group share nothing."""
    ws = [Weight(hsg, 1024, 2048, frac=0.7, seed=s) for s in (21, 22)]
    group = hsg.LinearGroupQ8([w.lin for w in ws])
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for i, st in enumerate(streams):
        x, sx = codes(gen("side", M, i), M, 2048).contiguous(), scales(gen("side", M, i), M)
        ys = [torch.empty(M, 1024, dtype=torch.float32, device="cuda") for _ in ws]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            for _ in range(5):
                group(x, sx, outs=ys)
        jobs.append((graph, x, sx, ys))
    for _ in range(10):
        for st, job in zip(streams, jobs):
            with torch.cuda.stream(st):
                job[0].replay()
    torch.cuda.synchronize()
    for _, x, sx, ys in jobs:
        for w, y in zip(ws, ys):
            assert_product(y, w.product(x, sx))


@pytest.mark.parametrize("M", [1, 16, 50, 130, 500])
def test_long_chain(hsg, M):
    """Each kernel's set-up overlaps the one before it: a chain of dependent calls
    on the same few buffers gives the bits that it gives one call at a time."""
    hidden = 512
    mix = Weight(hsg, hidden, hidden, frac=0.7, seed=31)
    gate, up = Weight(hsg, hidden, hidden, frac=0.5, seed=32), Weight(hsg, hidden, hidden, frac=0.9, seed=33)
    t = torch.bfloat16
    gamma = torch.ones(hidden, dtype=t, device="cuda")
    start = rows(gen("chain", M), M, hidden, t).contiguous()
    group = hsg.LinearGroupQ8([gate.lin, up.lin])

    def run(wait):
        x, h = start.clone(), start.clone()
        q, s = torch.empty(M, hidden, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        ys = [torch.empty(M, hidden, dtype=t, device="cuda") for _ in range(2)]
        for _ in range(25):
            hsg.patch_rmsnorm_q8(x, gamma, EPS, q, s, residual=h, residual_out=h)
            wait()
            group(q, s, outs=ys)
            wait()
            hsg.patch_silu_mul_q8(ys[0], ys[1], q, s)
            wait()
            mix.lin(q, s, out=x)
            wait()
            hsg.patch_quantize_q8(x, q, s)
            wait()
            hsg.patch_dequantize_q8(q, s, x)
            wait()
            x.clamp_(-100, 100)
        torch.cuda.synchronize()
        return x, h

    slow = run(torch.cuda.synchronize)
    for _ in range(3):
        fast = run(lambda: None)
        assert torch.equal(fast[0], slow[0]) and torch.equal(fast[1], slow[1])
    assert slow[0].isfinite().all() and slow[1].isfinite().all()


@pytest.mark.parametrize("M", [1, 40, 100, 300])
def test_streams_and_threads(hsg, M):
    w = Weight(hsg, 1024, 2048, frac=0.7, seed=8)
    x = [codes(gen("str", M, i), M, 2048).contiguous() for i in range(4)]
    sx = [scales(gen("str", M, i), M) for i in range(4)]
    want = [w.product(a, b) for a, b in zip(x, sx)]
    y = [torch.empty(M, 1024, dtype=torch.float32, device="cuda") for _ in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]

    def work(i):
        torch.cuda.set_device(0)
        for _ in range(10):
            w.lin(x[i], sx[i], out=y[i], stream=streams[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    w.lin.check()
    for a, b in zip(y, want):
        assert_product(a, b)


@pytest.mark.parametrize("raw", [False, True])
def test_memory_of_a_call_belongs_to_its_stream(hsg, raw, monkeypatch):
    """What a call on a named stream allocates is not handed to the current
    stream while the call may still run."""
    M, N, K = 40, 512, 1024
    w = Weight(hsg, N, K, frac=0.7, seed=9)
    group = hsg.LinearGroupQ8([w.lin])
    x = rows(gen("own"), M, K, torch.bfloat16).contiguous()
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    used = []
    for name in ("patch_quantize_q8", "patch_rmsnorm_q8", "patch_silu_mul_q8"):
        def record(*args, f=getattr(hsg, name), **kw):
            used.extend((t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in args
                        if isinstance(t, torch.Tensor) and t is not x and t is not gamma)
            return f(*args, **kw)
        monkeypatch.setattr(hsg, name, record)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for call in (lambda st: w.lin(x, stream=st), lambda st: group.quantize(x, stream=st)[0],
                 lambda st: group.norm(x, gamma, 1e-5, x, stream=st)[0][0],
                 lambda st: group.silu_mul(x, x, stream=st)[0]):
        used.clear()
        y = call(stream.cuda_stream if raw else stream)
        used.append((y.untyped_storage().data_ptr(), y.untyped_storage().nbytes()))
        assert len(used) >= 3
        del y
        fresh = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in used for _ in range(3)]
        assert not {t.data_ptr() for t in fresh} & {p for p, _ in used}
        torch.cuda.synchronize()
        assert torch.equal(call(stream), call(None).clone())
        torch.cuda.synchronize()
        del fresh


def test_capture_with_the_stream_named(hsg):
    """The memory of a captured call belongs to the graph, whether its stream is named or current."""
    M, K = 20, 512
    w = Weight(hsg, 512, K, frac=0.5, seed=4)
    group = hsg.LinearGroupQ8([w.lin])
    x = rows(gen("cap"), M, K, torch.bfloat16).contiguous()
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    want, h = group.norm(x, gamma, 1e-5, x)
    want = group.silu_mul(want[0], h)[0].clone()
    torch.cuda.synchronize()
    for raw in (False, True):
        side = torch.cuda.Stream()
        name = side.cuda_stream if raw else side
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y, h = group.norm(x, gamma, 1e-5, x, stream=name)
            y = group.silu_mul(y[0], h, stream=name)[0]
        junk = [torch.full((M * K * 4,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        for _ in range(2):
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
        assert all(bool((j == 7).all()) for j in junk)


def test_path_of_extreme_sizes(hsg):
    w = Weight(hsg, 512, 512, seed=1)
    group = hsg.LinearGroupQ8([w.lin])
    for M in (0, 1, 64, 65, 10**6, 2**30 - 1):
        for path in (hsg.PATH_AUTO, hsg.PATH_GEMM):
            kernels = {hsg.PATH_GEMM_SINGLE, hsg.PATH_GEMM_WIDE} | ({hsg.PATH_GEMV} if path == hsg.PATH_AUTO else set())
            assert group.path(M, path) in kernels
    for M in (2**30, 2**31, 2**62):
        with pytest.raises(hsg.PatchError) as e:
            group.path(M)
        assert hsg.STATUS_NAMES[e.value.status] == "PATCH_ERR_SHAPE"


def test_handles_come_and_go(hsg):
    before = None
    for i in range(6):
        w = Weight(hsg, 512, 512, seed=1)
        for M in (1, 30, 100, 300):
            w.lin(codes(gen(i, M), M, 512).contiguous(), scales(gen(i, M), M))
        torch.cuda.synchronize()
        w.lin.free()
        del w
        free = torch.cuda.mem_get_info()[0]
        if i == 1:
            before = free
    assert before - free < 32 << 20


@pytest.mark.parametrize("M,N,K", [(100003, 128, 64), (3, 28672, 512), (2049, 512, 8192)])
def test_large(hsg, M, N, K):
    w = Weight(hsg, N, K, C=64, frac=0.5, seed=1)
    x, sx = codes(gen("large", M), M, K).contiguous(), scales(gen("large", M), M)
    for path in paths(hsg, M):
        y = w.lin(x, sx, path=path)
        w.lin.check()
        assert_product(y, w.product(x, sx))


def test_rows_past_32_bits(hsg):
    """Offsets of the last rows exceed 2^31 elements."""
    M, K = 70000, 32768
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-2:] = rows(gen("far"), 2, K, torch.bfloat16)
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    hsg.patch_quantize_q8(x, q, s)
    assert_codes(q[-2:], s[-2:], x[-2:].double(), 2.02 * U, 1.01 * U)
    out = torch.empty_like(x)
    hsg.patch_dequantize_q8(q, s, out)
    assert torch.equal(out[-2:], (q[-2:].float() * s[-2:, None]).to(torch.bfloat16)) and not out[:-2].any()
