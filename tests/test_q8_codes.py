"""The codes of the row operators, to the last one: round(y / scale), ties to
even, with the quotient of an fp32 division, as numpy computes it on the CPU.

Random values seldom lie at a border between two codes, so most rows here are
made of values next to the ties n + 1/2 of their own scale. Everything compared
is exact: the scales are one fp32 division of exact maxima, and no tolerance is
needed.
"""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-5
LEAST = np.float32(2.0 ** -126)
# rows: aligned, off their boundaries, of one warp, of many groups a thread, read twice
LENGTHS = [(40, 64), (40, 100), (9, 1000), (300, 2048), (12, 4097), (12, 5120), (200, 8192), (5, 13824), (3, 20000)]


@pytest.fixture(scope="module")
def hsg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import hybrid_sparse_gemm_b200 as m
    return m


def steps(y):
    return np.maximum(np.abs(y).max(1) / np.float32(127), LEAST)


def divided(y, step):
    assert y.dtype == step.dtype == np.float32
    return np.rint(y / step[:, None]).astype(np.int8)


def at_borders(M, K, t, pad, seed):
    """Rows whose values lie at the ties of their own scale or beside them, as far
    as the type holds such values; some rows far smaller or larger than the others."""
    rng = np.random.default_rng([M, K, TYPES.index(t), pad, seed])
    top = (rng.uniform(1, 2, M) * 2.0 ** rng.integers(-3, 4, M)).astype(np.float32)
    top[0] = 381  # a scale of 3: 1.5 / 3 is a tie that 1.5 * (1 / 3) is not
    x = (rng.integers(-127, 127, (M, K)) + 0.5) * (top[:, None] / 127)
    x[:, 0] = top
    if t != torch.float16:
        far = rng.integers(0, 8, M)
        x *= np.choose(far, [2.0 ** -128, 2.0 ** -100, 2.0 ** 90] + [1.0] * 5)[:, None]
    x = x.astype(np.float32)
    beside = rng.integers(-2, 3, (M, K)) * (np.abs(x) < np.abs(x).max(1, keepdims=True))
    x = (x.view(np.int32) + beside.astype(np.int32)).view(np.float32)
    wide = torch.zeros(M, K + pad, dtype=t, device="cuda")
    wide[:, :K] = torch.from_numpy(x)
    return wide[:, :K]


def host(x):
    return x.float().cpu().numpy()


def outputs(M, K):
    return torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", LENGTHS)
@pytest.mark.parametrize("pad", [0, 3])
def test_quantize(hsg, t, M, K, pad):
    x, (q, s) = at_borders(M, K, t, pad, 0), outputs(M, K)
    hsg.patch_quantize_q8(x, q, s)
    step = steps(host(x))
    assert np.array_equal(s.cpu().numpy(), step)
    assert np.array_equal(q.cpu().numpy(), divided(host(x), step))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", LENGTHS)
@pytest.mark.parametrize("pad", [0, 3])
def test_silu_mul(hsg, t, M, K, pad):
    """A gate of 64 is its own silu in fp32, and the product with it exact."""
    u, (q, s) = at_borders(M, K, t, pad, 1), outputs(M, K)
    hsg.patch_silu_mul_q8(torch.full_like(u, 64), u, q, s)
    y = host(u) * np.float32(64)
    step = steps(y)
    assert np.array_equal(s.cpu().numpy(), step)
    assert np.array_equal(q.cpu().numpy(), divided(y, step))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", LENGTHS)
@pytest.mark.parametrize("pad,pad_r", [(0, 0), (3, 3), (3, 0)])
def test_norm(hsg, t, M, K, pad, pad_r):
    """The norm is a factor common to a row's values and its scale: the codes are
    those of h * gamma, a product of two numbers rounded to fp32."""
    x, (q, s) = at_borders(M, K, t, pad, 2), outputs(M, K)
    x = torch.where(x.float().abs() < 2.0 ** 60, x.float(), x.float() * 2.0 ** -60).to(t)  # squares stay finite
    if pad:
        wide = torch.zeros(M, K + pad, dtype=t, device="cuda")
        wide[:, :K] = x
        x = wide[:, :K]
    gamma = torch.from_numpy(np.random.default_rng(K).choice([0.5, 1.0, 1.25, -0.75], K).astype(np.float32)).to(t).cuda()
    gamma[0] = 1.25
    zero = torch.zeros(M, K + pad_r, dtype=t, device="cuda")[:, :K]
    y = host(x) * host(gamma)
    step = steps(y)
    for residual in (None, zero):
        hsg.patch_rmsnorm_q8(x, gamma, 2.0 ** -20, q, s, residual=residual,
                             residual_out=None if residual is None else torch.empty_like(zero))
        # (a value that the factor would lift over the least scale is divided after it)
        plain = (s.cpu().numpy() > LEAST) & (np.abs(y).max(1) / np.float32(127) >= LEAST)
        assert plain.sum() >= M // 2
        assert np.array_equal(q.cpu().numpy()[plain], divided(y, step)[plain])


def test_in_earnest(hsg):
    """Ordinary activations, whole rows: half a row's maximum is a tie that many rows hold."""
    g = synth.generator("cuda", "codes")
    x = (torch.randn(4096, 5120, generator=g, device="cuda") * torch.exp(torch.randn(4096, 1, generator=g, device="cuda"))).to(
        torch.bfloat16)
    q, s = outputs(*x.shape)
    hsg.patch_quantize_q8(x, q, s)
    y = host(x)
    assert np.array_equal(q.cpu().numpy(), divided(y, steps(y)))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", LENGTHS)
@pytest.mark.parametrize("pad,pad_q", [(0, 0), (3, 0), (0, 5)])
def test_dequantize(hsg, t, M, K, pad, pad_q):
    """The fp32 product, rounded to the type."""
    g = synth.generator("cuda", "values", M, K, pad)
    q = torch.randint(-127, 128, (M, K + pad_q), generator=g, device="cuda", dtype=torch.int8)[:, :K]
    s = torch.exp2(torch.randint(-20, 4, (M,), generator=g, device="cuda").float()) * (
        1 + torch.rand(M, generator=g, device="cuda"))
    out = torch.empty(M, K + pad, dtype=t, device="cuda")[:, :K]
    hsg.patch_dequantize_q8(q, s, out)
    assert torch.equal(out.cpu(), (q.cpu().float() * s.cpu()[:, None]).to(t))


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [64, 100, 4096, 20000])
def test_norms_that_leave_the_range(hsg, t, K):
    """An overflowing product with gamma, and squares that vanish without an eps,
    give NaN; with one, the row is an ordinary one."""
    x, (q, s) = torch.full((4, K), 0.5, dtype=t, device="cuda"), outputs(4, K)
    x[0] *= 2.0 ** 60
    x[1] *= 2.0 ** -100
    big = torch.full((K,), 2.0 ** 70, dtype=t, device="cuda")
    hsg.patch_rmsnorm_q8(x, big, EPS, q, s)
    assert s[0].isnan() and not q[0].any() and s[1:].isfinite().all() and (q[1:] == 127).all()
    hsg.patch_rmsnorm_q8(x, torch.ones_like(big), 0.0, q, s)
    assert s[1].isnan() and not q[1].any() and s[2:].isfinite().all() and (q[2:] == 127).all()
    # the first row's squares are 2^118 each: K of them overflow from K = 1024 on
    assert s[0].isnan() == (K * 2.0 ** 118 >= 2.0 ** 128) and (q[0] == (0 if K >= 1024 else 127)).all()
