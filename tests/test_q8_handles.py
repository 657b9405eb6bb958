"""What the thin calls on an 8-bit handle refuse, and what a handle holds, byte by
byte. Every refusal is raised before a kernel is launched."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
N, K = 384, 448


@pytest.fixture(scope="module")
def hsg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import hybrid_sparse_gemm_b200 as m
    return m


def pack(hsg, n=N, k=K, R=128, C=64, frac=0.6):
    p = synth.make_problem(n, k, 0, R=R, C=C, frac=frac, seed=17, device="cuda")
    g = synth.generator("cuda", "handles", n, k, R, C)
    W = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    scale = torch.rand(n, generator=g, device="cuda") + 0.5
    lin = hsg.PackedLinearQ8.pack(W, p.bits, p.flags.cpu(), R, C, w_scale=scale)
    return lin, W * p.keep, scale


def test_unpack_writes_into_fitting_tensors_only(hsg):
    lin, masked, scale = pack(hsg)
    W, s = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    for bad in (lambda: hsg.patch_unpack_q8(lin.handle, W[:-1], s), lambda: hsg.patch_unpack_q8(lin.handle, W[:, :-64], s),
                lambda: hsg.patch_unpack_q8(lin.handle, W.view(-1), s), lambda: hsg.patch_unpack_q8(lin.handle, W, s[:-1]),
                lambda: hsg.patch_unpack_q8(lin.handle, torch.empty(K, N, dtype=torch.int8, device="cuda").t(), s),
                lambda: hsg.patch_unpack_q8(lin.handle, torch.empty(N, K + 16, dtype=torch.int8, device="cuda")[:, :K], s),
                lambda: hsg.patch_unpack_q8(lin.handle, W, torch.empty(2 * N, device="cuda")[::2]),
                lambda: hsg.patch_unpack_q8(lin.handle, W.cpu(), s), lambda: hsg.patch_unpack_q8(lin.handle, W, s.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: hsg.patch_unpack_q8(lin.handle, W.view(torch.uint8), s),
                lambda: hsg.patch_unpack_q8(lin.handle, W.to(torch.bfloat16), s),
                lambda: hsg.patch_unpack_q8(lin.handle, W, s.double())):
        with pytest.raises(TypeError):
            bad()
    hsg.patch_unpack_q8(lin.handle, W, s)
    assert torch.equal(W, masked) and torch.equal(s, scale)


@pytest.mark.parametrize("M", [1, 4, 200])
def test_product_of_another_shape(hsg, M):
    """One row has no pitch to be checked by: the columns decide."""
    lin, masked, scale = pack(hsg)
    x, sx = torch.ones(M, K, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda")
    y = torch.empty(M, N, device="cuda")
    for a, b in ((x[:, :256].contiguous(), y), (x, y[:, :128].contiguous()), (x.new_ones(M, K + 64), y),
                 (x, y.new_empty(M, N + 128)), (x.new_ones(M, N), y.new_empty(M, K))):
        with pytest.raises(hsg.PatchError) as e:
            hsg.patch_linear_q8(lin.handle, a, sx, b)
        assert hsg.STATUS_NAMES[e.value.status] == "PATCH_ERR_SHAPE"
    for a, b in ((x[0], y), (x, y[0])):
        with pytest.raises(TypeError):
            hsg.patch_linear_q8(lin.handle, a, sx, b)
    hsg.patch_linear_q8(lin.handle, x, sx, y)
    # whole numbers below 2^24 times one scale: the product's rounding alone
    want = masked.double().sum(1) * scale.double()
    assert ((y.double() - want).abs() <= want.abs() * 1.01 * 2.0 ** -24).all()


@pytest.mark.parametrize("n,k,R,C,frac", [(384, 448, 128, 64, 0.6), (256, 384, 128, 128, 0.5), (128, 64, 64, 64, 1.0),
                                          (640, 320, 64, 64, 0.8), (256, 128, 128, 128, 0.0)])
def test_packed_bytes(hsg, n, k, R, C, frac):
    """Each record, decoded by the header's layout: 128 x 128 codes in 128-byte
    swizzled rows, or 64 kept codes a row in 64-byte swizzled ones and 16 bytes of
    position codes a row behind them."""
    lin, masked, _ = pack(hsg, n, k, R, C, frac)
    info = lin.info()
    packed, (slab, meta, gemm) = hsg.patch_copy_packed(lin.handle)
    S, KB = n // 128, (k + 127) // 128
    assert info.slabs_total == S * KB == slab.size == meta.size == gemm.size and packed.size == info.packed_bytes
    assert int((slab & 1).sum()) == info.slabs_sparse and int((gemm & 1).sum()) == info.slabs_pair_sparse
    want = np.zeros((n, KB * 128), np.int8)
    want[:, :k] = masked.cpu().numpy()

    def record(entry):
        at = int(entry >> 2) * 16
        got = np.zeros((128, 128), np.int8)
        if not entry & 1:
            for r in range(128):
                for c in range(8):
                    o = at + r * 128 + ((c ^ (r & 7)) << 4)
                    got[r, 16 * c:16 * c + 16] = packed[o:o + 16].view(np.int8)
            return got
        for r in range(128):
            kept = np.concatenate([packed[o:o + 16] for o in (at + r * 64 + ((c ^ ((r >> 1) & 3)) << 4) for c in range(4))])
            code = packed[at + 8192 + 16 * r:at + 8192 + 16 * r + 16]
            for g in range(32):
                p = (int(code[g // 2]) >> (4 * (g & 1))) & 15
                assert p & 3 < p >> 2
                got[r, 4 * g + (p & 3)], got[r, 4 * g + (p >> 2)] = kept.view(np.int8)[2 * g:2 * g + 2]
        return got

    for s in range(S):
        for b in range(KB):
            i = s * KB + b
            block = want[128 * s:128 * s + 128, 128 * b:128 * b + 128]
            assert np.array_equal(record(slab[i]), block) and np.array_equal(record(gemm[i]), block)
            assert meta[i] == ((slab[i] >> 2) + 512 if slab[i] & 1 else 0xFFFFFFFF)
            assert not (gemm[i] & 1) or slab[i] & 1


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), -1.0, -2.0 ** -140])
@pytest.mark.parametrize("row", [0, 127, 200, N - 1])
def test_pack_refuses_given_scales(hsg, bad, row):
    p = synth.make_problem(N, K, 0, C=64, frac=0.5, seed=1, device="cuda")
    W, s = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
    s[row] = bad
    with pytest.raises(hsg.PatchError) as e:
        hsg.PackedLinearQ8.pack(W, p.bits, p.flags.cpu(), 128, 64, w_scale=s)
    assert hsg.STATUS_NAMES[e.value.status] == "PATCH_ERR_ARG"
    s[row] = 0.0  # a channel of zeros
    s[row - 1] = 2.0 ** -140
    got = hsg.PackedLinearQ8.pack(W, p.bits, p.flags.cpu(), 128, 64, w_scale=s).unpack()[1]
    assert torch.equal(got, s)
