"""AUTO's choice between the two 8-bit kernels where their measured times are
furthest apart (the figures stand beside the rule). Nothing is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hsg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import hybrid_sparse_gemm_b200 as m
    return m


def group(hsg, N, K, frac):
    n = (N // 128) * (K // 128)
    flags = torch.zeros(n, dtype=torch.uint8)
    flags[torch.randperm(n, generator=torch.Generator().manual_seed(N + K))[:round(frac * n)]] = 1
    dense = ~flags.bool().view(N // 128, K // 128).repeat_interleave(128, 0).repeat_interleave(16, 1)
    bits = torch.where(dense, 255, 0b11001100).to(torch.uint8).contiguous().cuda()
    W = torch.ones(N, K, dtype=torch.int8, device="cuda")
    return hsg.LinearGroupQ8([hsg.PackedLinearQ8.pack(W, bits, flags, w_scale=torch.ones(N, device="cuda"))])


@pytest.mark.parametrize("frac", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("N,K,split,wide", [
    (2048, 2048, [65, 200, 512, 1024, 2048], []),
    (512, 2048, [65, 200, 512, 1024, 2048], []),
    (4096, 4096, [65, 200, 400, 512], []),
    (4096, 11008, [65, 200, 400, 512], []),
    (11008, 4096, [65, 100, 128], [400, 512, 1024, 2048]),
    (13824, 5120, [65, 100, 128], [400, 1024, 2048]),
    (8192, 2048, [448], []),
])
def test_the_faster_kernel(hsg, N, K, split, wide, frac):
    g = group(hsg, N, K, frac)
    for M in split:
        assert g.path(M) == g.path(M, hsg.PATH_GEMM) == hsg.PATH_GEMM_SINGLE, M
    for M in wide:
        assert g.path(M) == g.path(M, hsg.PATH_GEMM) == hsg.PATH_GEMM_WIDE, M


@pytest.mark.parametrize("N,K,M", [(4096, 11008, 768), (4096, 11008, 2048), (11008, 4096, 768), (13824, 5120, 512)])
def test_the_share_of_2_4_tiles_decides(hsg, N, K, M):
    assert group(hsg, N, K, 0.0).path(M) == hsg.PATH_GEMM_SINGLE
    assert group(hsg, N, K, 1.0).path(M) == hsg.PATH_GEMM_WIDE


def test_path_refuses_what_the_product_refuses(hsg):
    """2^23 tiles of 128 tokens times 32 strips are more than the launch counts."""
    g = group(hsg, 4096, 128, 0.5)
    M = 2 ** 30 - 1
    x, s = torch.empty(1, 128, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    with pytest.raises(hsg.PatchError) as product:
        hsg._check(hsg.library().patch_linear_q8(g.linears[0].handle, x.data_ptr(), 128, s.data_ptr(), M, x.data_ptr(), 4096,
                                                 hsg.TYPE_BF16, hsg.PATH_GEMM_SINGLE, None))
    with pytest.raises(hsg.PatchError) as asked:
        g.path(M, hsg.PATH_GEMM_SINGLE)
    assert product.value.status == asked.value.status and str(product.value) == str(asked.value)
    assert g.path(M, hsg.PATH_GEMM_WIDE) == hsg.PATH_GEMM_WIDE and g.path(2 ** 29, hsg.PATH_GEMM_SINGLE) == hsg.PATH_GEMM_SINGLE
