"""MXFP4 matrices anywhere in a larger buffer: scales at every 4 bytes and codes at
every 16 give the bits of arrays of their own, in every form of the quantiser
and of the product."""
import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def placed(mx, code_at, scale_at):
    """The matrix as slices of buffers that hold other bytes around it."""
    out = []
    for t, at in zip(mx, (code_at, scale_at)):
        buf = torch.full((t.numel() + at + 64,), 0xEE, dtype=torch.uint8, device=DEV)
        out.append(buf[at:at + t.numel()])
        out[-1].copy_(t)
        assert out[-1].data_ptr() % 16 == at % 16
    return tuple(out)


# every tile shape, the product of few rows, and the one that splits K
@pytest.mark.parametrize("M,N,K", [(5, 80, 1600), (16, 8208, 576), (160, 1536, 12288), (378, 16, 320),
                                   (642, 3408, 448), (871, 6080, 64), (4526, 1344, 1024),
                                   (962, 6192, 192), (1463, 4896, 1216), (1924, 3760, 576),
                                   (3480, 3088, 448), (5892, 1952, 320), (4578, 2576, 1728),
                                   (4857, 2352, 1472), (2585, 4880, 832), (2709, 4512, 1088)])
@pytest.mark.parametrize("x_at,w_at", [(4, 0), (0, 8), (12, 4), (8, 12)])
def test_product_of_scales_at_every_four_bytes(M, N, K, x_at, w_at):
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N + K)
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N) * torch.exp(normal(g, 1, N)))
    mx = S.segquant_quantize_mxfp4((normal(g, M, K) * torch.exp(normal(g, M, 1))).to(BF))
    want = S.segquant_gemm_mxfp4(None, w, N, K=K, xq=mx, M=M)
    got = S.segquant_gemm_mxfp4(None, placed(w, 16, w_at), N, K=K, xq=placed(mx, 48, x_at), M=M)
    assert torch.equal(got, want)


@pytest.mark.parametrize("M,N,K", [(3, 96, 576), (40, 80, 192), (300, 128, 1536)])
@pytest.mark.parametrize("at", [4, 8, 12])
def test_product_of_bf16_on_a_weight_at_every_four_bytes(M, N, K, at):
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    z = normal(g, M, K).to(BF)
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N))
    for act in (S.SEGQ_ACT_NONE, S.SEGQ_ACT_SILU):
        assert torch.equal(S.segquant_gemm_mxfp4(z, placed(w, 32, at), N, act_kind=act),
                           S.segquant_gemm_mxfp4(z, w, N, act_kind=act))


@pytest.mark.parametrize("at", [4, 8, 12])
def test_what_writes_and_unpacks_at_every_four_bytes(at):
    g = torch.Generator(device=DEV)
    g.manual_seed(at)
    M, K = 37, 576
    z, w = normal(g, M, K).to(BF), normal(g, K, 48)
    empty = placed(S.segquant_quantize_mxfp4(torch.zeros_like(z)), 16, at)
    for act in (S.SEGQ_ACT_NONE, S.SEGQ_ACT_SILU, S.SEGQ_ACT_GELU):
        for a, b in zip(S.segquant_quantize_mxfp4(z, act, out=empty),
                        S.segquant_quantize_mxfp4(z, act)):
            assert torch.equal(a, b)
    gamma = torch.rand(K, device=DEV, generator=g)
    norm = S.segquant_rmsnorm_quantize(z, gamma=gamma, mx_out=empty)[3]
    want = S.segquant_rmsnorm_quantize(z, gamma=gamma, mx_out=True)[3]
    assert torch.equal(S.segquant_unpack_mxfp4(norm, M, K), S.segquant_unpack_mxfp4(want, M, K))
    want = S.segquant_quantize_weight_mxfp4(w)
    for a, b in zip(S.segquant_quantize_weight_mxfp4(w, out=placed(want, 48, at)), want):
        assert torch.equal(a, b)
