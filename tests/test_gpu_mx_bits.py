"""The MXFP4 product of bf16 rows gives the bits of its codes' product: from
bf16, quantised inside the kernel or ahead of it, behind any activation.  Every
large product has its negative elsewhere in K, so what is left shows the order of
the sums."""
import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

ACTS = {"none": S.SEGQ_ACT_NONE, "silu": S.SEGQ_ACT_SILU, "gelu": S.SEGQ_ACT_GELU}


def operands(M, N, K):
    g = torch.Generator(device=DEV)
    g.manual_seed(M + K)
    z = torch.randn(M, K, generator=g, device=DEV).abs()
    w = torch.randn(K, N, generator=g, device=DEV)
    half = (K - 64) // 64 * 32
    if half:  # z w of 2^0 to 2^26, its negative, and some columns that nothing cancels
        of_block = torch.arange(K, device=DEV) // 32
        power = torch.randint(0, 14, (2, K), generator=g, device=DEV)[:, of_block].float()
        z, w = z * torch.exp2(power[0]), w * torch.exp2(power[1])[:, None]
        z[:, 64 + half:64 + 2 * half] = z[:, 64:64 + half]
        w[64 + half:64 + 2 * half] = -w[64:64 + half]
        order = torch.randperm(K // 32, generator=g, device=DEV)
        order = (32 * order[:, None] + torch.arange(32, device=DEV)).flatten()
        z, w = z[:, order].contiguous(), w[order].contiguous()
    return z.to(torch.bfloat16), S.segquant_quantize_weight_mxfp4(w)


def same_bits(M, N, K, act):
    z, w = operands(M, N, K)
    y = S.segquant_gemm_mxfp4(z, w, N, act_kind=ACTS[act])
    mx = S.segquant_quantize_mxfp4(z, ACTS[act])
    assert torch.equal(y, S.segquant_gemm_mxfp4(None, w, N, K=K, xq=mx, M=M))


# 4, 8 and 16 waves, one and two column tiles, quantised inside (the first ten) and ahead
@pytest.mark.parametrize("M,N,K", [(4, 64, 6144), (3, 80, 8192), (1, 4096, 24576), (6, 4096, 4096),
                                   (6, 4112, 4096), (5, 96, 2048), (7, 48, 1984), (2, 8192, 5120),
                                   (8, 8208, 1536), (3, 16, 64), (16, 1536, 6144), (9, 8192, 4096),
                                   (16, 80, 1984), (13, 4112, 2048)])
@pytest.mark.parametrize("act", list(ACTS))
def test_up_to_16_rows(M, N, K, act):
    same_bits(M, N, K, act)


# quantised inside by each workgroup (the first six, two and four column tiles) and ahead
@pytest.mark.parametrize("M,N,K", [(17, 48, 64), (31, 2064, 1472), (48, 4624, 1536), (77, 1536, 1536),
                                   (250, 512, 640), (1000, 64, 576), (77, 1536, 1600),
                                   (300, 6144, 512), (40, 96, 6144), (4429, 1536, 1536)])
def test_more_rows(M, N, K):
    same_bits(M, N, K, "none")


def test_which_are_quantised_inside():
    inside = [S.segquant_gemm_mxfp4_workspace_bytes(*s) == 0
              for s in [(4, 64, 6144), (1, 4096, 24576), (6, 4096, 4096), (7, 48, 1536), (8, 8208, 1536),
                        (16, 1536, 6144), (9, 8192, 4096), (16, 80, 1984), (13, 4112, 2048)]]
    assert inside == [True] * 5 + [False] * 4
