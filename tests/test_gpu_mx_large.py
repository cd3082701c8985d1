"""MXFP4 products of very many rows or columns: offsets that pass 32 bits, grids of
hundreds of thousands of workgroups; the ends and the middle are those of calls on
them alone (K = 64 is one instruction, so every form gives the same bits)."""
import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
K = 64


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def random_matrix(g, R):
    """Codes of every value, scales near 1."""
    n, m = S.segquant_mxfp4_bytes(R, K)
    codes = torch.randint(0, 256, (n,), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(124, 131, (m,), generator=g, device=DEV, dtype=torch.uint8)
    tile = codes.view(-1, 4, 256)
    tile[:, 2:] = 0  # columns 64 .. 127 of the tile
    scales.view(-1, 64, 4)[:, 32:] = 0
    return codes, scales


def part(mx, first, rows):
    """Rows first (a multiple of 16) and on, as a matrix of their own."""
    n, m = S.segquant_mxfp4_bytes(rows, K)
    return mx[0][first // 16 * 1024:][:n], mx[1][first // 16 * 256:][:m]


@pytest.mark.parametrize("M,N", [((1 << 25) + 77, 80), ((1 << 23) + 5, 512)])
def test_many_rows(M, N):
    g = gen(N)
    x, w = random_matrix(g, M), random_matrix(g, N)
    y = S.segquant_gemm_mxfp4(None, w, N, K=K, xq=x, M=M)
    for first in (0, M // 32 * 16, (M - 1) // 16 * 16 - 256):
        n = min(300, M - first)
        assert torch.equal(S.segquant_gemm_mxfp4(None, w, N, K=K, xq=part(x, first, n), M=n),
                           y[first:first + n])


@pytest.mark.parametrize("M,N", [(1, (1 << 25) + 16), (16, (1 << 24) + 48), (300, (1 << 24) + 16)])
def test_many_columns(M, N):
    g = gen(M)
    x, w = random_matrix(g, M), random_matrix(g, N)
    y = S.segquant_gemm_mxfp4(None, w, N, K=K, xq=x, M=M)
    for first in (0, N // 32 * 16, N - 256):
        n = min(304, N - first)
        assert torch.equal(S.segquant_gemm_mxfp4(None, part(w, first, n), n, K=K, xq=x, M=M),
                           y[:, first:first + n])


def test_no_rows_of_a_norm():
    h = torch.zeros(0, 128, device=DEV, dtype=BF)
    act = torch.ones(4, 1, device=DEV)
    q, x, stored, mx = S.segquant_rmsnorm_quantize(h, branch=h, act_scales=act, x_out=True, h_out=True,
                                                   mx_out=True)
    assert x.shape == stored.shape == (0, 128) and mx[0].numel() == mx[1].numel() == 0
    assert S.segquant_gemm_mxfp4(None, random_matrix(gen(1), 32), 32, K=K,
                                 xq=S.segquant_quantize_mxfp4(h[:, :64].contiguous()),
                                 M=0).shape == (0, 32)
    q = torch.zeros(0, 5, 2, 16, device=DEV, dtype=BF)
    pos = torch.zeros(5, 1, device=DEV, dtype=torch.int32)
    freq = S.segquant_rotary_frequencies([16]).to(DEV)
    assert S.segquant_qk_rotary(q, q, pos, freq, [16])[1].shape == q.shape
