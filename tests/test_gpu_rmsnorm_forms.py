"""Every form of the root-mean-square norm: several rows to a wave or workgroup, outputs
past the caches, rows beyond the registers and more of them than workgroups; all outputs
at once, with the residual stream in place.

h', codes and MXFP4 have to be equal bit for bit to their definitions on what the call
itself stored; x is within 2^-8 + 2^-15 of its value, as test_gpu_rmsnorm.py derives."""
import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV
from test_gpu_rmsnorm import close

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rows(g, M, K):
    out = torch.empty(M, -(-K // 8) * 8, device=DEV, dtype=BF)[:, :K]
    step = max(1, (1 << 27) // K)
    for i in range(0, M, step):
        part = out[i:i + step]
        part.copy_(torch.randn(part.shape, generator=g, device=DEV))
    return out


def parts(M, K):
    step = max(1, (1 << 26) // K)
    return [slice(i, min(M, i + step)) for i in range(0, M, step)]


def same_matrix(got, want, M, K):
    """Codes and scales that count: of M rows, of the columns up to the last tile's end."""
    n, kt, ks = -(-M // 16), -(-K // 128), -(-K // 512)
    a, b = (m[0].view(n, kt, 4, 16, 16).transpose(2, 3).transpose(1, 2).reshape(16 * n, -1)
            for m in (got, want))
    assert torch.equal(a[:M], b[:M])
    a, b = (m[1].view(n, ks, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(16 * n, -1)
            for m in (got, want))
    assert torch.equal(a[:M, :4 * kt], b[:M, :4 * kt])


# rows to a wave: 2 (a whole last row group or not), 9, 16; x and h' past the caches; five
# pieces a lane and more, where no row is loaded ahead; a workgroup a row
@pytest.mark.parametrize("M,K,place", [(9000, 576, "h"), (9001, 64, "branch"), (72000, 192, "h"),
                                       (140001, 64, None), (45000, 1536, "h"), (45001, 1536, None),
                                       (10007, 2560, "branch"), (8500, 4096, "h"), (600, 8192, "h"),
                                       (9000, 1531, "h"), (45000, 1533, "branch"),
                                       (2100, 16448, "h"), (700, 50000, "branch")])
def test_every_output_at_once(M, K, place):
    g = gen(M + K)
    h, branch = rows(g, M, K), rows(g, M, K)
    gamma = 1 + 0.3 * torch.randn(K, generator=g, device=DEV)
    first = 64 * max(1, K // 128)
    kseg = [first, K - first] if first < K else [K]
    act = torch.rand(4, len(kseg), generator=g, device=DEV) * 0.02 + 0.02
    act[2:] = 1 / act[:2]
    want = torch.empty(M, K, device=DEV, dtype=BF)
    for p in parts(M, K):
        want[p] = (h[p].float() + branch[p].float()).to(BF)
    h_out = dict(h=h, branch=branch).get(place, True)
    whole = K % 64 == 0
    q, x, stored, mx = S.segquant_rmsnorm_quantize(h, 1e-6, gamma, branch, act_scales=act, kseg=kseg,
                                                   x_out=True, h_out=h_out,
                                                   mx_out=True if whole else None)
    assert torch.equal(stored, want) and (place is None or stored is h_out)
    for p in parts(M, K):
        close(x[p], want[p], gamma, 1e-6)
    assert torch.equal(q[:, :K], S.segquant_quantize_dualscale(x, act, kseg)[:, :K])
    if whole:
        same_matrix(mx, S.segquant_quantize_mxfp4(x), M, K)


@pytest.mark.parametrize("M,K", [((1 << 24) + 77, 64), ((1 << 20) + 2051, 4160), (65539, 16448)])
def test_more_rows_than_groups_of_them(M, K):
    """More than 2^20 workgroups' worth of rows, one row to each: rows at the ends and in
    between are those of calls on them alone."""
    g = gen(K)
    h = rows(g, M, K)
    gamma = 1 + 0.3 * torch.randn(K, generator=g, device=DEV)
    mx = S.segquant_rmsnorm_quantize(h, 1e-6, gamma, mx_out=True)[3]
    kt, ks = -(-K // 128), -(-K // 512)
    for first in (0, 16 * (M // 32), 65536, (M - 1) // 16 * 16 - 512):
        n = min(544, M - first)
        part = S.segquant_rmsnorm_quantize(h[first:first + n], 1e-6, gamma, mx_out=True)[3]
        codes = mx[0][first // 16 * kt * 1024:][:part[0].numel()]
        scales = mx[1][first // 16 * ks * 256:][:part[1].numel()]
        same_matrix((codes, scales), part, n, K)
