"""Root-mean-square norms of rows and heads whose squares overflow fp32, against
the formula in fp64.

Tolerance of a row's x: its rounding to bf16 2^-8 |x|; at most 256 squares one after
another in the sum, so 2^-16 of it and 2^-17 of its root, the hardware's 1/sqrt
2^-22, that root below 2^-126 off by half of its last bit, 2^-22, and the two
products 2^-23: below 2^-15 |x| in all."""
import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
LARGEST = float(torch.finfo(BF).max)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def norm_ref(h, gamma, eps):
    h = h.double()
    ref = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return ref if gamma is None else ref * gamma.double()


def close(x, ref):
    err, tol = (x.double() - ref).abs(), (2.0 ** -8 + 2.0 ** -15) * ref.abs() + 2.0 ** -133
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))


def rows(g, M, K):
    """Ordinary rows, and among them rows of 2^59, 2^63, the largest value, one large
    value beside small ones, and values from 2^-40 to the largest."""
    h = normal(g, M, K)
    kind = torch.arange(M, device=DEV) % 7
    h[kind == 1] = 2.0 ** 59
    h[kind == 2] = torch.sign(h[kind == 2]) * 2.0 ** 63
    h[kind == 3] = torch.sign(h[kind == 3]) * LARGEST
    h[kind == 4, K // 2] = LARGEST
    wide = torch.rand(int((kind == 5).sum()), K, generator=g, device=DEV)
    h[kind == 5] = torch.sign(h[kind == 5]) * torch.exp2(-40 + 167 * wide)
    return h.to(BF)


# a workgroup a row, a wave a row, whole pieces or not, rows beyond the registers
@pytest.mark.parametrize("M,K", [(7, 1), (7, 8), (14, 1024), (21, 1533), (70, 8192), (15, 16384),
                                 (300, 512), (301, 1029), (300, 4096), (9000, 2048), (14, 16448),
                                 (7, 40003)])
@pytest.mark.parametrize("residual,affine", [(False, True), (True, False)])
def test_rows_whose_squares_overflow(M, K, residual, affine):
    g = gen(M + K)
    h = torch.zeros(M, -(-K // 8) * 8, device=DEV, dtype=BF)[:, :K]
    h.copy_(rows(g, M, K))
    gamma = 1 + 0.3 * normal(g, K) if affine else None
    branch = None
    if residual:  # never past the largest value
        branch = torch.zeros(M, -(-K // 8) * 8, device=DEV, dtype=BF)[:, :K]
        branch.copy_(torch.where(h.abs() > 2.0 ** 100, 0, normal(g, M, K)))
    q, x, stored, _ = S.segquant_rmsnorm_quantize(h, 1e-6, gamma, branch, x_out=True,
                                                  h_out=True if residual else None)
    want = stored if residual else h
    if residual:
        assert torch.equal(stored, (h.float() + branch.float()).to(BF))
    close(x, norm_ref(want, gamma, 1e-6))


@pytest.mark.parametrize("M,K", [(14, 1536), (280, 1536), (14, 16448)])
def test_codes_and_mxfp4_of_rows_whose_squares_overflow(M, K):
    g = gen(K)
    h = rows(g, M, K)
    kseg = [1024, K - 1024]
    x = S.segquant_rmsnorm_quantize(h, x_out=True)[1]
    act = S.segquant_calibrate_amax(x, kseg)
    q, again, _, mx = S.segquant_rmsnorm_quantize(h, x_out=True, act_scales=act, kseg=kseg,
                                                  mx_out=True)
    assert torch.equal(again, x)
    assert torch.equal(q[:, :K], S.segquant_quantize_dualscale(x, act, kseg)[:, :K])
    want = S.segquant_unpack_mxfp4(S.segquant_quantize_mxfp4(x), M, K)
    assert torch.equal(S.segquant_unpack_mxfp4(mx, M, K), want)


@pytest.mark.parametrize("eps", [2.0 ** -126, 1.0, 2.0 ** 127])
def test_an_eps_of_any_size(eps):
    g = gen(3)
    h = rows(g, 35, 1024)
    close(S.segquant_rmsnorm_quantize(h, eps, x_out=True)[1], norm_ref(h, None, eps))


def test_infinities_are_still_their_rows():
    g = gen(4)
    h = rows(g, 300, 640)
    clean = S.segquant_rmsnorm_quantize(h, x_out=True)[1]
    bad = h.clone()
    bad[5, 3], bad[290, 639] = float("inf"), float("nan")
    x = S.segquant_rmsnorm_quantize(bad, x_out=True)[1]
    hit = torch.zeros(300, dtype=torch.bool, device=DEV)
    hit[5] = hit[290] = True
    assert torch.equal(x[~hit], clean[~hit])
    assert x[5, 3].isnan() and x[290].isnan().all()


@pytest.mark.parametrize("B,L,Hq,Hk,D,R", [(1, 7, 3, 1, 16, 16), (2, 50, 7, 2, 40, 32),
                                           (1, 33, 24, 24, 64, 64), (1, 700, 24, 12, 64, 64),
                                           (1, 900, 16, 16, 128, 128), (1, 300, 40, 10, 72, 48),
                                           (1, 6, 4, 2, 256, 64), (1, 5, 3, 2, 512, 512)])
@pytest.mark.parametrize("style", [S.SEGQ_ROTARY_PAIRS, S.SEGQ_ROTARY_HALVES])
def test_heads_whose_squares_overflow(B, L, Hq, Hk, D, R, style):
    """The norm's factor is off by less than 2^-19 (21 * 2^-24 of the sum, halved by the
    root, that root's 2^-22 and a few roundings), sine and cosine by less than 2^-22:
    2^-18 (|a| + |b|) of a pair, besides the rounding to bf16."""
    g = gen(D + L)
    pos = torch.randint(-5000, 20000, (L, 1), generator=g, device=DEV, dtype=torch.int32)
    freq = S.segquant_rotary_frequencies([R]).to(DEV)
    q, k = (rows(g, B * L * H, D).view(B, L, H, D) for H in (Hq, Hk))
    gq, gk = 1 + 0.3 * normal(g, D), 1 + 0.3 * normal(g, D)
    got = S.segquant_qk_rotary(q, k, pos, freq, [R], style, gq, gk)
    u = pos.double() * freq
    c, s = torch.cos(u)[:, None], torch.sin(u)[:, None]
    for t, gamma, y in ((q, gq, got[0]), (k, gk, got[1])):
        t = norm_ref(t, gamma, 1e-6)
        out, size = t.clone(), t.abs()
        a, b = ((slice(0, R, 2), slice(1, R, 2)) if style == S.SEGQ_ROTARY_PAIRS
                else (slice(0, R // 2), slice(R // 2, R)))
        out[..., a] = t[..., a] * c - t[..., b] * s
        out[..., b] = t[..., b] * c + t[..., a] * s
        size[..., a] = size[..., b] = t[..., a].abs() + t[..., b].abs()
        err, tol = (y.double() - out).abs(), 2.0 ** -8 * out.abs() + 2.0 ** -18 * size + 2.0 ** -133
        assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))


def test_large_heads_without_the_norm():
    g = gen(6)
    q = rows(g, 70, 64).view(1, 10, 7, 64)
    freq = S.segquant_rotary_frequencies([16]).to(DEV)
    pos = torch.zeros(10, 1, device=DEV, dtype=torch.int32)
    assert torch.equal(S.segquant_qk_rotary(q, None, pos, freq, [16], norm=False)[0], q)
