"""Residual update and root-mean-square norm (segquant_rmsnorm_quantize) against
its formula in fp64.

Tolerance of x, element by element: its rounding to bf16 2^-8 |x|; the sum of
squares has positive terms only and runs over at most 256 of them one after
another, so it is off by at most 2^-16 of itself and its root by 2^-17, the
hardware's 1/sqrt by 2^-22 and the two products by 2^-23: 2^-15 |x| in all.  h',
codes and MXFP4 have to be equal bit for bit to their definitions on what the
call itself stored."""
import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def padded(data, ld, fill):
    buf = torch.full((*data.shape[:-1], ld), fill, device=DEV, dtype=BF)
    view = buf[..., :data.shape[-1]]
    view.copy_(data)
    return buf, view


def close(x, h, gamma, eps):
    h = h.double()
    ref = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    if gamma is not None:
        ref = ref * gamma.double()
    err, tol = (x.double() - ref).abs(), (2.0 ** -8 + 2.0 ** -15) * ref.abs() + 2.0 ** -133
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))


@pytest.mark.parametrize("M,K", [(1, 1), (2, 8), (3, 7), (77, 1536), (257, 64), (300, 1533),
                                 (1000, 72), (520, 2048), (300, 2560), (290, 4096), (9000, 328),
                                 (300, 4100), (20, 16384), (7, 16391), (3, 40000)])
@pytest.mark.parametrize("residual,affine", [(False, True), (True, False), (True, True)])
def test_rmsnorm(M, K, residual, affine):
    g = gen(M * 7 + K)
    ld = -(-K // 8) * 8 + 8
    h = (normal(g, M, K) * torch.exp(normal(g, M, 1))).to(BF)
    _, h = padded(h, ld, float("nan"))
    branch = padded(normal(g, M, K).to(BF), ld + 8, float("nan"))[1] if residual else None
    gamma = 1 + 0.3 * normal(g, K) if affine else None
    xbuf, x = padded(torch.zeros(M, K, device=DEV, dtype=BF), ld, 7.0)
    hbuf, h_out = padded(torch.zeros(M, K, device=DEV, dtype=BF), ld, 7.0)
    q, got, stored, mx = S.segquant_rmsnorm_quantize(h, 1e-6, gamma, branch, x_out=x,
                                                     h_out=h_out if residual else None)
    assert q is None and mx is None and got is x
    want = h
    if residual:
        want = (h.float() + branch.float()).to(BF)
        assert torch.equal(stored, want) and (hbuf[:, K:] == 7.0).all()
    close(x, want, gamma, 1e-6)
    assert (xbuf[:, K:] == 7.0).all()
    again = S.segquant_rmsnorm_quantize(h, 1e-6, gamma, branch, x_out=True)[1]
    assert torch.equal(again, x)
    if residual:  # in place
        for target in (h, branch):
            keep = target.clone()
            S.segquant_rmsnorm_quantize(h, 1e-6, gamma, branch, h_out=target)
            assert torch.equal(target, want)
            target.copy_(keep)


@pytest.mark.parametrize("layout", [S.SEGQ_Q_SIGNED, S.SEGQ_Q_PLANES])
@pytest.mark.parametrize("M,K,kseg", [(77, 1536, [1024, 512]), (300, 1533, [64, 1469]),
                                      (1, 64, [64]), (5, 20000, [10048, 9952]), (900, 83, [64, 19])])
def test_codes_are_the_quantiser_s(M, K, kseg, layout):
    g = gen(K)
    ld = -(-K // 8) * 8
    h = padded((2 * normal(g, M, K)).to(BF), ld, 0.0)[1]
    gamma = 1 + 0.3 * normal(g, K)
    x = S.segquant_rmsnorm_quantize(h, gamma=gamma, x_out=True)[1]
    act = S.segquant_calibrate_amax(x, kseg)
    want = S.segquant_quantize_dualscale(x, act, kseg, layout)
    q = torch.full((*want.shape[:-1], want.shape[-1] + 16), 99, device=DEV, dtype=torch.int8)
    got = S.segquant_rmsnorm_quantize(h, gamma=gamma, act_scales=act, kseg=kseg, layout=layout,
                                      out=q)[0]
    assert got is q and torch.equal(q[..., :K], want[..., :K]) and (q[..., K:] == 99).all()


@pytest.mark.parametrize("M,K", [(1, 64), (17, 192), (77, 1536), (300, 576), (600, 4096), (33, 8192),
                                 (5, 16448), (3, 20032)])
def test_mxfp4_is_the_quantiser_s(M, K):
    g = gen(K + M)
    h, branch = normal(g, M, K).to(BF), normal(g, M, K).to(BF)
    h[0] = 0  # a row of zeros
    branch[0] = 0
    gamma = 1 + 0.3 * normal(g, K)
    n, m = S.segquant_mxfp4_bytes(M, K)
    codes = torch.full((n,), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((m,), 0xAB, dtype=torch.uint8, device=DEV)
    act = torch.ones(4, 1, device=DEV)
    q, x, stored, _ = S.segquant_rmsnorm_quantize(h, gamma=gamma, branch=branch, x_out=True,
                                                  h_out=True, act_scales=act,
                                                  mx_out=(codes, scales))
    want = S.segquant_quantize_mxfp4(x)
    rows, kt, ks = -(-M // 16), -(-K // 128), -(-K // 512)

    def of_rows(mx):  # [row][...]: what belongs to rows and to the columns of whole tiles
        c = mx[0].view(rows, kt, 4, 16, 16).transpose(2, 3).transpose(1, 2).reshape(16 * rows, -1)
        s = mx[1].view(rows, ks, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(16 * rows, -1)
        return c[:M], s[:M, :4 * kt]
    for a, b in zip(of_rows((codes, scales)), of_rows(want)):
        assert torch.equal(a, b)
    if M % 16:  # rows behind the last are left alone
        assert (codes.view(rows, kt, 4, 16, 16)[-1, :, :, M % 16:] == 0xAB).all()
    assert torch.equal(q[:, :K], S.segquant_quantize_dualscale(x, act)[:, :K])
    close(x, stored, gamma, 1e-6)
    assert not x[0].any()


def test_large_and_small_values():
    """Up to 2^60, a row of one value, and a row whose squares vanish beside eps."""
    K = 512
    h = torch.zeros(5, K, device=DEV)
    h[0], h[1, 3], h[2], h[3] = 2.0 ** 59, 1e15, 1e-30, -3.0
    h[4, ::2] = 1e-3
    h = h.to(BF)
    x = S.segquant_rmsnorm_quantize(h, 1e-6, x_out=True)[1]
    close(x, h, None, 1e-6)


def test_no_rows_other_stream_and_graph():
    g = gen(1)
    x = S.segquant_rmsnorm_quantize(torch.zeros(0, 64, device=DEV, dtype=BF), x_out=True)[1]
    assert x.shape == (0, 64)
    h, branch = normal(g, 333, 640).to(BF), normal(g, 333, 640).to(BF)
    want = S.segquant_rmsnorm_quantize(h, branch=branch, x_out=True, h_out=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = S.segquant_rmsnorm_quantize(h, branch=branch, x_out=True, h_out=True)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    out = torch.empty_like(h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.segquant_rmsnorm_quantize(h, branch=branch, x_out=out)
    for _ in range(3):
        h.copy_(normal(g, 333, 640))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, S.segquant_rmsnorm_quantize(h, branch=branch, x_out=True)[1])


def test_rows_far_apart():
    """Row distances that pass 32 bits, in elements and in bytes."""
    g = gen(31)
    M, K, far = 4, 192, (1 << 30) + 64
    h = torch.empty(M * far, device=DEV, dtype=BF).view(M, far)[:, :K]
    x = torch.empty(M * far, device=DEV, dtype=BF).view(M, far)[:, :K]
    h.copy_(normal(g, M, K))
    S.segquant_rmsnorm_quantize(h, x_out=x)
    assert torch.equal(x, S.segquant_rmsnorm_quantize(h.contiguous(), x_out=True)[1])
