"""Group norm and modulated layer norm (segquant_groupnorm_quantize,
segquant_adanorm_quantize) against their formulas in fp64.

Tolerance of x, element by element.  Rounding to bf16 is off by at most 2^-8
relative.  Before it, in fp32: the sums behind the mean and the variance run
over at most 256 terms one after another (a thread's batches, then the joins),
so they are off by at most 256 * 2^-24 = 2^-16 of the sum of magnitudes, the
mean by 2^-16 max|z|, 1/sqrt(var + eps) by 2^-16 relative (half of twice
that), and the few products after it by less than 2^-20.  With A the factor in
front of z - mu that is 2^-16 (A max|z| + |t|); SiLU and GELU have slopes
below 1.13 and the activations' own error is below 2^-17.  Doubled: 2^-15 (A
max|z| + |t| + |x|).  Codes have to equal segquant_quantize_dualscale of x bit
for bit."""
import math

import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ACTS = {"none": S.SEGQ_ACT_NONE, "silu": S.SEGQ_ACT_SILU, "gelu": S.SEGQ_ACT_GELU}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def padded(data, ld, fill):
    """`data` [..., K] as bf16 rows `ld` apart, the padding set to `fill`."""
    buf = torch.full((*data.shape[:-1], ld), fill, device=DEV, dtype=BF)
    view = buf[..., :data.shape[-1]]
    view.copy_(data)
    return buf, view


def act_ref(t, act):
    if act == "silu":
        return t / (1 + torch.exp(-t))
    if act == "gelu":
        return t / 2 * torch.erfc(-t / math.sqrt(2.0))
    return t


def close(x, ref, A, zmax, t):
    """The module's tolerance; x bf16, the rest fp64 (broadcastable)."""
    err = (x.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -15 * (A.abs() * zmax + t.abs() + ref.abs()) + 2.0 ** -133
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err - tol)[bad].max()) if bad.any() else 0)


def groupnorm_ref(z, G, eps, gamma, beta, scale, shift, act):
    """(x, A, max|z| of the group, t) in fp64."""
    B, P, C = z.shape
    z = z.double().reshape(B, P, G, C // G)
    mu = z.mean((1, 3), keepdim=True)
    d = z - mu
    rstd = 1 / torch.sqrt((d * d).mean((1, 3), keepdim=True) + eps)
    zmax = z.abs().amax((1, 3), keepdim=True).expand_as(z).reshape(B, P, C)
    A = rstd.expand_as(z).reshape(B, P, C)
    t = (d * rstd).reshape(B, P, C)
    if gamma is not None:
        t, A = t * gamma.double(), A * gamma.double()
    if beta is not None:
        t = t + beta.double()
    if scale is not None:
        f = 1 + scale.double()[:, None]
        t, A = t * f, A * f
    if shift is not None:
        t = t + shift.double()[:, None]
    # cancelling terms of t are as large as their parts
    size = t.abs() + (beta.double().abs() * 4 if beta is not None else 0)
    return act_ref(t, act), A, zmax, size


GN = [
    # B, P, C, G, act, affine, modulated
    (1, 1, 1, 1, "none", False, False),
    (1, 1, 8, 8, "silu", True, False),        # one value per group: x = act(beta)
    (2, 1, 320, 32, "gelu", True, True),      # one pixel
    (2, 64, 1280, 32, "silu", True, False),   # one launch
    (3, 1369, 360, 24, "none", True, False),  # groups of 15
    (1, 5000, 72, 8, "gelu", True, True),     # groups of 9: 16-byte columns across groups
    (2, 4096, 640, 32, "silu", True, True),   # two launches
    (1, 33, 8, 8, "none", False, False),      # instance norm
    (2, 3001, 35, 5, "silu", True, False),    # C not a multiple of 8
    (1, 700, 5000, 4, "none", True, False),   # two column blocks, a group across them
    (1, 9000, 4104, 1, "silu", False, True),  # one group, two column blocks
    (1, 257, 8197, 1, "gelu", True, True),    # three column blocks, a short last piece
    (1, 65536, 128, 32, "silu", True, False),
    (4, 511, 24, 24, "none", True, True),     # groups of 1
    (1, 100000, 4, 2, "none", True, False),
]


@pytest.mark.parametrize("B,P,C,G,act,affine,mod", GN)
def test_groupnorm(B, P, C, G, act, affine, mod):
    g = gen(B * P + C)
    z = (normal(g, B, P, C) * torch.exp(normal(g, C)) + normal(g, C)).to(BF)
    gamma = 1 + 0.3 * normal(g, C) if affine else None
    beta = 0.3 * normal(g, C) if affine else None
    ld = -(-C // 8) * 8 + 8
    emb = (0.3 * normal(g, B, 2 * ld)).to(BF)
    scale, shift = (emb[:, :C], emb[:, ld:ld + C]) if mod else (None, None)
    zbuf, zv = padded(z, ld, float("nan"))        # what stands between rows is not read
    xbuf, xv = padded(torch.zeros_like(z), ld, 7.0)  # nor written
    S.segquant_groupnorm_quantize(zv, G, 1e-5, gamma, beta, scale, shift, ACTS[act], x_out=xv)
    ref, A, zmax, t = groupnorm_ref(z, G, 1e-5, gamma, beta, scale, shift, act)
    close(xv, ref, A, zmax, t)
    assert (xbuf[..., C:] == 7.0).all()
    # the same bits again, in place, and through codes
    x = S.segquant_groupnorm_quantize(zv, G, 1e-5, gamma, beta, scale, shift, ACTS[act],
                                      x_out=zv)[1]
    assert torch.equal(x.view(torch.int16), xv.view(torch.int16))


@pytest.mark.parametrize("layout", [S.SEGQ_Q_SIGNED, S.SEGQ_Q_PLANES])
@pytest.mark.parametrize("B,P,C,G,kseg,with_x", [
    (2, 64, 1280, 32, [1280], True),
    (2, 1024, 1920, 32, [1280, 640], False),
    (1, 3000, 200, 8, [64, 64, 72], True),
    (1, 77, 83, 1, [64, 19], False),
    (3, 2000, 83, 83, [64, 19], True),
])
def test_groupnorm_codes_are_the_quantiser_s(B, P, C, G, kseg, layout, with_x):
    g = gen(C)
    z = (normal(g, B, P, C) * 2).to(BF)
    _, z = padded(z, -(-C // 8) * 8, 0.0)
    args = (z, G, 1e-5, 1 + 0.3 * normal(g, C), 0.3 * normal(g, C), None, None, S.SEGQ_ACT_SILU)
    x = S.segquant_groupnorm_quantize(*args, x_out=True)[1]
    flat = x.reshape(B * P, C)
    _, flat = padded(flat, -(-C // 8) * 8, 0.0)
    act = S.segquant_calibrate_amax(flat, kseg)
    want = S.segquant_quantize_dualscale(flat, act, kseg, layout)
    ldq = want.shape[-1] + 16
    q = torch.full((*want.shape[:-1], ldq), 99, device=DEV, dtype=torch.int8)
    got, x2 = S.segquant_groupnorm_quantize(*args, act_scales=act, kseg=kseg, layout=layout, out=q,
                                            x_out=True if with_x else None)
    assert got is q and torch.equal(q[..., :C], want[..., :C])
    assert (q[..., C:] == 99).all()
    if with_x:
        assert torch.equal(x2, x)


@pytest.mark.parametrize("P", [40, 20000])  # one launch, two launches
def test_groupnorm_hard_values(P):
    """Equal values (variance 0), a mean far above the spread, and one huge value."""
    g = gen(P)
    C, G = 64, 8
    z = torch.empty(4, P, C, device=DEV, dtype=BF)
    z[0] = 3.0
    z[1] = 256 + 2 * (normal(g, P, C) > 0)
    z[2] = normal(g, P, C)
    z[2, 0, 0] = 1e6     # in the first batch of its group
    z[3] = normal(g, P, C)
    z[3, P - 1, C - 1] = -1e6  # in the last one
    x = S.segquant_groupnorm_quantize(z, G, 1e-5, x_out=True)[1]
    ref, A, zmax, t = groupnorm_ref(z, G, 1e-5, None, None, None, None, "none")
    assert (x[0] == 0).all()
    close(x, ref, A, zmax, t)
    # a mean of 2^8 spreads costs no more than the values' own size says, far
    # less than squares around zero would: var 1 against mean^2 2^16
    assert (x[1].double() - ref[1]).abs().max() < 2.0 ** -7


@pytest.mark.parametrize("value", [37.0, 255.0, 300.0, 1000.0])
def test_groupnorm_a_group_that_starts_in_the_last_channel_of_a_column_block(value):
    """Group 1 has one of its 2047 channels in the first block of 2048, whose
    first rows are unlike the rest: 8 of its 1.4 million values carry all the
    variance, so statistics joined around those 8 would lose 17 bits."""
    z = torch.zeros(1, 680, 3 * 2047, device=DEV, dtype=BF)
    _, z = padded(z, 6144, 0.0)
    z[0, :8, 2047] = value
    x = S.segquant_groupnorm_quantize(z, 3, 1e-5, x_out=True)[1]
    ref, A, zmax, t = groupnorm_ref(z, 3, 1e-5, None, None, None, None, "none")
    close(x, ref, A, zmax, t)


def test_groupnorm_rows_beyond_32_bit_offsets():
    B, P, C = 3, 700_000, 1032
    assert B * P * C > 2 ** 31
    z = torch.empty(B, P, C, device=DEV, dtype=BF)
    g = gen(5)
    for i in range(B):
        z[i] = torch.randn(P, C, generator=g, device=DEV, dtype=BF) * (i + 1) + i
    x = S.segquant_groupnorm_quantize(z, 8, 1e-5, x_out=True)[1]
    for i in range(B):
        for j in range(0, C, 129):  # one group at a time
            one = z[i:i + 1, :, j:j + 129]
            close(x[i:i + 1, :, j:j + 129],
                  *groupnorm_ref(one, 1, 1e-5, None, None, None, None, "none"))


# ------------------------------------------------------------- adanorm ----
def adanorm_ref(h, eps, gamma, beta, scale, shift, gate, branch, req):
    """(h', x, A, max|h'|, t) in fp64; req: request of each row."""
    h = h.double()
    if branch is not None:
        h = h + (gate.double()[req] * branch.double() if gate is not None else branch.double())
    stored = h.to(BF).double() if branch is not None else h
    d = stored - stored.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    t, A = d * rstd, rstd.expand_as(d)
    size = 0
    if gamma is not None:
        t, A = t * gamma.double(), A * gamma.double()
    if beta is not None:
        t = t + beta.double()
        size = 4 * beta.double().abs()
    if scale is not None:
        f = 1 + scale.double()[req]
        t, A = t * f, A * f
    if shift is not None:
        t = t + shift.double()[req]
        size = size + shift.double()[req].abs()
    return h, t, A, stored.abs().amax(1, keepdim=True), t.abs() + size


ADA = [
    # rows per request (None: equal requests), M, K, residual, affine
    ([1], 1, 1, False, False),
    ([77], 77, 1536, False, False),
    ([4096, 333], 4429, 1536, True, False),
    ([3, 0, 0, 5, 1], 9, 64, True, True),
    ([1] * 300, 300, 200, True, False),          # single rows, more requests than a wave
    ([2] * 3000, 6000, 72, False, True),         # many requests, several rows per wave
    ([i % 3 for i in range(270000)], 270000, 24, False, False),  # three steps of the search
    ([20000, 1, 0, 9999], 30000, 520, True, False),
    ([260], 260, 4096, True, True),              # the most a wave holds
    ([50, 250], 300, 4099, True, True),          # past it, a short last piece
    ([5, 6], 11, 16384, True, False),            # the most a workgroup holds
    ([5, 6], 11, 16391, True, True),             # rows read again
    ([7], 7, 61, False, False),
    (None, 12, 1000, True, False),
    (None, 900, 1003, False, True),
]


@pytest.mark.parametrize("lens,M,K,residual,affine", ADA)
def test_adanorm(lens, M, K, residual, affine):
    g = gen(M + K)
    R = 3 if lens is None else len(lens)
    if lens is None:
        off, req = None, torch.arange(M, device=DEV) // (M // R)
        before = after = 0
    else:
        before, after = 2, 5  # rows of no request around the batch
        off = torch.tensor([before] + lens, device=DEV).cumsum(0).to(torch.int32)
        req = torch.repeat_interleave(torch.arange(R, device=DEV), torch.tensor(lens, device=DEV))
    rows = M + before + after
    ld = -(-K // 8) * 8 + 8
    data = (normal(g, rows, K) * torch.exp(normal(g, K)) + 0.5).to(BF)
    _, h = padded(data, ld, float("nan"))
    mods = (0.4 * normal(g, R, 3 * ld)).to(BF)
    shift, scale, gate = (mods[:, i * ld:i * ld + K] for i in range(3))
    gamma = 1 + 0.3 * normal(g, K) if affine else None
    beta = 0.3 * normal(g, K) if affine else None
    branch = None
    if residual:
        _, branch = padded(normal(g, rows, K), ld, float("nan"))
    xbuf, x = padded(torch.zeros_like(data), ld, 7.0)
    xbuf.fill_(7.0)
    hbuf, ho = padded(torch.zeros_like(data), ld, 5.0)
    hbuf.fill_(5.0)
    args = dict(eps=1e-6, gamma=gamma, beta=beta, scale=scale, shift=shift,
                gate=gate if residual else None, branch=branch, row_offset=off)
    S.segquant_adanorm_quantize(h, x_out=x, h_out=ho if residual else None, **args)
    mine = slice(before, before + M)
    href, ref, A, hmax, t = adanorm_ref(
        data[mine], 1e-6, gamma, beta, scale, shift, gate if residual else None,
        branch[mine] if residual else None, req)
    if residual:
        # h' rounds once, so it may be the neighbour of the fp64 sum's rounding
        err = (ho[mine].double() - href).abs()
        assert (err <= 2.0 ** -8 * href.abs() * (1 + 2.0 ** -14) + 2.0 ** -133).all()
        # and x is held to the h' that was stored
        _, ref, A, hmax, t = adanorm_ref(ho[mine], 1e-6, gamma, beta, scale, shift, None, None, req)
    close(x[mine], ref, A, hmax, t)
    for buf, fill in ((xbuf, 7.0), (hbuf, 5.0)):
        if buf is hbuf and not residual:
            continue
        assert (buf[:before] == fill).all() and (buf[before + M:] == fill).all()
        assert (buf[:, K:] == fill).all()
    if residual:  # the residual stream updated in place
        x2 = torch.zeros_like(data)
        _, x2 = padded(x2, ld, 0.0)
        S.segquant_adanorm_quantize(h, x_out=x2, h_out=h, **args)
        assert torch.equal(x2[mine], x[mine]) and torch.equal(h[mine], ho[mine])
        assert torch.equal(h[before + M:], data[before + M:])


@pytest.mark.parametrize("layout", [S.SEGQ_Q_SIGNED, S.SEGQ_Q_PLANES])
@pytest.mark.parametrize("M,K,kseg", [
    (77, 1536, [1536]), (600, 1536, [64] * 24), (40, 83, [64, 19]), (9, 16448, [16384, 64])])
def test_adanorm_codes_are_the_quantiser_s(M, K, kseg, layout):
    g = gen(M)
    _, h = padded(normal(g, M, K), -(-K // 8) * 8, 0.0)
    mods = (0.3 * normal(g, 1, 2 * (-(-K // 8) * 8))).to(BF)
    scale, shift = mods[:, :K], mods[:, -(-K // 8) * 8:][:, :K]
    x = S.segquant_adanorm_quantize(h, scale=scale, shift=shift, x_out=True)[1]
    act = S.segquant_calibrate_amax(x, kseg)
    want = S.segquant_quantize_dualscale(x, act, kseg, layout)
    for x_out in (True, None):
        q, x2, _ = S.segquant_adanorm_quantize(h, scale=scale, shift=shift, act_scales=act,
                                               kseg=kseg, layout=layout, x_out=x_out)
        assert torch.equal(q[..., :K], want[..., :K])
        assert x2 is None or torch.equal(x2, x)


def test_adanorm_only_the_residual_and_an_empty_batch():
    g = gen(1)
    h, y = normal(g, 20, 128).to(BF), normal(g, 20, 128).to(BF)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)  # three requests without rows
    out = torch.full_like(h, 3.0)
    S.segquant_adanorm_quantize(h, branch=y, h_out=out, row_offset=off)
    assert (out == 3.0).all()
    _, x, ho = S.segquant_adanorm_quantize(h, branch=y, h_out=True)
    assert x is None and torch.equal(ho, (h.float() + y.float()).to(BF))
    _, x, _ = S.segquant_adanorm_quantize(h[:0], x_out=True)
    assert x.shape == (0, 128)


@pytest.mark.parametrize("off", [[0, 100, 50, 120], [120, 0, 0, 0], [-5, 40, 4000, 70], [7] * 4])
def test_offsets_out_of_order_stay_in_bounds(off):
    """Unordered or far offsets name rows inside the batch only; rows that an
    ordered pair covers alone are right."""
    g = gen(3)
    M, K = 130, 128
    buf = torch.full((M + 64, K), 9.0, device=DEV, dtype=BF)
    h = normal(g, M, K).to(BF)
    S.segquant_adanorm_quantize(h, x_out=buf[32:32 + M],
                                row_offset=torch.tensor(off, device=DEV, dtype=torch.int32))
    assert (buf[:32] == 9.0).all() and (buf[32 + M:] == 9.0).all()


def test_adanorm_rows_beyond_32_bit_offsets():
    M, K = 1_400_000, 1600
    assert M * K > 2 ** 31
    h = torch.randn(M, K, generator=gen(2), device=DEV, dtype=BF)
    off = torch.tensor([0, 1_000_000, M], device=DEV, dtype=torch.int32)
    shift = torch.tensor([[1.0], [-2.0]], device=DEV, dtype=BF).expand(2, K).contiguous()
    x = S.segquant_adanorm_quantize(h, shift=shift, row_offset=off, x_out=True)[1]
    for at in (0, 999_999, 1_000_000, 1_350_000, M - 2):
        rows = slice(at, min(M, at + 2))
        req = (torch.arange(at, min(M, at + 2), device=DEV) >= 1_000_000).long()
        _, ref, A, hmax, t = adanorm_ref(h[rows], 1e-6, None, None, None, shift, None, None, req)
        close(x[rows], ref, A, hmax, t)


def test_norms_on_another_stream_and_in_a_graph():
    """Captured once, replayed on new inputs between eager calls, both kernels
    of each path among them."""
    g = gen(8)
    z, h = normal(g, 2, 4096, 320).to(BF), normal(g, 500, 256).to(BF)
    off = torch.tensor([0, 100, 480], device=DEV, dtype=torch.int32)
    ws = torch.empty(S.segquant_groupnorm_workspace_bytes(2, 4096, 320, 32), dtype=torch.uint8,
                     device=DEV)
    assert ws.numel() > 0
    x, y = torch.zeros_like(z), torch.zeros_like(h)

    def both(xo, yo, work):
        S.segquant_groupnorm_quantize(z, 32, act_kind=S.SEGQ_ACT_SILU, x_out=xo, workspace=work)
        S.segquant_adanorm_quantize(h, x_out=yo, row_offset=off)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(x, y, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(x, y, ws)
    for i in range(4):
        z.copy_(normal(g, 2, 4096, 320))
        h.copy_(normal(g, 500, 256))
        off.copy_(torch.tensor([i, 90 + i, 470 + i], device=DEV))
        x.zero_(), y.zero_()
        graph.replay()
        ex, ey = torch.zeros_like(z), torch.zeros_like(h)
        both(ex, ey, "auto")
        torch.cuda.synchronize()
        assert torch.equal(x, ex) and torch.equal(y, ey)
