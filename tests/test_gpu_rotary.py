"""Norm and rotary positions of q and k (segquant_qk_rotary) against the formula
in fp64.

Tolerance, element by element, with a pair (a, b) of the normalised head: the
rounding to bf16 2^-8 |out|; the norm's factor is off by less than 2^-19 (up to
16 squares one after another in a lane, then five joins: 21 * 2^-24, halved by
the root, and a few roundings), sine and cosine by less than 2^-22: 2^-18 (|a| +
|b|) in all."""
import math
from fractions import Fraction

import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
PAIRS, HALVES = S.SEGQ_ROTARY_PAIRS, S.SEGQ_ROTARY_HALVES


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def rotary_ref(x, pos, freq, widths, style, gamma, eps, norm):
    """(out, tolerance) in fp64; x [B][L][H][D], pos [L][A] or [B][L][A]."""
    t = x.double()
    D, R = t.shape[-1], sum(widths)
    if norm:
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)
        if gamma is not None:
            t = t * gamma.double()
    out, size, at = t.clone(), t.abs().clone(), 0
    for axis, w in enumerate(widths):
        for i in range(at, at + w // 2):
            u = pos[..., axis].double() * freq[i].to(pos.device)
            c, s = torch.cos(u)[..., None], torch.sin(u)[..., None]
            a, b = (2 * i, 2 * i + 1) if style == PAIRS else (i, i + R // 2)
            out[..., a] = t[..., a] * c - t[..., b] * s
            out[..., b] = t[..., b] * c + t[..., a] * s
            size[..., a] = size[..., b] = t[..., a].abs() + t[..., b].abs()
        at += w // 2
    return out, 2.0 ** -8 * out.abs() + 2.0 ** -18 * size + 2.0 ** -133


def close(got, ref, tol):
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))


CASES = [
    # B, L, Hq, Hk, D, widths, style, norm, gamma
    (1, 1, 1, 1, 8, [0], PAIRS, True, True),
    (1, 1, 1, 1, 16, [16], PAIRS, True, True),
    (1, 7, 3, 1, 16, [16], HALVES, True, False),
    (2, 5, 2, 2, 40, [32], HALVES, True, True),
    (1, 77, 24, 24, 64, [64], HALVES, True, True),
    (1, 333, 24, 24, 64, [16, 24, 24], PAIRS, True, True),
    (2, 50, 24, 8, 64, [32, 32], PAIRS, False, False),
    (1, 600, 12, 12, 128, [44, 42, 42], HALVES, True, True),
    (3, 200, 16, 4, 128, [16, 56, 56], PAIRS, True, False),
    (1, 40, 5, 3, 72, [10, 54], PAIRS, True, True),
    (1, 9, 7, 7, 96, [0, 96, 0], HALVES, True, True),
    (2, 11, 4, 2, 256, [64], HALVES, True, True),
    (1, 6, 3, 1, 512, [200, 2, 310], PAIRS, True, True),
    (1, 1500, 48, 16, 64, [64], PAIRS, False, False),
    (1, 3000, 9, 3, 80, [20, 28, 32], HALVES, True, True),
    (2, 1500, 40, 40, 128, [2, 2, 2, 2, 2, 2, 2, 98], PAIRS, True, True),
]


@pytest.mark.parametrize("B,L,Hq,Hk,D,widths,style,norm,affine", CASES)
@pytest.mark.parametrize("where", ["packed", "in place", "heads first"])
def test_rotary(B, L, Hq, Hk, D, widths, style, norm, affine, where):
    g = gen(B * L + D + Hq)
    own = (L + D) % 2 == 0
    shape = (B, L, len(widths)) if own else (L, len(widths))
    pos = torch.randint(-5000, 20000, shape, generator=g, device=DEV, dtype=torch.int32)
    freq = S.segquant_rotary_frequencies(widths).to(DEV)
    gq, gk = (1 + 0.3 * normal(g, D), 1 + 0.3 * normal(g, D)) if affine else (None, None)
    n, m = Hq * D, Hk * D
    qkv = torch.full((B, L, n + 2 * m + 8), 9.0, device=DEV, dtype=BF)
    qkv[..., :n + m] = normal(g, B, L, n + m) * torch.exp(normal(g, B, L, 1))
    q = qkv[..., :n].unflatten(2, (Hq, D))
    k = qkv[..., n:n + m].unflatten(2, (Hk, D))
    want = [rotary_ref(t, pos, freq, widths, style, gamma, 1e-6, norm)
            for t, gamma in ((q, gq), (k, gk))]
    outs = {}
    if where == "in place":
        outs = dict(q_out=q, k_out=k)
    elif where == "heads first":
        outs = dict(q_out=torch.empty(B, Hq, L, D, device=DEV, dtype=BF).transpose(1, 2),
                    k_out=torch.empty(B, Hk, L, D, device=DEV, dtype=BF).transpose(1, 2))
    before = qkv.clone()
    got = S.segquant_qk_rotary(q, k, pos, freq, widths, style, gq, gk, 1e-6, norm, **outs)
    for x, (ref, tol) in zip(got, want):
        close(x, ref, tol)
    if where == "in place":
        assert (qkv[..., n + m:] == 9.0).all()
    else:
        assert torch.equal(qkv, before)
        alone = S.segquant_qk_rotary(q, None, pos, freq, widths, style, gq, None, 1e-6, norm)
        assert alone[1] is None and torch.equal(alone[0], got[0])


@pytest.mark.parametrize("style", [PAIRS, HALVES])
def test_heads_before_tokens_and_slices_of_samples(style):
    """Inputs with heads first, and samples that are parts of longer ones, in place."""
    g = gen(3)
    B, L, H, D = 2, 20, 6, 64
    pos = torch.arange(L, device=DEV, dtype=torch.int32)[:, None].contiguous()
    freq = S.segquant_rotary_frequencies([64]).to(DEV)
    x = normal(g, B, H, L, D).to(BF)
    q = x.transpose(1, 2)
    ref, tol = rotary_ref(q, pos, freq, [64], style, None, 1e-6, True)
    close(S.segquant_qk_rotary(q, None, pos, freq, [64], style)[0], ref, tol)
    long = torch.full((B, L + 5, 2 * H * D), 3.0, device=DEV, dtype=BF)
    long[:, :L] = normal(g, B, L, 2 * H * D)
    q, k = (long[:, :L, i * H * D:(i + 1) * H * D].unflatten(2, (H, D)) for i in range(2))
    want = [rotary_ref(t, pos, freq, [64], style, None, 1e-6, True) for t in (q, k)]
    S.segquant_qk_rotary(q, k, pos, freq, [64], style, q_out=q, k_out=k)
    close(q, *want[0])
    close(k, *want[1])
    assert (long[:, L:] == 3.0).all()
    shared = normal(g, B, L, 1, D).to(BF).expand(B, L, H, D)  # one head for all, as input only
    ref, tol = rotary_ref(shared, pos, freq, [64], style, None, 1e-6, True)
    close(S.segquant_qk_rotary(shared, None, pos, freq, [64], style)[0], ref, tol)


def test_angles_of_far_positions():
    """The largest int32 positions, against exact arithmetic."""
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    places = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 16777217, -99999989, 3, 0]
    pos = torch.tensor(places, device=DEV, dtype=torch.int32)[:, None].contiguous()
    freq = S.segquant_rotary_frequencies([64], 10000.0)
    freq[1] = 3.0  # more than a radian a step
    x = torch.zeros(1, len(places), 1, 64, device=DEV)
    x[..., ::2] = 1.0  # out = (cos, sin)
    out = S.segquant_qk_rotary(x.to(BF), None, pos, freq.to(DEV), [64], PAIRS, norm=False)[0]
    for l, p in enumerate(places):
        for i in range(32):
            u = float(Fraction(p) * Fraction(float(freq[i])) % two_pi)
            for got, want in zip(out[0, l, 0, 2 * i:2 * i + 2].tolist(), (math.cos(u), math.sin(u))):
                assert abs(got - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -20, (p, i)


def test_a_nan_stays_in_its_head():
    g = gen(9)
    q = normal(g, 1, 10, 8, 64).to(BF)
    pos = torch.arange(10, device=DEV, dtype=torch.int32)[:, None].contiguous()
    freq = S.segquant_rotary_frequencies([64]).to(DEV)
    clean = S.segquant_qk_rotary(q, None, pos, freq, [64])[0]
    bad = q.clone()
    bad[0, 4, 2, 7] = float("nan")
    out = S.segquant_qk_rotary(bad, None, pos, freq, [64])[0]
    hit = torch.zeros(1, 10, 8, dtype=torch.bool, device=DEV)
    hit[0, 4, 2] = True
    assert out[hit].isnan().all() and torch.equal(out[~hit], clean[~hit])


def test_no_tokens_other_stream_and_graph():
    g = gen(4)
    freq = S.segquant_rotary_frequencies([16, 48]).to(DEV)
    none = torch.zeros(1, 0, 4, 64, device=DEV, dtype=BF)
    pos = torch.zeros(0, 2, device=DEV, dtype=torch.int32)
    assert S.segquant_qk_rotary(none, none, pos, freq, [16, 48])[0].shape == none.shape
    q, k = normal(g, 2, 100, 4, 64).to(BF), normal(g, 2, 100, 2, 64).to(BF)
    pos = torch.randint(0, 99, (100, 2), generator=g, device=DEV, dtype=torch.int32)
    want = S.segquant_qk_rotary(q, k, pos, freq, [16, 48])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = S.segquant_qk_rotary(q, k, pos, freq, [16, 48])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    outs = [torch.empty_like(q), torch.empty_like(k)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.segquant_qk_rotary(q, k, pos, freq, [16, 48], q_out=outs[0], k_out=outs[1])
    for _ in range(3):  # another batch, other positions
        q.copy_(normal(g, 2, 100, 4, 64))
        pos.copy_(torch.randint(0, 99, (100, 2), generator=g, device=DEV, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = S.segquant_qk_rotary(q, k, pos, freq, [16, 48])
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_the_chain_of_a_block():
    """Residual and norm to MXFP4, the QKV product, norm and rotary of q and k in
    place: each step is what the step before stored, and v is left alone."""
    g = gen(8)
    M, K, H, D = 150, 640, 5, 64
    h, branch = normal(g, M, K).to(BF), normal(g, M, K).to(BF)
    gamma, gq, gk = 1 + 0.2 * normal(g, K), 1 + 0.2 * normal(g, D), 1 + 0.2 * normal(g, D)
    w = S.segquant_quantize_weight_mxfp4(0.05 * normal(g, K, 3 * H * D))
    pos = torch.randint(0, 64, (M, 3), generator=g, device=DEV, dtype=torch.int32)
    freq = S.segquant_rotary_frequencies([16, 24, 24]).to(DEV)
    _, x, stored, mx = S.segquant_rmsnorm_quantize(h, gamma=gamma, branch=branch, x_out=True,
                                                   h_out=True, mx_out=True)
    y = S.segquant_gemm_mxfp4(None, w, 3 * H * D, K=K, xq=mx, M=M)
    xv = S.segquant_unpack_mxfp4(mx, M, K).double()
    wv = S.segquant_unpack_mxfp4(w, 3 * H * D, K).double()
    err = (y.double() - xv @ wv.t()).abs()
    assert (err <= 2.0 ** -8 * (xv @ wv.t()).abs() + 2.0 ** -19 * (xv.abs() @ wv.abs().t())).all()
    t = y.clone().view(1, M, 3, H, D)
    q, k = t[:, :, 0], t[:, :, 1]
    want = [rotary_ref(a, pos, freq, [16, 24, 24], PAIRS, b, 1e-6, True)
            for a, b in ((q, gq), (k, gk))]
    S.segquant_qk_rotary(q, k, pos, freq, [16, 24, 24], PAIRS, gq, gk, q_out=q, k_out=k)
    close(q, *want[0])
    close(k, *want[1])
    assert torch.equal(t[0, :, 2].reshape(M, -1), y[:, 2 * H * D:])


@pytest.mark.parametrize("style", [PAIRS, HALVES])
def test_elements_that_do_not_turn_keep_to_themselves(style):
    """Without the norm, an infinity or a NaN behind the turned part is one element's."""
    g = gen(12)
    q = normal(g, 1, 3, 2, 64).to(BF)
    q[0, 1, 1, 40], q[0, 1, 1, 51] = float("inf"), float("nan")
    pos = torch.randint(0, 99, (3, 1), generator=g, device=DEV, dtype=torch.int32)
    freq = S.segquant_rotary_frequencies([32]).to(DEV)
    out = S.segquant_qk_rotary(q, None, pos, freq, [32], style, norm=False)[0]
    assert torch.equal(out[..., 32:].view(torch.int16), q[..., 32:].view(torch.int16))
    assert not out[..., :32].isnan().any()


def test_tokens_and_heads_far_apart():
    """Strides that pass 32 bits, in elements and in bytes."""
    g = gen(32)
    far, D = (1 << 30) + 64, 64
    freq = S.segquant_rotary_frequencies([64]).to(DEV)
    for shape, dims in (((1, 3, 2, D), (0, 1, 2)), ((1, 2, 3, D), (0, 2, 1)), ((3, 1, 2, D), (1, 0, 2))):
        big = torch.empty(3 * far, device=DEV, dtype=BF).view(1, 3, far)[..., :2 * D]
        q = big.unflatten(2, (2, D)).permute(*dims, 3)
        assert q.shape == shape
        q.copy_(normal(g, *shape))
        pos = torch.randint(0, 99, (shape[1], 1), generator=g, device=DEV, dtype=torch.int32)
        want = S.segquant_qk_rotary(q.contiguous(), None, pos, freq, [64])[0]
        S.segquant_qk_rotary(q, None, pos, freq, [64], q_out=q)
        assert torch.equal(q, want)
        del big, q
