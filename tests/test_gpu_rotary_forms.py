"""Every form of the rotary kernel: the lanes of a head (1 to 32), the heads of a wave
(one, two and three times 64 over those), pairs and halves, whole heads and heads with
lanes to spare, one row of the grid and more; against the formula in fp64, with
the tolerance of test_gpu_rotary.py: 2^-8 |out| + 2^-18 (|a| + |b|)."""
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


def check(got, x, pos, freq, axis, style, gamma, norm):
    """x [B][L][H][D] before the call, pos [L][axes] or [B][L][axes]."""
    t = x.double()
    if norm:
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)
        if gamma is not None:
            t = t * gamma.double()
    u = (pos.double()[..., axis] * freq)[..., None, :]
    c, s, R = torch.cos(u), torch.sin(u), 2 * len(axis)
    a, b = ((slice(0, R, 2), slice(1, R, 2)) if style == PAIRS
            else (slice(0, R // 2), slice(R // 2, R)))
    out, size = t.clone(), t.abs()
    out[..., a] = t[..., a] * c - t[..., b] * s
    out[..., b] = t[..., b] * c + t[..., a] * s
    size[..., a] = size[..., b] = t[..., a].abs() + t[..., b].abs()
    err, tol = (got.double() - out).abs(), 2.0 ** -8 * out.abs() + 2.0 ** -18 * size + 2.0 ** -133
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))


def run(g, B, L, Hq, Hk, D, widths, style, norm=True, in_place=False):
    R = sum(widths)
    axis = torch.repeat_interleave(torch.arange(len(widths)), torch.tensor(widths) // 2).to(DEV)
    pos = torch.randint(-5000, 20000, (L, len(widths)), generator=g, device=DEV, dtype=torch.int32)
    freq = S.segquant_rotary_frequencies(widths).to(DEV)
    gq, gk = ((1 + 0.3 * normal(g, D), 1 + 0.3 * normal(g, D)) if norm else (None, None))
    n, m = Hq * D, Hk * D
    qkv = torch.full((B, L, n + 2 * m), 9.0, device=DEV, dtype=BF)
    qkv[..., :n + m] = normal(g, B, L, n + m) * torch.exp(normal(g, B, L, 1))
    q = qkv[..., :n].unflatten(2, (Hq, D))
    k = qkv[..., n:n + m].unflatten(2, (Hk, D)) if Hk else None
    before = qkv.clone()
    outs = dict(q_out=q, k_out=k) if in_place else {}
    got = S.segquant_qk_rotary(q, k, pos, freq, widths, style, gq, gk if Hk else None, 1e-6, norm,
                               **outs)
    check(got[0], before[..., :n].unflatten(2, (Hq, D)), pos, freq, axis, style, gq, norm)
    if Hk:
        check(got[1], before[..., n:n + m].unflatten(2, (Hk, D)), pos, freq, axis, style, gk, norm)
    assert torch.equal(qkv[..., n + m:] if in_place else qkv, before[..., n + m:] if in_place else before)


# head widths that fill their lanes, and that do not (with the part that turns)
@pytest.mark.parametrize("lanes,D,R", [(1, 16, 16), (1, 8, 0), (2, 32, 32), (2, 24, 16), (4, 64, 64),
                                       (4, 40, 32), (4, 64, 48), (8, 128, 128), (8, 72, 48),
                                       (16, 256, 256), (16, 200, 64), (32, 512, 512), (32, 264, 256)])
@pytest.mark.parametrize("times", [2, 3])
@pytest.mark.parametrize("style", [PAIRS, HALVES])
def test_several_heads_a_wave(lanes, D, R, times, style):
    per = 64 // lanes
    Hq = times * per - (1 if per * times > 2 else 0)  # the last wave's lanes not all used
    Hk = max(1, per // 2)
    g = gen(lanes * times + D)
    run(g, 1, 2048 // times + 77, Hq, Hk, D, [R], style, in_place=times == 2)


@pytest.mark.parametrize("B,L,Hq,Hk,D,widths,style", [
    (1, 4429, 24, 24, 64, [16, 24, 24], PAIRS), (1, 2100, 12, 12, 128, [44, 42, 42], HALVES),
    (2, 1100, 24, 8, 64, [64], HALVES), (1, 2100, 48, 24, 64, [32, 32], PAIRS),
    (3, 700, 9, 27, 128, [128], HALVES), (1, 1500, 30, 6, 80, [20, 28, 32], PAIRS)])
@pytest.mark.parametrize("norm", [True, False])
def test_sizes_of_models(B, L, Hq, Hk, D, widths, style, norm):
    run(gen(B * L + D), B, L, Hq, Hk, D, widths, style, norm, in_place=True)


@pytest.mark.parametrize("style", [PAIRS, HALVES])
def test_more_workgroups_than_a_row_of_the_grid(style):
    """More than 2^22 waves: tokens of one short head each."""
    run(gen(3), 1, (1 << 22) + 1029, 1, 0, 16, [16], style)


@pytest.mark.parametrize("style", [PAIRS, HALVES])
@pytest.mark.parametrize("B,L,H,D,tokens", [(2, 10, 4, 64, 13), (3, 700, 12, 64, 701)])
def test_q_k_and_v_of_each_head_side_by_side(B, L, H, D, tokens, style):
    """In place in a part of [B][tokens][H][3][D]: v and the other tokens are left alone."""
    g = gen(L)
    whole = normal(g, B, tokens, H, 3, D).to(BF)
    before = whole.clone()
    pos = torch.randint(0, 999, (L, 1), generator=g, device=DEV, dtype=torch.int32)
    freq = S.segquant_rotary_frequencies([D]).to(DEV)
    q, k = whole[:, :L, :, 0], whole[:, :L, :, 1]
    S.segquant_qk_rotary(q, k, pos, freq, [D], style, q_out=q, k_out=k)
    axis = torch.zeros(D // 2, dtype=torch.long, device=DEV)
    check(q, before[:, :L, :, 0], pos, freq, axis, style, None, True)
    check(k, before[:, :L, :, 1], pos, freq, axis, style, None, True)
    assert torch.equal(whole[..., 2, :], before[..., 2, :])
    assert torch.equal(whole[:, L:], before[:, L:])
