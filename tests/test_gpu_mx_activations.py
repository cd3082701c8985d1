"""SiLU and GELU in front of MXFP4 quantisation: every bf16 value, infinities, NaN.

act(z) may be off by 2^-17 of its value (below 2^-125 by that much at most), so the
bf16 value that is quantised lies between the roundings of the two ends, and its
4-bit value, by a block scale that one of the ends gives, between theirs: beside a
border the neighbour, and equal elsewhere."""
import math

import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV
from test_gpu_mxfp4 import act_ref, mx_ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ACTS = {"silu": S.SEGQ_ACT_SILU, "gelu": S.SEGQ_ACT_GELU}
ROWS = [[0, 1, 2, 3, 16, 17, 18, 19], [4, 5, 6, 7, 20, 21, 22, 23], [8, 9, 10, 11, 24, 25, 26, 27],
        [12, 13, 14, 15, 28, 29, 30, 31]]


def every_value(rows, K):
    """Finite bf16 values, neighbours in blocks, the infinities' and NaNs' places zeros."""
    bits = torch.arange(65536, device=DEV, dtype=torch.int32).view(32, K)[rows]
    bits = torch.where((bits & 0x7f80) == 0x7f80, torch.zeros_like(bits), bits)
    return (bits << 16).view(torch.float32).to(BF)


def scaled(x, exponent):
    """x as 4-bit values by the given exponents of its blocks, as mx_ref by its own."""
    unit = torch.exp2(exponent.double())
    block = x.unflatten(1, (-1, 32)) / unit
    lead = torch.full_like(block[..., :1], 4.0)  # fixes the scale of mx_ref at 1
    out = [mx_ref(torch.cat([block[:, :, i:i + 16], lead.expand(-1, -1, 16)], 2).flatten(1))
           .unflatten(1, (-1, 32))[..., :16] for i in (0, 16)]
    return (torch.cat(out, 2) * unit).flatten(1)


def exponents(x):
    top = x.unflatten(1, (-1, 32)).abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top.clamp(min=2.0 ** -300)).exponent - 3, -127)
    return e.clamp(min=-127)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("rows,power", list(zip(ROWS, (100.0, 0.0, 0.0, 0.0))))
def test_every_value(rows, power, act):
    K = 2048
    z = every_value(rows, K)
    got = S.segquant_unpack_mxfp4(S.segquant_quantize_mxfp4(z, ACTS[act]), 8, K)
    # quantised inside the product, read off a weight with one power of two in each column
    assert S.segquant_gemm_mxfp4_workspace_bytes(8, K, K) == 0
    w = S.segquant_quantize_weight_mxfp4(2.0 ** power * torch.eye(K, device=DEV))
    y = S.segquant_gemm_mxfp4(z, w, K, act_kind=ACTS[act])
    assert torch.equal(y.double(), got.double() * 2.0 ** power)

    a = act_ref(z.double().cpu(), act)
    slack = 2.0 ** -17 * a.abs().clamp(min=2.0 ** -125)
    ends = [(a - slack).to(BF).double(), (a + slack).to(BF).double()]
    got = got.cpu().double()
    fits = torch.zeros(8, K // 32, dtype=torch.bool)
    for e in map(exponents, ends):
        lo, hi = (scaled(x, e) for x in ends)
        fits |= ((lo <= got) & (got <= hi)).unflatten(1, (-1, 32)).all(2)
    # blocks below 2^-118 take their scale from values below 2^-125
    low = a.abs().unflatten(1, (-1, 32)).amax(2) < 2.0 ** -118
    assert (fits | low).all(), (fits | low).logical_not().nonzero().tolist()
    assert float((got == mx_ref(a.to(BF))).double().mean()) > 1 - 2.0 ** -9


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M", [3, 16, 40, 300])
def test_infinities_and_nan_make_their_rows_nan(act, M):
    """As the formulas have it: an infinity times 0 at one end, an infinity at the other."""
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    K, N = 2048, 80
    z = torch.randn(M, K, generator=g, device=DEV).to(BF)
    w = S.segquant_quantize_weight_mxfp4(torch.randn(K, N, generator=g, device=DEV))
    clean = S.segquant_gemm_mxfp4(z, w, N, act_kind=ACTS[act])
    bad = z.clone()
    bad[0, 100], bad[1, 2047], bad[2, 64] = float("inf"), -float("inf"), float("nan")
    y = S.segquant_gemm_mxfp4(bad, w, N, act_kind=ACTS[act])
    assert y[:3].isnan().all() and torch.equal(y[3:], clean[3:])
    values = S.segquant_unpack_mxfp4(S.segquant_quantize_mxfp4(bad, ACTS[act]), M, K)
    want = torch.zeros(M, K, dtype=torch.bool, device=DEV)
    want[0, 96:128] = want[1, 2016:] = want[2, 64:96] = True
    assert torch.equal(values.isnan(), want)
    assert math.isnan(act_ref(torch.tensor(-math.inf, dtype=torch.float64), act))


@pytest.mark.parametrize("act", list(ACTS))
def test_far_below_zero(act):
    """Values whose e^-z overflows, beside ordinary ones and on their own."""
    z = torch.zeros(4, 64, device=DEV)
    z[0], z[1], z[2, ::2], z[3] = -70.0, -3e38, -95.0, -87.5
    z[0, 0] = z[1, 5] = 2.0
    z = z.to(BF)
    x = S.segquant_unpack_mxfp4(S.segquant_quantize_mxfp4(z, ACTS[act]), 4, 64).cpu().double()
    assert torch.equal(x, mx_ref(act_ref(z.double().cpu().clamp(min=-200), act).to(BF)))
