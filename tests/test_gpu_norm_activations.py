"""The activations of segquant_groupnorm_quantize by themselves.  One pixel in
groups of one channel has variance 0, so x = act(beta) to the bit.

An activation within 2^-17 of the true value v, relative, rounds to a bf16
between those of v (1 - 2^-17) and v (1 + 2^-17): roundings are monotone, and
no other error is in x.  Results below 2^-125, where the hardware's exp2 may
flush, are held to 2^-125."""
import math

import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def silu(v):
    return v / (1 + torch.exp(-v))


def gelu(v):
    return v / 2 * torch.erfc(-v / math.sqrt(2.0))


ACTS = {"silu": (S.SEGQ_ACT_SILU, silu, 128.0), "gelu": (S.SEGQ_ACT_GELU, gelu, 14.0)}


def through_the_norm(t, kind):
    """bf16 act(t) for fp32 t of up to 2^20 elements."""
    z = torch.full((1, 1, t.numel()), 3.0, device=DEV, dtype=BF)
    return S.segquant_groupnorm_quantize(z, t.numel(), 1e-5, None, t, act_kind=kind,
                                         x_out=True)[1].flatten()


def check(t, name):
    kind, f, _ = ACTS[name]
    x = through_the_norm(t, kind).double()
    v = f(t.double())
    step = 2.0 ** -17 * v.abs()
    lo, hi = ((v - step).float().to(BF).double(), (v + step).float().to(BF).double())
    ok = ((x >= lo) & (x <= hi)) | ((v.abs() < 2.0 ** -125) & (x.abs() <= 2.0 ** -125))
    assert ok.all(), (int((~ok).sum()), t[~ok][:5].tolist(), x[~ok][:5].tolist(),
                      v[~ok][:5].tolist())


@pytest.mark.parametrize("name", ACTS)
def test_every_finite_bf16_value(name):
    t = (torch.arange(65536, device=DEV, dtype=torch.int32) << 16).view(torch.float32)
    check(t[t.isfinite()].contiguous(), name)


@pytest.mark.parametrize("name", ACTS)
def test_fp32_values(name):
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    top = ACTS[name][2]
    for scale in (top, top / 8, 1.0):
        check((torch.rand(1 << 20, generator=g, device=DEV) * 2 - 1) * scale, name)


@pytest.mark.parametrize("name", ACTS)
def test_nan_and_infinity(name):
    t = torch.tensor([float("nan"), float("inf")] + [0.5] * 6, device=DEV)
    x = through_the_norm(t, ACTS[name][0])
    assert x[0].isnan() and x[1] == math.inf and x[2:].isfinite().all()
