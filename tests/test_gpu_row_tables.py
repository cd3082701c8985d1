"""Row offsets that decrease or leave the batch, in segquant_adanorm_quantize
and segquant_adapter_add.  Rows whose request no order of the table puts in doubt
get theirs.  The others are left as they are or hold what the header leaves
open: the norm's result with one of the call's own requests, and any sum of the
call's own factors.  What stands around the arrays that a wrong request number
would reach is NaN."""
import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAN = float("nan")
LEFT = 9.0
TABLES = [[0, 100, 50, 120], [120, 0, 0, 0], [-5, 40, 4000, 70], [7] * 4, [130, 90, 60, 10],
          [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31], [20, 60, 60, 500], [-9, -3, 5, 77],
          [i * 37 % 131 for i in range(80)], [2 * (i % 66) for i in range(131)]]


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def guarded(data, before=3, fill=NAN):
    """data inside a buffer with rows of `fill` before and behind it."""
    buf = torch.full((len(data) + 2 * before, *data.shape[1:]), fill, device=DEV, dtype=data.dtype)
    buf[before:before + len(data)] = data
    return buf[before:before + len(data)]


def certain(off, M):
    """Request of each row that every reading of the table agrees on, -1 for
    rows that none holds, None for the others."""
    out = []
    for m in range(M):
        past = [o <= m for o in off]
        n = sum(past)
        if past != sorted(past, reverse=True):
            out.append(None)
        else:
            out.append(n - 1 if 0 < n < len(off) else -1)
    return out


def check(y, candidates, off, of_one_request=True):
    """y [M][N]; candidates [R][M][N] with their tolerance."""
    ref, tol = candidates
    left = (y == LEFT).all(1)
    ok = ((y.double() - ref).abs() <= tol)  # [R][M][N]
    fine = ok.any(0).all(1) | left if of_one_request else y.isfinite().all(1)
    assert fine.all(), [(int(m), y[m, :4].tolist()) for m in (~fine).nonzero()[:3, 0]]
    for m, r in enumerate(certain(off, len(y))):
        if r is not None and r >= 0:
            assert ok[r, m].all(), (m, r)
        elif r == -1:
            assert left[m], m


@pytest.mark.parametrize("off", TABLES, ids=str)
@pytest.mark.parametrize("K", [128, 1000])
def test_adanorm(off, K):
    g = gen(K)
    M, R = 130, len(off) - 1
    ld = -(-K // 8) * 8
    h, branch = normal(g, M, ld).to(BF)[:, :K], normal(g, M, ld).to(BF)[:, :K]
    mods = guarded(normal(g, R, 3 * ld).to(BF))
    shift, scale, gate = (mods[:, i * ld:i * ld + K] for i in range(3))
    out = guarded(torch.full((M, 2 * ld), LEFT, device=DEV, dtype=BF), fill=LEFT)
    x, h2 = out[:, :K], out[:, ld:ld + K]
    S.segquant_adanorm_quantize(h, scale=scale, shift=shift, gate=gate, branch=branch, x_out=x,
                                h_out=h2, row_offset=torch.tensor(off, device=DEV,
                                                                  dtype=torch.int32))
    hd = h.double() + gate.double()[:, None] * branch.double()  # [R][M][K]
    check(h2, (hd, 2.0 ** -8 * hd.abs() * (1 + 2.0 ** -14)), off)
    t = hd.to(BF).double()
    t = t - t.mean(2, keepdim=True)
    t = t / torch.sqrt(t.square().mean(2, keepdim=True) + 1e-6)
    t = t * (1 + scale.double()[:, None]) + shift.double()[:, None]
    # two bf16 steps: x's rounding, and h' one step aside where fp32 rounds it
    # the other way (|t| moves by no more than that of its row's largest h')
    check(x, (t, 2.0 ** -7 * (t.abs() + t.abs().amax(2, keepdim=True))), off)
    rows = torch.cat([buf for buf in (out._base[:3], out._base[-3:])])
    assert (rows == LEFT).all() and (x == LEFT).all(1).equal((h2 == LEFT).all(1))


@pytest.mark.parametrize("off", TABLES, ids=str)
@pytest.mark.parametrize("rank", [16, 128])
def test_adapters(off, rank):
    g = gen(rank)
    M, K, N, R, n = 130, 64, 32, len(off) - 1, 3
    x = guarded(normal(g, M, K).to(BF))
    a = guarded((normal(g, n, rank, K) / 8).to(BF))
    b = guarded((normal(g, n, N, rank) / 4).to(BF))
    base = guarded(normal(g, M, N).to(BF))
    ids = torch.arange(R, device=DEV, dtype=torch.int32) % 2
    a[2:], b[2:] = NAN, NAN  # the third adapter belongs to no request
    ids = guarded(ids, fill=2)
    y = guarded(torch.full((M, N), LEFT, device=DEV, dtype=BF), fill=LEFT)
    S.segquant_adapter_add(x, a, b, ids, torch.tensor(off, device=DEV, dtype=torch.int32),
                           base=base, out=y)
    t = x.double() @ a[:2].double().transpose(1, 2).contiguous()
    bt = b[:2].double().transpose(1, 2).contiguous()
    ref = (base.double() + t @ bt)[ids.long()]
    size = (base.double().abs() + (x.double().abs() @ a[:2].double().abs().transpose(1, 2)
                                   .contiguous()) @ bt.abs())[ids.long()]
    # bf16 rounding, and fp32 sums of 64 and 3 rank terms
    check(y, (ref, 2.0 ** -8 * ref.abs() + (64 + 3 * rank + 2) * 2.0 ** -24 * size), off,
          of_one_request=False)
    assert (y._base[:3] == LEFT).all() and (y._base[-3:] == LEFT).all()
