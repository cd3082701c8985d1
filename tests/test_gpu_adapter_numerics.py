"""segquant_adapter_add on values that show how t = alpha (x a^T) is carried
between its two products, in each of the kernel's forms."""
import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
INF = float("inf")

# rows per request, K, stored rank: one launch, two launches, ranks above 64
FORMS = [([3, 14], 64, r) for r in (16, 32, 48, 64)] + [
    ([70, 40], 4160, r) for r in (16, 32, 48, 64)] + [([40, 25], 64, 80), ([5, 4], 64, 128)]


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def int32(*v):
    return torch.tensor(v, device=DEV, dtype=torch.int32)


def call(x, a, b, lens, ids=None, **kw):
    off = torch.tensor([0] + list(lens), device=DEV).cumsum(0).to(torch.int32)
    ids = int32(*(ids if ids is not None else [0] * len(lens)))
    return S.segquant_adapter_add(x, a, b, ids, off, **kw)


def test_the_forms_take_the_launches_they_stand_for():
    for lens, K, rank in FORMS:
        nb = S.segquant_adapter_workspace_bytes(sum(lens), 80, K, len(lens), rank)
        assert (nb == 0) == (K == 64 and rank <= 64)


@pytest.mark.parametrize("lens,K,rank", FORMS)
def test_infinite_factors_give_the_formula_s_infinities(lens, K, rank):
    """t of one to twenty-four significant bits, of either sign, zero and infinite,
    against infinite and finite b: y is infinite, NaN and finite where the formula is."""
    M, N = sum(lens), 80
    g = gen(rank + K)
    x = torch.zeros(M, K, device=DEV, dtype=BF)
    x[:, :3] = torch.randn(M, 3, generator=g, device=DEV)
    x[0, :3] = torch.tensor([1.0, 0.0, 0.0])      # t is a power of two
    x[1, :3] = torch.tensor([-1.5, 0.0, 0.0])
    x[2, :3] = torch.tensor([0.0, 0.0, 0.0])      # t = 0: NaN against infinity
    x[3, :3] = torch.tensor([INF, 0.0, 0.0])
    x[4, :3] = torch.tensor([2.0 ** -50, 0.0, 0.0])
    x[5, :3] = torch.tensor([-2.0 ** 60, 0.0, 0.0])
    a = torch.zeros(1, rank, K, device=DEV, dtype=BF)
    a[0, :, 0] = 2.0 ** torch.randint(-50, 3, (rank,), generator=g, device=DEV)
    a[0, ::2, 0] *= -1
    a[0, ::3, 1:3] = torch.randn(-(-rank // 3), 2, generator=g, device=DEV).to(BF)
    b = torch.randn(1, N, rank, generator=g, device=DEV).to(BF)
    for n in range(64):  # one infinite factor a column, then two, then none
        b[0, n, n % rank] = INF if n % 3 else -INF
        if n >= 48:
            b[0, n, (n + 5) % rank] = INF
    b[0, 70, rank - 1] = float("nan")
    b[0, :, rank - 2] = INF                        # past the second adapter's rank
    used = rank - 2
    base = torch.randn(M, N, generator=g, device=DEV).to(BF)
    y = call(x, a, b, lens, base=base, rank=int32(used)).double()
    t = x[:, :3].double() @ a[0, :used, :3].double().t().contiguous()
    t[3] = INF * a[0, :used, 0].double() + 0.0 * a[0, :used, 1]
    ref = base.double() + (t[:, None] * b[0, :, :used].double()).sum(-1)
    assert ref.isinf().sum() > M * 20 and ref.isnan().any() and ref.isfinite().any()
    assert torch.equal(y.isnan(), ref.isnan())
    assert torch.equal(y.isinf(), ref.isinf())
    assert torch.equal(y[ref.isinf()], ref[ref.isinf()])


@pytest.mark.parametrize("lens,K,rank", FORMS)
def test_t_keeps_its_24_bits(lens, K, rank):
    """Every y is one product t b and a base that cancels its upper bits, so
    what t loses shows.  t = x0 a0 + x1 a1 in fp32 is off by 2^-24 of |x0 a0| + |x1
    a1| (a sum, its parts exact), and so is its product with b; the sum of t's
    parts against b, and the base, by at most 8 2^-24 of |t b| + |base| (at most
    four terms that are not 0, alignment inside an instruction); y rounds at
    2^-8."""
    M, N = sum(lens), 3 * 80
    g = gen(rank * K + 1)
    x = torch.zeros(M, K, device=DEV, dtype=BF)
    x[:, [1, 40]] = torch.randn(M, 2, generator=g, device=DEV).to(BF)
    a = torch.zeros(1, rank, K, device=DEV, dtype=BF)
    a[:, :, [1, 40]] = torch.randn(1, rank, 2, generator=g, device=DEV).to(BF)
    b = torch.zeros(1, N, rank, device=DEV, dtype=BF)
    n = torch.arange(N, device=DEV)
    b[0, n, n % rank] = torch.randn(N, generator=g, device=DEV).to(BF)
    parts = x[:, None, [1, 40]].double() * a[:, :, [1, 40]].double()  # [M][rank][2]
    pick = b[0, n, n % rank].double()
    tb = parts.sum(-1)[:, n % rank] * pick
    U = parts.abs().sum(-1)[:, n % rank] * pick.abs()
    base = (-tb).to(BF)
    ref = base.double() + tb
    err = (call(x, a, b, lens, base=base).double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -24 * (U + 8 * (tb.abs() + base.double().abs()))
    assert (err <= tol).all(), float((err / tol).max())
