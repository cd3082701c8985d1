"""segquant_adapter_add against its formula in fp64, and the run of norm,
quantised layer and adapters together.

Tolerance of y, element by element, with the sums of magnitudes T = |x||a| and
U = sum |alpha| T |b|, V = sum |t||b|: bf16 rounding 2^-8 |y|; the sum over K
in fp32, at most K/32 instructions and 32 terms inside one, (K/32 + 64) 2^-24
U; t in two bf16 parts, the upper half truncated (rest below 2^-7 |t|) and the
rest rounded at 2^-8 of itself, 2^-15 V; the sum over the rank and the base,
(rank/16 + 36) 2^-24 (V + |base|)."""
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


def offsets(lens, before=0):
    return torch.tensor([before] + list(lens), device=DEV).cumsum(0).to(torch.int32)


class Case:
    def __init__(self, lens, K, N, nseg, rank, ids, ranks=None, tail=0, before=0, seed=0):
        g = gen(seed + K + N + rank)
        self.lens, self.nseg, self.ids, self.before = list(lens), list(nseg), list(ids), before
        M = sum(lens) + before + tail
        n = max(max(ids) + 1, 1)
        S_ = len(nseg)
        self.x = (normal(g, M, K) * torch.exp(0.5 * normal(g, K))).to(BF)
        self.a = (normal(g, n, S_ * rank, K) / K ** 0.5).to(BF)
        self.b = (normal(g, n, N, rank) / rank ** 0.5).to(BF)
        self.alpha = 0.5 + torch.rand(n, generator=g, device=DEV)
        self.base = normal(g, M, N).to(BF)
        self.ranks = list(ranks) if ranks else [rank] * n
        self.rank_of = torch.tensor(self.ranks, device=DEV, dtype=torch.int32)
        self.off = offsets(lens, before)
        self.adapter = torch.tensor(ids, device=DEV, dtype=torch.int32)
        for i, r in enumerate(self.ranks):  # what is stored past a rank must not matter
            if r < rank:
                self.a.view(n, S_, rank, K)[i, :, r:] = float("nan")
                self.b[i, :, r:] = float("inf")

    def run(self, **kw):
        args = dict(base=self.base, alpha=self.alpha, rank=self.rank_of, nseg=self.nseg)
        args.update(kw)
        return S.segquant_adapter_add(self.x, self.a, self.b, self.adapter, self.off, **args)

    def check(self, y, before=None, base=True):
        """y against the formula; rows of no request against `before`."""
        K, rank = self.x.shape[1], self.b.shape[2]
        seen = torch.zeros(len(y), dtype=torch.bool, device=DEV)
        at = self.before
        for length, i in zip(self.lens, self.ids):
            rows = slice(at, at + length)
            at += length
            seen[rows] = True
            b0 = self.base[rows].double() if base else torch.zeros_like(y[rows]).double()
            if not 0 <= i < len(self.a):
                assert torch.equal(y[rows], self.base[rows] if base else torch.zeros_like(y[rows]))
                continue
            r, n0 = self.ranks[i], 0
            x, al = self.x[rows].double(), float(self.alpha[i])
            for j, w in enumerate(self.nseg):
                a = self.a[i, j * rank:j * rank + r].double().t().contiguous()
                b = self.b[i, n0:n0 + w, :r].double().t().contiguous()
                t, T = al * (x @ a), abs(al) * (x.abs() @ a.abs())
                ref = b0[:, n0:n0 + w] + t @ b
                U, V = T @ b.abs(), t.abs() @ b.abs()
                tol = (2.0 ** -8 * ref.abs() + (K / 32 + 64) * 2.0 ** -24 * U + 2.0 ** -15 * V +
                       (rank / 16 + 36) * 2.0 ** -24 * (V + b0[:, n0:n0 + w].abs()))
                err = (y[rows, n0:n0 + w].double() - ref).abs()
                assert (err <= tol).all(), (i, j, float((err - tol).max()))
                n0 += w
        if before is not None:
            assert torch.equal(y[~seen], before[~seen])


CASES = [
    # rows per request, K, N, N-segments, stored rank, adapter of each request, ranks
    ([1], 64, 16, [16], 16, [0], None),
    ([1, 1], 1536, 9216, [1536] * 6, 16, [1, 0], [16, 5]),
    ([1] * 70, 512, 400, [64, 336], 32, [i % 7 - 1 for i in range(70)], [32, 17, 1, 0, 16, 31]),
    ([5, 0, 17, 1, 0, 64, 33], 256, 96, [96], 16, [0, 1, 2, 2, 0, -1, 1], [16, 8, 3]),
    ([4096, 333], 1536, 1536, [1536], 16, [0, 1], None),
    ([100, 300, 15], 192, 272, [16, 80, 176], 48, [0, 0, 1], [48, 33]),
    ([63, 65, 129], 6144, 208, [208], 64, [0, 2, 1], None),
    ([31, 2], 320, 64, [64], 256, [1, 0], [256, 200]),
    ([16, 16, 16], 64, 2048, [16] * 128, 16, [0, 1, 0], None),
    ([2000], 64, 48, [48], 16, [-1], None),
    ([i % 5 for i in range(5000)], 64, 32, [32], 16, [i % 3 - 1 for i in range(5000)], None),
    ([0] * 100 + [40] + [0] * 29 + [1], 64, 32, [32], 16, [i % 2 for i in range(131)], [3, 16]),
    ([1] * 60 + [0, 0, 17, 1, 35] + [1] * 60, 64, 32, [32], 16, [i % 3 - 1 for i in range(125)], None),
    # two launches
    ([3] * 150, 4160, 96, [96], 48, [i % 4 - 1 for i in range(150)], None),
    ([1] * 5, 8192, 160, [80, 80], 16, [0, 1, -1, 2, 0], [16, 7, 16]),
    ([1, 0, 3, 16, 2], 4160, 336, [336], 32, [0, 2, 1, 0, -1], [32, 30, 5]),
    ([90, 200, 17], 4224, 208, [208], 16, [1, 0, -1], [11, 16]),
    ([500, 33], 4096 + 64, 400, [64, 336], 48, [1, 0], [48, 20]),
    ([5, 40], 128, 320, [16] * 20, 64, [1, 0], None),
    ([7] * 9, 64, 32, [32], 128, [i % 2 for i in range(9)], [128, 1]),
    # whole tiles of rows and columns, several blocks of columns to a wave
    *[([4000, 33, 64], 1536, 1536, [1536], r, [0, 1, -1], [r, r - 9]) for r in (16, 32, 48, 64)],
    *[([8000, 70, 128], 4160, 1600, [64, 1536], r, [0, 1, -1], [r - 7, r]) for r in (16, 32, 48, 64)],
]


@pytest.mark.parametrize("lens,K,N,nseg,rank,ids,ranks", CASES)
def test_adapter_add(lens, K, N, nseg, rank, ids, ranks):
    c = Case(lens, K, N, nseg, rank, ids, ranks, tail=5, before=3)
    out = torch.full_like(c.base, 7.0)
    c.check(c.run(out=out), torch.full_like(c.base, 7.0))
    again = c.run()  # allocated here: zeros in rows of no request
    c.check(again, torch.zeros_like(again))
    rows = slice(3, 3 + sum(lens))
    assert torch.equal(again[rows], out[rows])
    base = c.base.clone()
    c.check(c.run(base=base, out=base), c.base)  # in place
    c.check(c.run(base=None), torch.zeros_like(again), base=False)


@pytest.mark.parametrize("n_req,length", [(64 * 64 * 64 + 1, 1), (70001, 2), (5000, 40)])
def test_very_many_requests(n_req, length):
    """Three and four steps of the search for a tile's request; the formula for
    all rows with each of the two adapters at a time."""
    K, N, rank = 64, 32, 16
    lens = [i % (length + 1) for i in range(n_req)]
    c = Case([sum(lens)], K, N, [N], rank, [1], None)
    c.off = offsets(lens)
    c.adapter = torch.arange(n_req, device=DEV, dtype=torch.int32) % 5 % 2
    y = c.run()
    row_id = torch.repeat_interleave(c.adapter, torch.tensor(lens, device=DEV))
    for i in (0, 1):
        rows = row_id == i
        one = Case.__new__(Case)
        one.__dict__.update(c.__dict__, x=c.x[rows], base=c.base[rows], lens=[int(rows.sum())],
                            ids=[i])
        one.check(y[rows])


def test_defaults_and_strided_rows():
    c = Case([40, 9], 128, 96, [96], 32, [1, 0])
    M = 49
    c.alpha = torch.ones_like(c.alpha)
    want = c.run(alpha=None, rank=None, nseg=None)
    c.check(want)
    x = torch.full((M, 136), float("nan"), device=DEV, dtype=BF)
    base = torch.full((M, 104), float("nan"), device=DEV, dtype=BF)
    y = torch.full((M, 112), 7.0, device=DEV, dtype=BF)
    x[:, :128], base[:, :96] = c.x, c.base
    c.x = x[:, :128]
    c.run(base=base[:, :96], out=y[:, :96], alpha=None, rank=None, nseg=None)
    assert torch.equal(y[:, :96], want) and (y[:, 96:] == 7.0).all()


@pytest.mark.parametrize("ids", [[5, -7], [2, 1 << 30]])
def test_an_index_outside_the_table_is_no_adapter(ids):
    c = Case([20, 30], 64, 32, [32], 16, [1, 1])
    c.adapter = torch.tensor(ids, device=DEV, dtype=torch.int32)
    c.ids = ids
    c.check(c.run())


def test_infinities_and_nan_stay_in_their_rows():
    c = Case([8, 8], 64, 32, [32], 16, [0, 0])
    c.x[3, 5] = float("inf")
    c.x[9, 0] = float("nan")
    y = c.run()
    clean = torch.ones(16, dtype=torch.bool, device=DEV)
    clean[[3, 9]] = False
    assert torch.isfinite(y[clean]).all() and y[9].isnan().all()
    # +-inf in every t of the row: each product is +-inf or cancels to NaN
    t = c.x[3].double() @ c.a[0].double().t().contiguous()
    ref = c.alpha[0].double() * (t @ c.b[0].double().t().contiguous()) + c.base[3].double()
    assert torch.equal(torch.isnan(y[3]), torch.isnan(ref))
    assert torch.equal(y[3][~torch.isnan(ref)].double(), ref[~torch.isnan(ref)])


@pytest.mark.parametrize("off", [[0, 100, 50, 120], [120, 0, 0, 0], [-5, 40, 4000, 70], [7] * 4])
def test_offsets_out_of_order_stay_in_bounds(off):
    g = gen(3)
    M, K, N = 130, 64, 32
    x = normal(g, M, K).to(BF)
    a, b = normal(g, 2, 16, K).to(BF), normal(g, 2, N, 16).to(BF)
    buf = torch.full((M + 64, N), 9.0, device=DEV, dtype=BF)
    S.segquant_adapter_add(x, a, b, torch.tensor([0, 1, 0], device=DEV, dtype=torch.int32),
                           torch.tensor(off, device=DEV, dtype=torch.int32),
                           out=buf[32:32 + M])
    assert (buf[:32] == 9.0).all() and (buf[32 + M:] == 9.0).all()


def test_workspace_of_the_exact_size_is_kept_to():
    for lens, K, rank in (([1] * 3, 8192, 16), ([700, 20], 5120, 64), ([9], 64, 80)):
        c = Case(lens, K, 64, [64], rank, [0] * len(lens))
        nb = S.segquant_adapter_workspace_bytes(sum(lens), 64, K, len(lens), rank)
        assert nb > 0
        ws = torch.full((nb + 4096,), 77, dtype=torch.uint8, device=DEV)
        c.check(c.run(workspace=ws[:nb]))
        assert (ws[nb:] == 77).all()


def test_rows_beyond_32_bit_offsets():
    M, K, N = 180_000, 12288, 32
    assert M * K > 2 ** 31
    c = Case([8], K, N, [N], 16, [0])
    x = torch.zeros(M, K, device=DEV, dtype=BF)
    for at in (0, 100_000, M - 8):
        x[at:at + 8] = c.x
    off = torch.tensor([0, 150_000, M], device=DEV, dtype=torch.int32)
    ids = torch.tensor([0, 0], device=DEV, dtype=torch.int32)
    base = torch.zeros(M, N, device=DEV, dtype=BF)
    for at in (0, 100_000, M - 8):
        base[at:at + 8] = c.base
    y = S.segquant_adapter_add(x, c.a, c.b, ids, off, base=base, alpha=c.alpha)
    for at in (0, 100_000, M - 8):
        c.check(y[at:at + 8])
    assert (y[8:100_000] == 0).all()


def test_adapters_beyond_32_bit_offsets():
    n, K, rank = 11, 12288, 256
    nseg = [16] * 64
    assert n * len(nseg) * rank * K > 2 ** 31
    c = Case([3, 4], K, 1024, nseg, rank, [0, n - 1])
    c.check(c.run())


def test_on_another_stream_and_in_graphs_that_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn between eager
    calls on new inputs and new request tables."""
    cs = [Case([1] * 20, 4224, 192, [96, 96], 16, [i % 3 for i in range(20)], tail=4),
          Case([100, 200, 40], 4160, 64, [64], 32, [0, 1, -1]),
          Case([70, 30], 256, 64, [64], 32, [0, 1])]
    nb = max(S.segquant_adapter_workspace_bytes(len(c.x), c.b.shape[1], c.x.shape[1],
                                                len(c.ids), c.b.shape[2], c.nseg) for c in cs)
    assert nb > 0
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(c.base) for c in cs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, o in zip(cs, outs):
            c.run(out=o, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in cs]
    for gr, c, o in zip(graphs, cs, outs):
        with torch.cuda.graph(gr):
            c.run(out=o, workspace=ws)
    g = gen(9)
    for i in range(4):
        for c, o in zip(cs, outs):
            c.x.copy_(normal(g, *c.x.shape))
            c.adapter.copy_(c.adapter.roll(1))
            c.ids = c.ids[-1:] + c.ids[:-1]
            o.zero_()
        for gr in graphs:
            gr.replay()
        eager = [c.run() for c in cs]
        torch.cuda.synchronize()
        for c, o, e in zip(cs, outs, eager):
            assert torch.equal(o, e)
            c.check(o)


# ---------------------------------------------------- the run of them ----
def layer_ref(codes, act, wq, ws, kseg):
    """The W8A8 layer on signed codes, fp64."""
    y, at = 0, 0
    act = act.double()
    for i, w in enumerate(kseg):
        q = codes[:, at:at + w].double()
        x = torch.where(q < 0, q * act[1, i], q * act[0, i])
        y = y + (x @ wq[at:at + w].double()) * ws[i].double()
        at += w
    return y


@pytest.mark.parametrize("M,lens,K,N,nseg", [
    (12, [1] * 12, 256, 384, [128] * 3),
    (333, [200, 133], 512, 192, [192]),
])
def test_adanorm_layer_and_adapters(M, lens, K, N, nseg):
    """The conditioning layer's chunks modulate the norm, its codes feed the
    layer, the adapters of each request add to the layer's output in place."""
    g = gen(M)
    off, R = offsets(lens), len(lens)
    h, branch = normal(g, M, K).to(BF), normal(g, M, K).to(BF)
    cond = normal(g, R, 256).to(BF)
    cw, cs = S.segquant_quantize_weight(0.02 * normal(g, 256, 3 * K), nseg=[K] * 3)
    mods = S.segquant_gemm_w8a8_seg(cond, cw, cs, S.segquant_calibrate_amax(cond))
    shift, scale, gate = mods.chunk(3, dim=1)
    args = dict(scale=scale, shift=shift, gate=gate, branch=branch, row_offset=off)
    x = S.segquant_adanorm_quantize(h, x_out=True, **args)[1]
    act = S.segquant_calibrate_amax(x)
    w = 0.05 * normal(g, K, N)
    wp, ws = S.segquant_quantize_weight(w, nseg=nseg, per_column=True)
    codes, x, h2 = S.segquant_adanorm_quantize(h, act_scales=act, x_out=x, h_out=True, **args)
    y0 = S.segquant_gemm_w8a8_seg(None, wp, ws, act, [K], xq=codes)
    ref0 = layer_ref(codes[:, :K], act, S.segquant_unpack_weight(wp, K, N), ws, [K])
    assert ((y0.double() - ref0).abs() <= 8e-3 * ref0.abs() + 1e-3 * ref0.abs().max()).all()
    c = Case(lens, K, N, nseg, 16, [i % 3 - (i == 5) for i in range(R)])
    c.x, c.base = x, y0.clone()
    c.check(c.run(base=y0, out=y0))


def test_groupnorm_layer_on_concatenated_channels():
    g = gen(4)
    B, P, kseg, N = 2, 300, [128, 64], 96
    C = sum(kseg)
    z = torch.cat([normal(g, B, P, 128), 4 * normal(g, B, P, 64)], 2).to(BF)
    args = (z, 8, 1e-5, 1 + 0.1 * normal(g, C), 0.1 * normal(g, C), None, None, S.SEGQ_ACT_SILU)
    x = S.segquant_groupnorm_quantize(*args, x_out=True)[1].reshape(B * P, C)
    act = S.segquant_calibrate_amax(x, kseg)
    wp, ws = S.segquant_quantize_weight(0.05 * normal(g, C, N), kseg, per_column=True)
    codes, _ = S.segquant_groupnorm_quantize(*args, act_scales=act, kseg=kseg)
    y = S.segquant_gemm_w8a8_seg(None, wp, ws, act, kseg, xq=codes)
    # the same kernel on the same codes, quantised from x in a pass of their own
    y2 = S.segquant_gemm_w8a8_seg(None, wp, ws, act, kseg,
                                  xq=S.segquant_quantize_dualscale(x, act, kseg))
    ref = layer_ref(codes, act, S.segquant_unpack_weight(wp, C, N), ws, kseg)
    assert ((y.double() - ref).abs() <= 8e-3 * ref.abs() + 1e-3 * ref.abs().max()).all()
    assert torch.equal(y, y2)
