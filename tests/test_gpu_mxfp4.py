"""The microscaled 4-bit layer (segquant_quantize_mxfp4,
segquant_quantize_weight_mxfp4, segquant_unpack_mxfp4, segquant_gemm_mxfp4)
against the format's definition in fp64.

Quantising is exact but for the one rounding to the 4-bit values, so codes have
to be equal.  Tolerance of the product, with S = sum |x w| of an output: its
rounding to bf16 2^-8 |y|; in fp32, one addition to the running sum per 128
columns, 2^-24 S each, and the matrix core's own sum of an instruction's 128
products, taken to lose no more than 2^-20 of their magnitudes."""
import math

import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ACTS = {"none": S.SEGQ_ACT_NONE, "silu": S.SEGQ_ACT_SILU, "gelu": S.SEGQ_ACT_GELU}
VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def padded(data, ld, fill):
    buf = torch.full((*data.shape[:-1], ld), fill, device=DEV, dtype=data.dtype)
    view = buf[..., :data.shape[-1]]
    view.copy_(data)
    return buf, view


def mx_ref(x):
    """The values that x [R][K] takes, fp64, by distance to every 4-bit value."""
    b = x.detach().cpu().double().unflatten(1, (-1, 32))
    top = b.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top.clamp(min=2.0 ** -300)).exponent - 3, -127)
    scale = torch.exp2(e.clamp(min=-127).double())
    v = b.abs() / scale
    far = (v[..., None] - VALUES).abs()
    best = far.amin(-1, keepdim=True)
    # ties: the even code
    code = torch.arange(8)
    pick = torch.where(far == best, code % 2 * 8 + code, 99).argmin(-1)
    return (VALUES[pick] * torch.sign(b) * scale).flatten(1)


def act_ref(t, act):
    if act == "silu":
        return t / (1 + torch.exp(-t))
    if act == "gelu":
        return t / 2 * torch.erfc(-t / math.sqrt(2.0))
    return t


def edge_values(g, M, K):
    """Blocks of all sizes: normal, all zero, one value, ties, subnormal, the largest."""
    x = normal(g, M, K)
    kind = torch.randint(0, 8, (M, K // 32), generator=g, device=DEV).repeat_interleave(32, 1)
    x = torch.where(kind == 1, torch.zeros_like(x), x)
    ties = torch.randint(-32, 33, (M, K), generator=g, device=DEV) / 4.0
    x = torch.where(kind == 2, ties, x)
    x = torch.where(kind == 3, x * 2.0 ** -130, x)
    x = torch.where(kind == 4, x * 2.0 ** 125, x)
    x = torch.where(kind == 5, x * torch.exp2(8 * normal(g, M, K)), x)
    x = torch.where((kind == 6) & (torch.rand(M, K, generator=g, device=DEV) < 0.97), 0.0, x)
    return x


@pytest.mark.parametrize("M,K", [(1, 64), (2, 1536), (15, 128), (16, 576), (17, 192), (33, 2048),
                                 (300, 640), (4429, 64)])
def test_quantize(M, K):
    g = gen(M + K)
    x = edge_values(g, M, K).clamp(-3e38, 3e38).to(BF)
    _, x = padded(x, K + 8, float("nan"))  # what stands between rows is not read
    n, m = S.segquant_mxfp4_bytes(M, K)
    codes = torch.full((n + 64,), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((m + 64,), 0xAB, dtype=torch.uint8, device=DEV)
    S.segquant_quantize_mxfp4(x, out=(codes[:n], scales[:m]))
    assert (codes[n:] == 0xAB).all() and (scales[m:] == 0xAB).all()
    got = S.segquant_unpack_mxfp4((codes[:n], scales[:m]), M, K)
    assert torch.equal(got.cpu().double(), mx_ref(x))
    # columns up to the end of the last tile are zeros
    tile = codes[:n].view(-1, -(-K // 128), 4, 16, 16)
    if K % 128:
        for r in range(M):
            assert not tile[r // 16, -1, 2:, r % 16].any()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_quantize_behind_an_activation(act):
    """The values are those of the bf16 activation that the group norm of one
    pixel gives, whose act() is the same function."""
    g = gen(5)
    M, K = 70, 1024
    z = (3 * normal(g, M, K)).to(BF)
    want = act_ref(z.double(), act).to(BF)
    got = S.segquant_unpack_mxfp4(S.segquant_quantize_mxfp4(z, ACTS[act]), M, K)
    ref = mx_ref(want)
    # act() within 2^-17: about one bf16 value in 2^9 may round the other way, and
    # a 4-bit value changes only where that one stands next to a border
    same = (got.cpu().double() == ref).double().mean()
    assert same > 1 - 2.0 ** -9, float(same)


@pytest.mark.parametrize("rows,power", [([0, 1, 2, 3, 16, 17, 18, 19], 100.0),
                                        ([4, 5, 6, 7, 20, 21, 22, 23], 0.0),
                                        ([8, 9, 10, 11, 24, 25, 26, 27], 0.0),
                                        ([12, 13, 14, 15, 28, 29, 30, 31], 0.0)])
def test_gelu_of_every_value_in_both_forms(rows, power):
    """Every finite bf16 value behind GELU, blocks of 32 neighbours: the quantiser
    against the product that quantises its rows itself, read off a weight with one
    power of two in each column, so that each y is one value, exactly."""
    K = 2048
    bits = torch.arange(65536, device=DEV, dtype=torch.int32).view(32, K)[rows]
    bits = torch.where((bits & 0x7f80) == 0x7f80, torch.zeros_like(bits), bits)
    z = (bits << 16).view(torch.float32).to(BF)
    got = S.segquant_unpack_mxfp4(S.segquant_quantize_mxfp4(z, S.SEGQ_ACT_GELU), 8, K)
    assert S.segquant_gemm_mxfp4_workspace_bytes(8, K, K) == 0
    w = S.segquant_quantize_weight_mxfp4(2.0 ** power * torch.eye(K, device=DEV))
    y = S.segquant_gemm_mxfp4(z, w, K, act_kind=S.SEGQ_ACT_GELU)
    assert torch.equal(y.double(), got.double() * 2.0 ** power)
    want = act_ref(z.double().cpu(), "gelu").to(BF)
    same = (got.cpu().double() == mx_ref(want)).double().mean()
    assert same > 1 - 2.0 ** -9, float(same)  # as above


@pytest.mark.parametrize("K,N", [(64, 16), (128, 48), (192, 80), (1536, 144), (2112, 32)])
def test_quantize_weight(K, N):
    g = gen(K + N)
    w = edge_values(g, N, K).t().contiguous()
    _, w = padded(w, N + 3, float("nan"))
    got = S.segquant_unpack_mxfp4(S.segquant_quantize_weight_mxfp4(w), N, K)
    assert torch.equal(got.cpu().double(), mx_ref(w.t()))


def product_close(y, x, w, K):
    x, w = x.to(DEV).double(), w.to(DEV).double()
    ref, size = x @ w.t(), x.abs() @ w.abs().t()
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -20 + 2.0 ** -24 * (K / 128 + 1)) * size + 2.0 ** -133
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))


SHAPES = [(1, 16, 64), (2, 9216, 1536), (5, 48, 128), (16, 1536, 6144), (16, 16, 16384),
          (17, 32, 192), (31, 1040, 320), (64, 512, 512), (77, 4608, 1536), (100, 176, 704),
          (128, 128, 1024), (129, 272, 2112), (257, 1536, 576), (333, 1536, 1536), (600, 4096, 256),
          (1000, 208, 4096), (1025, 2064, 128), (4429, 1536, 1536), (2048, 6144, 640)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("codes", [False, True])
def test_product(M, N, K, codes):
    g = gen(M + N + K)
    z = (normal(g, M, K) * torch.exp(normal(g, M, 1))).to(BF)
    _, z = padded(z, K + 8, float("nan"))
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N) * torch.exp(normal(g, 1, N)))
    mx = S.segquant_quantize_mxfp4(z)
    ybuf, y = padded(torch.zeros(M, N, device=DEV, dtype=BF), N + 8, 7.0)
    args = dict(K=K, xq=mx) if codes else {}
    assert S.segquant_gemm_mxfp4(None if codes else z, w, N, out=y, **args) is y
    product_close(y, S.segquant_unpack_mxfp4(mx, M, K), S.segquant_unpack_mxfp4(w, N, K), K)
    assert (ybuf[:, N:] == 7.0).all()
    again = S.segquant_gemm_mxfp4(None if codes else z, w, N, M=M, **args)
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))


# every tile shape, K ending in every stage of a block of scales, ragged rows and columns
FORMS = [(1551, 4656, 960), (1171, 6208, 1088), (1463, 4896, 1216), (3909, 1968, 832),
         (3480, 3088, 448), (5486, 1824, 576), (5991, 1600, 704), (5892, 1952, 320),
         (4742, 2656, 960), (2709, 4512, 1088), (2624, 5024, 704), (2585, 4880, 832),
         (4871, 2848, 448), (5786, 2336, 576), (4719, 2848, 704), (3266, 4368, 320),
         (4509, 1296, 448), (4101, 1424, 576), (3429, 2048, 192), (4545, 1312, 320),
         (388, 5136, 448), (4593, 1136, 64), (488, 6272, 192), (1190, 1968, 320),
         (25, 48, 1472), (188, 80, 64), (29, 96, 192), (378, 16, 320), (160, 1536, 12288),
         (4857, 2352, 1472), (3663, 3168, 1600), (4578, 2576, 1728), (4844, 2336, 1856),
         (642, 3408, 448), (871, 6080, 64), (3173, 1008, 192), (2532, 1008, 320),
         (962, 6192, 192), (1924, 3760, 576), (1199, 5680, 704), (4526, 1344, 1024),
         (4590, 1312, 640), (1525, 4000, 1728), (3472, 1712, 1408), (5136, 1568, 448),
         (4642, 1712, 576), (1897, 5280, 192), (2370, 3392, 320), (2990, 3184, 1088)]


@pytest.mark.parametrize("M,N,K", FORMS)
def test_every_form_of_the_product(M, N, K):
    g = gen(M + N + K)
    z = (normal(g, M, K) * torch.exp(normal(g, M, 1))).to(BF)
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N) * torch.exp(normal(g, 1, N)))
    mx = S.segquant_quantize_mxfp4(z)
    ybuf, y = padded(torch.zeros(M, N, device=DEV, dtype=BF), N + 8, 7.0)
    S.segquant_gemm_mxfp4(None, w, N, K=K, xq=mx, out=y)
    product_close(y, S.segquant_unpack_mxfp4(mx, M, K), S.segquant_unpack_mxfp4(w, N, K), K)
    assert (ybuf[:, N:] == 7.0).all()
    for _ in range(2):  # the same bits again
        assert torch.equal(S.segquant_gemm_mxfp4(z, w, N), y)


def test_rows_far_apart():
    """Row distances that pass 32 bits, in elements and in bytes."""
    g = gen(11)
    M, N, K, far = 4, 64, 192, (1 << 30) + 64
    z = torch.empty(M * far, device=DEV, dtype=BF).view(M, far)[:, :K]
    y = torch.empty(M * far, device=DEV, dtype=BF).view(M, far)[:, :N]
    z.copy_(normal(g, M, K))
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N))
    want = S.segquant_gemm_mxfp4(z.contiguous(), w, N)
    mx = S.segquant_quantize_mxfp4(z)
    assert torch.equal(S.segquant_gemm_mxfp4(z, w, N, out=y), want)
    y.zero_()
    assert torch.equal(S.segquant_gemm_mxfp4(None, w, N, K=K, xq=mx, out=y), want)


@pytest.mark.parametrize("act", list(ACTS))
def test_more_rows_than_a_launch_takes(act):
    """1048544 rows fill one launch of the quantiser; its rows and the product's, on
    both sides of the border, are those of a call on them alone."""
    g = gen(12)
    M, N, K, border = 1048544 + 41, 48, 64, 1048544
    z = normal(g, M, K).to(BF)
    codes, scales = S.segquant_quantize_mxfp4(z, ACTS[act])
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N))
    y = S.segquant_gemm_mxfp4(z, w, N, act_kind=ACTS[act])
    for first, last in [(0, 64), (border - 32, border + 32), (border, M)]:
        c, s = S.segquant_quantize_mxfp4(z[first:last], ACTS[act])
        assert torch.equal(codes[first * 64:][:c.numel()], c)
        assert torch.equal(scales[first * 16:][:s.numel()], s)
        # K = 64 is one instruction: every form of the product gives the same bits
        assert torch.equal(S.segquant_gemm_mxfp4(z[first:last], w, N, act_kind=ACTS[act]),
                           y[first:last])


def test_calls_at_once_on_two_streams():
    g = gen(21)
    N, K = 1536, 1536
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N))
    z = [normal(g, M, K).to(BF) for M in (900, 40)]
    want = [S.segquant_gemm_mxfp4(x, w, N) for x in z]
    streams = [torch.cuda.Stream() for _ in z]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(S.segquant_gemm_mxfp4(z[i], w, N))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])


@pytest.mark.parametrize("M", [1, 7, 16, 60, 200])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_product_behind_an_activation_is_the_quantiser_s(M, act):
    g = gen(M)
    z = (2 * normal(g, M, 1600)).to(BF)
    w = S.segquant_quantize_weight_mxfp4(normal(g, 1600, 96))
    mx = S.segquant_quantize_mxfp4(z, ACTS[act])
    y = S.segquant_gemm_mxfp4(z, w, 96, act_kind=ACTS[act])
    product_close(y, S.segquant_unpack_mxfp4(mx, M, 1600), S.segquant_unpack_mxfp4(w, 96, 1600),
                  1600)


@pytest.mark.parametrize("M,N,K", [(8, 9216, 1536), (4, 64, 6144), (12, 8208, 1024), (3, 80, 8192),
                                   (4, 9216, 1536), (5, 96, 1600), (4, 48, 4096), (1, 32, 16384),
                                   (8, 8208, 2048), (16, 16, 512), (3, 16, 64), (2, 8192, 192)])
@pytest.mark.parametrize("act", list(ACTS))
def test_few_rows_are_quantised_inside(M, N, K, act):
    assert S.segquant_gemm_mxfp4_workspace_bytes(M, N, K) == 0
    g = gen(M + K)
    z = (2 * normal(g, M, K) * torch.exp(normal(g, M, 1))).to(BF)
    z[0, :64] = 0
    _, z = padded(z, K + 8, float("nan"))
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N))
    mx = S.segquant_quantize_mxfp4(z, ACTS[act])
    y = S.segquant_gemm_mxfp4(z, w, N, act_kind=ACTS[act], workspace=None)
    product_close(y, S.segquant_unpack_mxfp4(mx, M, K), S.segquant_unpack_mxfp4(w, N, K), K)


@pytest.mark.parametrize("M,N,K", [(17, 48, 64), (31, 2064, 1472), (32, 16, 128), (33, 80, 192),
                                   (48, 4624, 1536), (77, 1536, 1536), (77, 4608, 1536),
                                   (250, 512, 640), (345, 176, 320), (1000, 64, 576)])
def test_rows_without_an_activation_give_the_bits_of_their_codes(M, N, K):
    g = gen(M + N + K)
    z = (normal(g, M, K) * torch.exp(normal(g, M, 1))).to(BF)
    z[M // 2, K // 2:] = 0
    z[M - 1, 3] = float("inf")  # a row of NaN
    _, z = padded(z, K + 8, float("nan"))
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N))
    mx = S.segquant_quantize_mxfp4(z)
    ybuf, y = padded(torch.zeros(M, N, device=DEV, dtype=BF), N + 8, 7.0)
    S.segquant_gemm_mxfp4(z, w, N, out=y)
    want = S.segquant_gemm_mxfp4(None, w, N, K=K, xq=mx, M=M)
    assert torch.isnan(y[-1]).all() and torch.isnan(want[-1]).all()
    assert torch.equal(y[:-1], want[:-1])
    product_close(y[:-1], S.segquant_unpack_mxfp4(mx, M, K)[:-1], S.segquant_unpack_mxfp4(w, N, K), K)
    assert (ybuf[:, N:] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(3, 64, 256), (200, 128, 192), (700, 1024, 512)])
def test_ones_and_powers_are_exact(M, N, K):
    """Small integers and powers of two: every sum is exact in fp32."""
    g = gen(K)
    x = torch.randint(-6, 7, (M, K), generator=g, device=DEV).float()
    x[x.abs() == 5] = 4.0
    x[:, ::32] = 6.0  # the scale of every block is 1
    x = x * torch.exp2(torch.randint(-40, 40, (M, 1), generator=g, device=DEV).float())
    w = torch.exp2(torch.randint(-1, 2, (K, N), generator=g, device=DEV).float())
    mx = S.segquant_quantize_weight_mxfp4(w)
    y = S.segquant_gemm_mxfp4(x.to(BF), mx, N)
    want = (x.double() @ w.double()).float().to(BF)
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [4, 40, 400, 6000])
def test_nan_and_infinity_reach_their_rows_only(M):
    g = gen(M)
    K, N = 640, 144
    z = normal(g, M, K).to(BF)
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N))
    clean = S.segquant_gemm_mxfp4(z, w, N)
    bad = z.clone()
    bad[1, 70], bad[3, 639] = float("inf"), float("nan")
    y = S.segquant_gemm_mxfp4(bad, w, N)
    hit = torch.zeros(M, dtype=torch.bool, device=DEV)
    hit[1] = hit[3] = True
    assert y[hit].isnan().all() and torch.equal(y[~hit], clean[~hit])
    assert S.segquant_unpack_mxfp4(S.segquant_quantize_mxfp4(bad), M, K)[1, 64:96].isnan().all()


def test_rows_of_padding_do_not_matter():
    """The codes and scales of the rows behind the last hold anything."""
    g = gen(2)
    M, N, K = 37, 64, 320
    mx = S.segquant_quantize_mxfp4(normal(g, M, K).to(BF))
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N))
    y = S.segquant_gemm_mxfp4(None, w, N, K=K, xq=mx, M=M)
    codes, scales = mx[0].clone(), mx[1].clone()
    codes.view(-1, 3, 4, 16, 16)[2, :, :, 5:] = 0x77
    scales.view(-1, 1, 4, 16, 4)[2, :, :, 5:] = 0xFF
    assert torch.equal(S.segquant_gemm_mxfp4(None, w, N, K=K, xq=(codes, scales), M=M), y)


def test_no_rows():
    w = S.segquant_quantize_weight_mxfp4(torch.ones(64, 16, device=DEV))
    z = torch.zeros(0, 64, device=DEV, dtype=BF)
    assert S.segquant_gemm_mxfp4(z, w, 16).shape == (0, 16)
    codes, scales = S.segquant_quantize_mxfp4(z)
    assert codes.numel() == scales.numel() == 0


@pytest.mark.parametrize("M", [3, 300, 3000])
def test_other_stream_and_two_graphs_on_one_workspace(M):
    g = gen(M)
    N, K = 256, 512
    w = S.segquant_quantize_weight_mxfp4(normal(g, K, N))
    z = [normal(g, M, K).to(BF) for _ in range(2)]
    ws = torch.empty(max(16, S.segquant_gemm_mxfp4_workspace_bytes(M, N, K)), dtype=torch.uint8,
                     device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = S.segquant_gemm_mxfp4(z[0], w, N, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    out = [torch.empty(M, N, device=DEV, dtype=BF) for _ in range(2)]
    graphs = []
    for i in range(2):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            S.segquant_gemm_mxfp4(z[i], w, N, act_kind=ACTS["silu"], out=out[i], workspace=ws)
        graphs.append(graph)
    assert torch.equal(first, S.segquant_gemm_mxfp4(z[0], w, N))
    for step in range(3):
        for i in range(2):
            z[i].copy_(normal(g, M, K))
        for i in range(2):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(out[i], S.segquant_gemm_mxfp4(z[i], w, N, act_kind=ACTS["silu"]))
