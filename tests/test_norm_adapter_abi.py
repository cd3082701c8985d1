"""Refusals of segquant_groupnorm_quantize, segquant_adanorm_quantize and
segquant_adapter_add without a GPU: the documented status before any HIP call,
through the C ABI with fake device addresses, and the Python binding's own
checks of types, shapes and strides."""
import ctypes

import numpy as np
import pytest
import torch

import segmented_dual_scale_amd as S
from test_abi import _gpu_present, segs

pytestmark = pytest.mark.skipif(_gpu_present(), reason="fake device pointers: CPU-only tests")

P = ctypes.c_void_p
FAKE, FAKE2, ODD8, ODD2 = 0x10000, 0x20000, 0x10008, 0x10002


def lib():
    return S.load_library()


def groupnorm(B=2, Px=4, C=64, z=FAKE, ld_z=None, groups=8, eps=1e-5, gamma=FAKE, beta=FAKE,
              scale=None, shift=None, ld_mod=64, act_kind=1, widths=None, act=FAKE, q=FAKE2,
              ld_q=64, layout=0, x=FAKE2, ld_xo=64, work=None, work_bytes=0):
    o, w = segs(widths if widths is not None else [C])
    return lib().segquant_groupnorm_quantize(
        z, B, Px, C, C if ld_z is None else ld_z, groups, eps, gamma, beta, scale, shift, ld_mod,
        act_kind, len(w), o.ctypes.data, w.ctypes.data, act, q, ld_q, layout, x, ld_xo, work,
        work_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), S.SEGQ_ERR_NULL),
    (dict(z=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(ld_z=68), S.SEGQ_ERR_ALIGN),
    (dict(ld_z=56), S.SEGQ_ERR_SHAPE),
    (dict(B=-1), S.SEGQ_ERR_SHAPE),
    (dict(C=0), S.SEGQ_ERR_SHAPE),
    (dict(B=1 << 16, Px=1 << 16), S.SEGQ_ERR_SHAPE),
    (dict(B=1 << 16, Px=1), S.SEGQ_ERR_UNSUPPORTED),
    (dict(C=1 << 21, groups=8, ld_q=1 << 21, ld_xo=1 << 21), S.SEGQ_ERR_UNSUPPORTED),
    (dict(groups=0), S.SEGQ_ERR_SHAPE),
    (dict(groups=7), S.SEGQ_ERR_SHAPE),
    (dict(eps=0.0), S.SEGQ_ERR_SHAPE),
    (dict(eps=1e-39), S.SEGQ_ERR_SHAPE),
    (dict(eps=float("nan")), S.SEGQ_ERR_SHAPE),
    (dict(eps=float("inf")), S.SEGQ_ERR_SHAPE),
    (dict(gamma=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(beta=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(scale=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(shift=FAKE, ld_mod=60), S.SEGQ_ERR_SHAPE),
    (dict(shift=FAKE, ld_mod=68), S.SEGQ_ERR_ALIGN),
    (dict(act_kind=3), S.SEGQ_ERR_SHAPE),
    (dict(q=None, x=None), S.SEGQ_ERR_NULL),
    (dict(act=None), S.SEGQ_ERR_NULL),
    (dict(layout=2), S.SEGQ_ERR_SHAPE),
    (dict(ld_q=48), S.SEGQ_ERR_SHAPE),
    (dict(ld_q=72), S.SEGQ_ERR_ALIGN),
    (dict(q=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(x=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(ld_xo=60), S.SEGQ_ERR_SHAPE),
    (dict(C=128, ld_q=128, ld_xo=128, widths=[64]), S.SEGQ_ERR_SEGMENTS),
    (dict(widths=[32, 32]), S.SEGQ_ERR_ALIGN),
    (dict(x=FAKE, ld_z=72), S.SEGQ_ERR_SHAPE),          # in place with another row distance
    (dict(Px=100000), S.SEGQ_ERR_UNSUPPORTED),          # two launches: no workspace
    (dict(Px=100000, work=FAKE, work_bytes=64), S.SEGQ_ERR_UNSUPPORTED),
    (dict(Px=100000, work=ODD8, work_bytes=1 << 30), S.SEGQ_ERR_ALIGN),
])
def test_groupnorm_refusals(kw, status):
    assert groupnorm(**kw) == status
    assert S.segquant_last_error() != ""


def test_groupnorm_of_no_rows_is_ok():
    assert groupnorm(B=0, z=None, q=None, x=None) == S.SEGQ_OK
    assert groupnorm(Px=0, z=None, q=None, x=None) == S.SEGQ_OK
    assert S.segquant_last_error() == ""


def test_groupnorm_workspace_bytes():
    assert S.segquant_groupnorm_workspace_bytes(2, 64, 1280, 32) == 0  # fits the registers
    big = S.segquant_groupnorm_workspace_bytes(1, 1 << 20, 128, 32)
    assert 0 < big < 1 << 20
    assert S.segquant_groupnorm_workspace_bytes(0, 1 << 20, 128, 32) == 0
    assert S.segquant_groupnorm_workspace_bytes(1, 64, 100, 3) == 0
    assert "groups" in S.segquant_last_error()


def adanorm(M=8, K=64, h=FAKE, ld_h=None, branch=FAKE, ld_b=64, gate=FAKE, h_out=FAKE2, ld_ho=64,
            eps=1e-6, gamma=None, beta=None, scale=FAKE, shift=FAKE, ld_mod=64, n_req=2,
            row_offset=FAKE, widths=None, act=FAKE, q=FAKE2, ld_q=64, layout=0, x=FAKE2, ld_xo=64):
    o, w = segs(widths if widths is not None else [K])
    return lib().segquant_adanorm_quantize(
        h, M, K, K if ld_h is None else ld_h, branch, ld_b, gate, h_out, ld_ho, eps, gamma, beta,
        scale, shift, ld_mod, n_req, row_offset, len(w), o.ctypes.data, w.ctypes.data, act, q, ld_q,
        layout, x, ld_xo, None)


@pytest.mark.parametrize("kw,status", [
    (dict(h=None), S.SEGQ_ERR_NULL),
    (dict(h=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(ld_h=72 + 4), S.SEGQ_ERR_ALIGN),
    (dict(M=-1), S.SEGQ_ERR_SHAPE),
    (dict(n_req=0), S.SEGQ_ERR_SHAPE),
    (dict(row_offset=None, n_req=3), S.SEGQ_ERR_SHAPE),
    (dict(row_offset=ODD2), S.SEGQ_ERR_ALIGN),
    (dict(branch=None), S.SEGQ_ERR_NULL),
    (dict(branch=None, gate=None), S.SEGQ_ERR_NULL),
    (dict(branch=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(ld_b=56), S.SEGQ_ERR_SHAPE),
    (dict(h_out=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(ld_ho=60), S.SEGQ_ERR_SHAPE),
    (dict(h_out=FAKE, ld_ho=72), S.SEGQ_ERR_SHAPE),
    (dict(gate=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(scale=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(shift=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(ld_mod=56), S.SEGQ_ERR_SHAPE),
    (dict(gamma=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(eps=-1.0), S.SEGQ_ERR_SHAPE),
    (dict(q=None, x=None, h_out=None), S.SEGQ_ERR_NULL),
    (dict(act=None), S.SEGQ_ERR_NULL),
    (dict(ld_q=72), S.SEGQ_ERR_ALIGN),
    (dict(ld_xo=56), S.SEGQ_ERR_SHAPE),
    (dict(widths=[32, 32]), S.SEGQ_ERR_ALIGN),
])
def test_adanorm_refusals(kw, status):
    assert adanorm(**kw) == status
    assert S.segquant_last_error() != ""


def test_adanorm_of_no_rows_is_ok():
    assert adanorm(M=0, h=None, q=None, x=None, h_out=None) == S.SEGQ_OK


def adapter(M=8, N=64, K=64, x=FAKE, ld_x=None, n_req=2, row_offset=FAKE, ids=FAKE, n_adapters=2,
            rank=16, rank_of=FAKE, a=FAKE, b=FAKE, alpha=FAKE, widths=None, base=FAKE, ld_base=64,
            y=FAKE2, ld_y=64, work=FAKE, work_bytes=1 << 30, n_nseg=None):
    o, w = segs(widths if widths is not None else [N])
    return lib().segquant_adapter_add(
        M, N, K, x, K if ld_x is None else ld_x, n_req, row_offset, ids, n_adapters, rank, rank_of,
        a, b, alpha, len(w) if n_nseg is None else n_nseg, o.ctypes.data, w.ctypes.data, base,
        ld_base, y, ld_y, work, work_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), S.SEGQ_ERR_SHAPE),
    (dict(N=1 << 20, ld_base=1 << 20, ld_y=1 << 20), S.SEGQ_ERR_UNSUPPORTED),
    (dict(K=72, ld_x=72), S.SEGQ_ERR_ALIGN),
    (dict(N=40), S.SEGQ_ERR_ALIGN),
    (dict(M=(1 << 27) + 1), S.SEGQ_ERR_UNSUPPORTED),
    (dict(n_req=(1 << 22) + 1), S.SEGQ_ERR_UNSUPPORTED),
    (dict(n_req=0), S.SEGQ_ERR_SHAPE),
    (dict(n_adapters=0), S.SEGQ_ERR_SHAPE),
    (dict(rank=8), S.SEGQ_ERR_ALIGN),
    (dict(rank=0), S.SEGQ_ERR_ALIGN),
    (dict(rank=272), S.SEGQ_ERR_UNSUPPORTED),
    (dict(x=None), S.SEGQ_ERR_NULL),
    (dict(x=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(ld_x=68), S.SEGQ_ERR_ALIGN),
    (dict(row_offset=None), S.SEGQ_ERR_NULL),
    (dict(ids=None), S.SEGQ_ERR_NULL),
    (dict(a=None), S.SEGQ_ERR_NULL),
    (dict(b=None), S.SEGQ_ERR_NULL),
    (dict(y=None), S.SEGQ_ERR_NULL),
    (dict(a=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(b=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(row_offset=ODD2), S.SEGQ_ERR_ALIGN),
    (dict(ids=ODD2), S.SEGQ_ERR_ALIGN),
    (dict(rank_of=ODD2), S.SEGQ_ERR_ALIGN),
    (dict(alpha=ODD2), S.SEGQ_ERR_ALIGN),
    (dict(base=ODD8), S.SEGQ_ERR_ALIGN),
    (dict(ld_base=66), S.SEGQ_ERR_ALIGN),
    (dict(ld_y=56), S.SEGQ_ERR_SHAPE),
    (dict(y=FAKE, ld_base=72), S.SEGQ_ERR_SHAPE),
    (dict(widths=[32]), S.SEGQ_ERR_SEGMENTS),
    (dict(widths=[24, 40]), S.SEGQ_ERR_ALIGN),
    (dict(n_nseg=0), S.SEGQ_ERR_SEGMENTS),
    (dict(N=16 * 129, widths=[16] * 129), S.SEGQ_ERR_UNSUPPORTED),
    (dict(M=64, rank=256, work=None), S.SEGQ_ERR_UNSUPPORTED),  # two launches
    (dict(M=64, rank=256, work_bytes=64 * 256 * 4 - 1), S.SEGQ_ERR_UNSUPPORTED),
    (dict(M=64, rank=256, work=ODD8), S.SEGQ_ERR_ALIGN),
])
def test_adapter_refusals(kw, status):
    assert adapter(**kw) == status
    assert S.segquant_last_error() != ""


def test_adapter_of_no_rows_is_ok():
    assert adapter(M=0, x=None, y=None, work=None) == S.SEGQ_OK
    assert S.segquant_adapter_workspace_bytes(0, 64, 64, 1, 16) == 0


def test_adapter_workspace_bytes():
    assert S.segquant_adapter_workspace_bytes(100, 64, 64, 3, 16, [16, 48]) == 0  # one launch
    two = S.segquant_adapter_workspace_bytes(4096, 64, 65536, 3, 16, [16, 48])
    assert two > 0 and two % (4096 * 2 * 16 * 4) == 0
    assert S.segquant_adapter_workspace_bytes(100, 64, 60, 3, 16) == 0
    assert "K" in S.segquant_last_error()


B2 = 2  # bytes of a bf16 element
ADANORM_APART = dict(M=8, K=64, q=None, h_out=0x30000, x=0x40000)


@pytest.mark.parametrize("kw,status", [
    # x_out one row, one 16-byte step, or one row's end into z
    (dict(x=FAKE + 64 * B2, q=None), S.SEGQ_ERR_SHAPE),
    (dict(x=FAKE + 8 * B2, q=None), S.SEGQ_ERR_SHAPE),
    (dict(x=FAKE - 7 * 64 * B2, q=None), S.SEGQ_ERR_SHAPE),
    (dict(x=FAKE + 64 * B2, ld_z=120, ld_xo=120, q=None), S.SEGQ_ERR_SHAPE),
    (dict(x=FAKE + 7 * 64 * B2, ld_xo=1 << 40, q=None), S.SEGQ_ERR_SHAPE),
])
def test_groupnorm_outputs_that_overlap(kw, status):
    assert groupnorm(**kw) == status and "overlaps" in S.segquant_last_error()


@pytest.mark.parametrize("kw", [
    dict(h_out=FAKE + 64 * B2), dict(h_out=FAKE - 64 * B2), dict(x=FAKE), dict(x=0x30000),
    dict(branch=0x50000, h_out=0x50000 + 64 * B2), dict(branch=0x50000, x=0x50000),
    dict(branch=0x50000, h_out=0x50000, ld_ho=72),
])
def test_adanorm_outputs_that_overlap(kw):
    assert adanorm(**{**ADANORM_APART, **kw}) == S.SEGQ_ERR_SHAPE
    assert "overlaps" in S.segquant_last_error()


@pytest.mark.parametrize("kw", [
    dict(x=FAKE2), dict(x=FAKE2 + 7 * 64 * B2), dict(base=FAKE2 + 64 * B2),
    dict(base=FAKE2 - 63 * 64 * B2, M=64), dict(x=FAKE2 + 64 * B2, ld_x=72, ld_y=128),
    dict(x=FAKE2 + 64 * B2, ld_x=120, ld_y=120),
])
def test_adapter_outputs_that_overlap(kw):
    assert adapter(**kw) == S.SEGQ_ERR_SHAPE and "overlaps" in S.segquant_last_error()


@pytest.mark.parametrize("kw", [
    dict(x=FAKE2 + 64 * B2, ld_x=128, ld_y=128),   # side by side in one buffer
    dict(x=FAKE2 + 64 * B2, ld_x=72, ld_y=1024),   # between two rows
    dict(x=FAKE2 + 8 * 64 * B2), dict(base=FAKE2), dict(x=FAKE2 - 8 * 64 * B2),
])
def test_outputs_beside_inputs_reach_the_launch(kw):
    assert adapter(**kw) == S.SEGQ_ERR_HIP


# The binding looks at its operands before it calls: these never reach a GPU.
def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("kw,text", [
    (dict(z=torch.zeros(1, 4, 64)), "bfloat16"),
    (dict(z=bf(4, 64)), r"\[B\]\[P\]\[C\]"),
    (dict(gamma=torch.zeros(32)), "gamma"),
    (dict(gamma=torch.zeros(64, dtype=torch.float64)), "gamma"),
    (dict(beta=torch.zeros(128)[::2]), "beta"),
    (dict(scale=bf(2, 64)), "scale"),
    (dict(x_out=bf(1, 4, 32)), "x_out"),
    (dict(act_scales=torch.zeros(4, 2)), "act_scales"),
    (dict(act_scales=torch.zeros(4, 1), out=torch.zeros(4, 64)), "out"),
    (dict(act_scales=torch.zeros(4, 1), out=torch.zeros(3, 64, dtype=torch.int8)), "out"),
    (dict(z=bf(1, 64, 4).transpose(1, 2)), "unit stride"),
    (dict(z=bf(2, 9, 64)[:, :4]), "evenly spaced"),
    (dict(workspace="mine"), "workspace"),
    (dict(x_out=True, scale=bf(1, 64), shift=bf(1, 128)[:, ::2]), "unit stride"),
    (dict(x_out=True, z=bf(2, 4, 64), scale=bf(2, 64), shift=bf(2, 72)[:, :64]), "row stride"),
    (dict(x_out=True), "on a GPU"),
])
def test_groupnorm_binding_refusals(kw, text):
    with pytest.raises(ValueError, match=text):
        S.segquant_groupnorm_quantize(kw.pop("z", bf(1, 4, 64)), 8, **kw)


@pytest.mark.parametrize("kw,text", [
    (dict(h=bf(1, 4, 64)), r"\[M\]\[K\]"),
    (dict(scale=bf(2, 64), row_offset=torch.zeros(2, dtype=torch.int32)), "scale"),
    (dict(scale=bf(2, 64), shift=bf(2, 128)[:, :64]), "row stride"),
    # a request alone has no row stride, its columns have one all the same
    (dict(x_out=True, scale=bf(1, 64), shift=bf(64, 1).t(), gate=bf(1, 128)[:, ::2],
          branch=bf(4, 64)), "unit stride"),
    (dict(x_out=True, shift=bf(2, 64), gate=bf(2, 128)[:, ::2], branch=bf(4, 64)), "unit stride"),
    (dict(act_scales=torch.zeros(4, 1), h=bf(1, 64),
          out=torch.zeros(1, 128, dtype=torch.int8)[:, ::2]), "unit stride"),
    (dict(act_scales=torch.zeros(4, 1), h=bf(1, 64), layout=S.SEGQ_Q_PLANES,
          out=torch.zeros(2, 1, 128, dtype=torch.int8)[:, :, ::2]), "unit stride"),
    (dict(x_out=True, n_req=2, row_offset=torch.zeros(2, dtype=torch.int32)), "n_req"),
    (dict(branch=bf(4, 32)), "branch"),
    (dict(row_offset=torch.zeros(3, dtype=torch.int64)), "row_offset"),
    (dict(branch=bf(4, 64), h_out=torch.zeros(4, 64)), "h_out"),
    (dict(x_out=True), "on a GPU"),
])
def test_adanorm_binding_refusals(kw, text):
    with pytest.raises(ValueError, match=text):
        S.segquant_adanorm_quantize(kw.pop("h", bf(4, 64)), **kw)


@pytest.mark.parametrize("kw,text", [
    (dict(x=torch.zeros(4, 64)), "bfloat16"),
    (dict(a=bf(2, 32, 64)), "a must be"),
    (dict(a=bf(2, 16, 128)[:, :, :64]), "a must be contiguous"),
    (dict(adapter=torch.zeros(1, dtype=torch.int64)), "adapter"),
    (dict(row_offset=torch.zeros(3, dtype=torch.int32)), "row_offset"),
    (dict(rank=torch.zeros(3, dtype=torch.int32)), "rank"),
    (dict(alpha=torch.zeros(2, dtype=torch.bfloat16)), "alpha"),
    (dict(base=bf(4, 64)), "base"),
    (dict(out=bf(5, 32)), "out"),
    (dict(), "on a GPU"),
])
def test_adapter_binding_refusals(kw, text):
    args = dict(x=bf(4, 64), a=bf(2, 16, 64), b=bf(2, 32, 16),
                adapter=torch.zeros(1, dtype=torch.int32),
                row_offset=torch.zeros(2, dtype=torch.int32), base=bf(4, 32))
    args.update(kw)
    with pytest.raises(ValueError, match=text):
        S.segquant_adapter_add(**args)


def test_row_distance_of_views():
    assert S._row_ld(bf(3, 5, 64), "t") == 64
    assert S._row_ld(bf(3, 5, 72)[:, :, :64], "t") == 72
    assert S._row_ld(bf(3, 5, 64)[:, :1], "t") == 5 * 64  # one row per sample
    assert S._row_ld(bf(1, 5, 61), "t") == 61
    assert S._row_ld(bf(1, 1, 61), "t") == 64             # a single row: any distance
    assert S._row_ld(bf(8, 64)[::2], "t") == 128
    assert np.int64(S._row_ld(None, "t")) == 0


def test_segment_widths_are_read_at_every_call():
    w = [torch.tensor(64), torch.tensor(64)]
    assert S._segs(w, 128)[1].tolist() == [64, 64]
    w[0] += 64
    assert S._segs(w, 192)[1].tolist() == [128, 64]
    assert S._segs(w, 192)[0].tolist() == [0, 128]


def test_the_layer_s_calls_on_a_cpu_tensor():
    with pytest.raises(ValueError, match="on a GPU"):
        S.segquant_quantize_dualscale(bf(4, 64), torch.zeros(4, 1), [64])
