"""Refusals of segquant_rmsnorm_quantize, segquant_qk_rotary and the MXFP4 calls
without a GPU: the documented status before any HIP call, through the C ABI with
fake device addresses, and the Python binding's own checks."""
import ctypes
import random
import time

import numpy as np
import pytest
import torch

import segmented_dual_scale_amd as S
from test_abi import _gpu_present, segs

pytestmark = pytest.mark.skipif(_gpu_present(), reason="fake device pointers: CPU-only tests")

# every operand in 4 MiB of its own
A = {name: 0x1000000 + (i << 22) for i, name in enumerate(
    ["h", "branch", "h_out", "gamma", "act", "q", "x", "codes", "scales", "z", "xc", "xs", "wc", "ws",
     "y", "work", "k", "q_out", "k_out", "qg", "kg", "pos", "freq"])}
BIG = 1 << 60


def lib():
    return S.load_library()


def rms(M=8, K=64, h=A["h"], ld_h=None, branch=A["branch"], ld_b=None, h_out=A["h_out"], ld_ho=None,
        eps=1e-6, gamma=A["gamma"], widths=None, act=A["act"], q=A["q"], ld_q=None, layout=0,
        x=A["x"], ld_xo=None, codes=A["codes"], scales=A["scales"]):
    o, w = segs(widths if widths is not None else [K])
    def ld(v):
        return -(-K // 16) * 16 if v is None else v
    return lib().segquant_rmsnorm_quantize(
        h, M, K, ld(ld_h), branch, ld(ld_b), h_out, ld(ld_ho), eps, gamma, len(w), o.ctypes.data,
        w.ctypes.data, act, q, ld(ld_q), layout, x, ld(ld_xo), codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(h=None), S.SEGQ_ERR_NULL), (dict(h=A["h"] + 8), S.SEGQ_ERR_ALIGN),
    (dict(ld_h=56), S.SEGQ_ERR_SHAPE), (dict(ld_h=68), S.SEGQ_ERR_ALIGN),
    (dict(M=-1), S.SEGQ_ERR_SHAPE), (dict(branch=None), S.SEGQ_ERR_NULL),
    (dict(branch=A["branch"] + 8), S.SEGQ_ERR_ALIGN), (dict(ld_b=60), S.SEGQ_ERR_SHAPE),
    (dict(h_out=A["h_out"] + 2), S.SEGQ_ERR_ALIGN), (dict(h_out=A["h"], ld_ho=72), S.SEGQ_ERR_SHAPE),
    (dict(eps=0.0), S.SEGQ_ERR_SHAPE), (dict(eps=float("nan")), S.SEGQ_ERR_SHAPE),
    (dict(gamma=A["gamma"] + 4), S.SEGQ_ERR_ALIGN), (dict(act=None), S.SEGQ_ERR_NULL),
    (dict(layout=2), S.SEGQ_ERR_SHAPE), (dict(ld_q=72), S.SEGQ_ERR_ALIGN),
    (dict(ld_xo=56), S.SEGQ_ERR_SHAPE), (dict(widths=[32, 32]), S.SEGQ_ERR_ALIGN),
    (dict(codes=None), S.SEGQ_ERR_NULL), (dict(scales=None), S.SEGQ_ERR_NULL),
    (dict(codes=A["codes"] + 8), S.SEGQ_ERR_ALIGN), (dict(scales=A["scales"] + 2), S.SEGQ_ERR_ALIGN),
    (dict(K=72), S.SEGQ_ERR_ALIGN),  # MXFP4 takes whole steps of 64
    (dict(K=1 << 23, widths=[1 << 23]), S.SEGQ_ERR_UNSUPPORTED),
    (dict(branch=None, h_out=None, q=None, x=None, codes=None, scales=None), S.SEGQ_ERR_NULL),
])
def test_rmsnorm_refusals(kw, status):
    assert rms(**kw) == status
    assert S.segquant_last_error() != ""


@pytest.mark.parametrize("kw", [
    dict(x=A["h"]), dict(x=A["h_out"] + 128), dict(h_out=A["h"] + 128), dict(codes=A["h"] + 1024 - 16),
    dict(scales=A["codes"] + 1020), dict(codes=A["q"] + 496), dict(codes=A["gamma"] + 240),
    dict(scales=A["act"] + 12), dict(x=A["branch"] + 16), dict(scales=A["x"] - 252),
])
def test_rmsnorm_outputs_that_overlap(kw):
    assert rms(**kw) == S.SEGQ_ERR_SHAPE and "overlaps" in S.segquant_last_error()


@pytest.mark.parametrize("kw", [
    dict(), dict(h_out=A["h"]), dict(h_out=A["branch"]), dict(codes=A["h"] + 1024),
    dict(scales=A["codes"] + 1024), dict(K=72, codes=None, scales=None),
    dict(x=A["h"] + 128, ld_h=128, ld_xo=128),
])
def test_rmsnorm_calls_that_reach_the_launch(kw):
    assert rms(**kw) == S.SEGQ_ERR_HIP


def test_no_rows_is_ok():
    assert rms(M=0, h=None, branch=None, h_out=None, q=None, x=None, codes=None,
               scales=None) == S.SEGQ_OK
    assert gemm(M=0, z=None, y=None, wc=None, ws=None) == S.SEGQ_OK
    assert quantize(M=0, z=None, codes=None, scales=None) == S.SEGQ_OK
    assert rotary(B=0, q=None, q_out=None) == S.SEGQ_OK
    assert rotary(L=0, q=None, q_out=None, pos=None) == S.SEGQ_OK


def quantize(M=20, K=192, z=A["z"], ld_z=None, act=0, codes=A["codes"], scales=A["scales"]):
    return lib().segquant_quantize_mxfp4(z, M, K, K if ld_z is None else ld_z, act, codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), S.SEGQ_ERR_NULL), (dict(z=A["z"] + 8), S.SEGQ_ERR_ALIGN),
    (dict(K=96), S.SEGQ_ERR_ALIGN), (dict(K=1 << 23), S.SEGQ_ERR_UNSUPPORTED),
    (dict(M=(1 << 27) + 1), S.SEGQ_ERR_UNSUPPORTED), (dict(M=-1), S.SEGQ_ERR_SHAPE),
    (dict(ld_z=184), S.SEGQ_ERR_SHAPE), (dict(ld_z=196), S.SEGQ_ERR_ALIGN),
    (dict(act=3), S.SEGQ_ERR_SHAPE), (dict(codes=None), S.SEGQ_ERR_NULL),
    (dict(scales=None), S.SEGQ_ERR_NULL), (dict(codes=A["codes"] + 4), S.SEGQ_ERR_ALIGN),
    (dict(scales=A["scales"] + 1), S.SEGQ_ERR_ALIGN),
    (dict(codes=A["z"] + 16), S.SEGQ_ERR_SHAPE), (dict(scales=A["codes"] + 4092), S.SEGQ_ERR_SHAPE),
])
def test_quantize_refusals(kw, status):
    assert quantize(**kw) == status
    assert S.segquant_last_error() != ""
    assert quantize(scales=A["codes"] + 4096) == S.SEGQ_ERR_HIP


def weight(K=192, N=32, w=A["z"], ld_w=32, codes=A["codes"], scales=A["scales"]):
    return lib().segquant_quantize_weight_mxfp4(w, K, N, ld_w, codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), S.SEGQ_ERR_NULL), (dict(w=A["z"] + 2), S.SEGQ_ERR_ALIGN),
    (dict(K=100), S.SEGQ_ERR_ALIGN), (dict(N=24), S.SEGQ_ERR_ALIGN), (dict(N=0), S.SEGQ_ERR_SHAPE),
    (dict(ld_w=31), S.SEGQ_ERR_SHAPE), (dict(codes=None), S.SEGQ_ERR_NULL),
    (dict(codes=A["z"]), S.SEGQ_ERR_SHAPE),
])
def test_quantize_weight_refusals(kw, status):
    assert weight(**kw) == status
    assert S.segquant_last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), S.SEGQ_ERR_NULL), (dict(x=None), S.SEGQ_ERR_NULL),
    (dict(x=A["x"] + 2), S.SEGQ_ERR_ALIGN), (dict(ld_x=60), S.SEGQ_ERR_SHAPE),
    (dict(K=32), S.SEGQ_ERR_ALIGN), (dict(x=A["codes"] + 64), S.SEGQ_ERR_SHAPE),
    (dict(), S.SEGQ_ERR_HIP),
])
def test_unpack_refusals(kw, status):
    a = dict(codes=A["codes"], scales=A["scales"], R=5, K=64, x=A["x"], ld_x=64)
    a.update(kw)
    assert lib().segquant_unpack_mxfp4(*a.values(), None) == status


def gemm(M=40, N=64, K=192, z=A["z"], ld_z=None, act=0, xc=None, xs=None, wc=A["wc"], ws=A["ws"],
         y=A["y"], ld_y=None, work=A["work"], work_bytes=1 << 20):
    return lib().segquant_gemm_mxfp4(M, N, K, z, K if ld_z is None else ld_z, act, xc, xs, wc, ws, y,
                                     N if ld_y is None else ld_y, work, work_bytes, None)


CODES = dict(z=None, xc=A["xc"], xs=A["xs"], work=None, work_bytes=0)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), S.SEGQ_ERR_SHAPE), (dict(N=0), S.SEGQ_ERR_SHAPE), (dict(N=40), S.SEGQ_ERR_ALIGN),
    (dict(K=96), S.SEGQ_ERR_ALIGN), (dict(K=0), S.SEGQ_ERR_SHAPE),
    (dict(M=(1 << 27) + 1), S.SEGQ_ERR_UNSUPPORTED), (dict(N=1 << 28), S.SEGQ_ERR_UNSUPPORTED),
    (dict(M=1 << 20, N=1 << 18), S.SEGQ_ERR_UNSUPPORTED), (dict(act=9), S.SEGQ_ERR_SHAPE),
    (dict(z=None), S.SEGQ_ERR_NULL), (dict(xc=A["xc"], xs=A["xs"]), S.SEGQ_ERR_NULL),
    (dict(CODES, xs=None), S.SEGQ_ERR_NULL), (dict(CODES, xc=A["xc"] + 8), S.SEGQ_ERR_ALIGN),
    (dict(CODES, xs=A["xs"] + 2), S.SEGQ_ERR_ALIGN), (dict(CODES, act=1), S.SEGQ_ERR_UNSUPPORTED),
    (dict(z=A["z"] + 8), S.SEGQ_ERR_ALIGN), (dict(ld_z=184), S.SEGQ_ERR_SHAPE),
    (dict(wc=None), S.SEGQ_ERR_NULL), (dict(ws=A["ws"] + 1), S.SEGQ_ERR_ALIGN),
    (dict(y=None), S.SEGQ_ERR_NULL), (dict(y=A["y"] + 8), S.SEGQ_ERR_ALIGN),
    (dict(ld_y=56), S.SEGQ_ERR_SHAPE), (dict(ld_y=68), S.SEGQ_ERR_ALIGN),
    (dict(work=A["work"] + 8), S.SEGQ_ERR_ALIGN), (dict(M=400, work=None), S.SEGQ_ERR_UNSUPPORTED),
    (dict(M=400, work_bytes=400 * 96), S.SEGQ_ERR_UNSUPPORTED),
    (dict(M=400, y=A["work"] + 64), S.SEGQ_ERR_SHAPE), (dict(y=A["z"] + 128), S.SEGQ_ERR_SHAPE),
    (dict(y=A["wc"] + 32), S.SEGQ_ERR_SHAPE), (dict(y=A["ws"] + 16), S.SEGQ_ERR_SHAPE),
    (dict(CODES, y=A["xc"] + 16), S.SEGQ_ERR_SHAPE), (dict(CODES, y=A["xs"]), S.SEGQ_ERR_SHAPE),
    (dict(M=400, work=A["wc"]), S.SEGQ_ERR_SHAPE),
    (dict(), S.SEGQ_ERR_HIP), (CODES, S.SEGQ_ERR_HIP),
])
def test_gemm_refusals(kw, status):
    assert gemm(**kw) == status
    assert S.segquant_last_error() != ""


def test_sizes_in_bytes():
    code, scale = lib().segquant_mxfp4_code_bytes, lib().segquant_mxfp4_scale_bytes
    assert S.segquant_mxfp4_bytes(1, 64) == (1024, 256)
    assert S.segquant_mxfp4_bytes(17, 576) == (2 * 5 * 1024, 2 * 2 * 256)
    assert S.segquant_mxfp4_bytes(0, 64) == (0, 0)
    assert code(4, 60) == 0 and scale(-1, 64) == 0 and S.segquant_last_error() != ""
    with pytest.raises(ValueError, match="64"):
        S.segquant_mxfp4_bytes(4, 60)
    ws = S.segquant_gemm_mxfp4_workspace_bytes
    assert ws(4096, 512, 1536) == sum(S.segquant_mxfp4_bytes(4096, 1536))
    assert ws(0, 512, 1536) == 0 and ws(4096, 500, 1536) == 0


I3 = ctypes.c_int64 * 3
DEFAULT = object()


def rotary(B=2, L=10, D=64, q=A["q"], Hq=4, qs=None, q_out=A["q_out"], qos=None, k=None, Hk=4, ks=None,
           k_out=DEFAULT, kos=None, norm=1, eps=1e-6, qg=None, kg=None, pos=A["pos"], per=0,
           widths=(32, 32), n=None, freq=A["freq"], style=0):
    if k_out is DEFAULT:
        k_out = A["k_out"] if k else None
    w = np.array(widths, dtype=np.int32)

    def st(s, H):
        return None if s == 0 else I3(*(s or (L * H * D, H * D, D)))
    return lib().segquant_qk_rotary(B, L, D, q, Hq, st(qs, Hq), q_out, st(qos, Hq), k, Hk, st(ks, Hk),
                                    k_out, st(kos, Hk), norm, eps, qg, kg, pos, per,
                                    len(w) if n is None else n, w.ctypes.data, freq, style, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), S.SEGQ_ERR_SHAPE), (dict(D=0), S.SEGQ_ERR_SHAPE), (dict(Hq=0), S.SEGQ_ERR_SHAPE),
    (dict(k=A["k"], Hk=0), S.SEGQ_ERR_SHAPE), (dict(D=68), S.SEGQ_ERR_ALIGN),
    (dict(D=520), S.SEGQ_ERR_UNSUPPORTED), (dict(L=1 << 29), S.SEGQ_ERR_UNSUPPORTED),
    (dict(n=0), S.SEGQ_ERR_SHAPE), (dict(widths=[8] * 9), S.SEGQ_ERR_SHAPE),
    (dict(widths=[31, 33]), S.SEGQ_ERR_SHAPE), (dict(widths=[-32, 64]), S.SEGQ_ERR_SHAPE),
    (dict(widths=[32, 8]), S.SEGQ_ERR_SHAPE), (dict(widths=[64, 64]), S.SEGQ_ERR_SHAPE),
    (dict(style=2), S.SEGQ_ERR_SHAPE), (dict(norm=0, qg=A["qg"]), S.SEGQ_ERR_SHAPE),
    (dict(kg=A["kg"]), S.SEGQ_ERR_NULL), (dict(k_out=A["k_out"]), S.SEGQ_ERR_NULL),
    (dict(eps=0.0), S.SEGQ_ERR_SHAPE), (dict(qg=A["qg"] + 4), S.SEGQ_ERR_ALIGN),
    (dict(q=None), S.SEGQ_ERR_NULL), (dict(q_out=None), S.SEGQ_ERR_NULL),
    (dict(qs=0), S.SEGQ_ERR_NULL), (dict(k=A["k"], k_out=None), S.SEGQ_ERR_NULL),
    (dict(q=A["q"] + 8), S.SEGQ_ERR_ALIGN), (dict(qs=(2560, 260, 64)), S.SEGQ_ERR_ALIGN),
    (dict(qs=(2560, -256, 64)), S.SEGQ_ERR_SHAPE), (dict(pos=None), S.SEGQ_ERR_NULL),
    (dict(pos=A["pos"] + 2), S.SEGQ_ERR_ALIGN), (dict(freq=None), S.SEGQ_ERR_NULL),
    (dict(freq=A["freq"] + 4), S.SEGQ_ERR_ALIGN), (dict(per=19), S.SEGQ_ERR_SHAPE),
    (dict(qos=(0, 256, 64)), S.SEGQ_ERR_SHAPE), (dict(qos=(2560, 256, 56)), S.SEGQ_ERR_SHAPE),
    (dict(qos=(2560, 248, 64)), S.SEGQ_ERR_SHAPE),
    (dict(q_out=A["q"] + 16), S.SEGQ_ERR_SHAPE), (dict(q_out=A["q"], qos=(5120, 512, 64)), S.SEGQ_ERR_SHAPE),
    (dict(k=A["k"], k_out=A["q_out"] + 10224), S.SEGQ_ERR_SHAPE), (dict(k=A["k"], q_out=A["k"]), S.SEGQ_ERR_SHAPE),
    (dict(q_out=A["pos"] + 64), S.SEGQ_ERR_SHAPE), (dict(q_out=A["freq"] - 10240 + 16), S.SEGQ_ERR_SHAPE),
    (dict(qg=A["qg"], q_out=A["qg"] + 240), S.SEGQ_ERR_SHAPE),
    # in place inside one matrix, but k begins inside q
    (dict(q_out=A["q"], qs=(7680, 768, 64), qos=(7680, 768, 64), k=A["q"] + 384, k_out=A["q"] + 384,
          ks=(7680, 768, 64), kos=(7680, 768, 64)), S.SEGQ_ERR_SHAPE),
])
def test_rotary_refusals(kw, status):
    assert rotary(**kw) == status, S.segquant_last_error()
    assert S.segquant_last_error() != ""


@pytest.mark.parametrize("kw", [
    dict(), dict(q_out=A["q"]), dict(k=A["k"], per=20), dict(norm=0, eps=0.0),
    dict(widths=[0, 0], freq=None), dict(qos=(2560, 64, 640)), dict(qs=(0, 0, 0)),
    dict(q_out=A["q"], qs=(7680, 768, 64), qos=(7680, 768, 64), k=A["q"] + 512, k_out=A["q"] + 512,
         ks=(7680, 768, 64), kos=(7680, 768, 64)),
    # the same with samples further apart than their tokens reach
    dict(q_out=A["q"], qs=(9216, 768, 64), qos=(9216, 768, 64), k=A["q"] + 512, k_out=A["q"] + 512,
         ks=(9216, 768, 64), kos=(9216, 768, 64)),
    dict(k=A["k"], k_out=A["q_out"] + 10240),
    # strides of a single sample, token and head do not count
    dict(B=1, L=1, Hq=1, qs=(3, 5, 7), qos=(-1, 0, 9)),
])
def test_rotary_calls_that_reach_the_launch(kw):
    assert rotary(**kw) == S.SEGQ_ERR_HIP, S.segquant_last_error()


def test_every_overlap_of_q_and_k_in_one_buffer_is_found():
    """q and k in place in one matrix at random strides, against sets of elements."""
    rng = random.Random(5)
    both = [0, 0]
    for _ in range(1500):
        B, L, Hq, Hk, D = rng.randint(1, 3), rng.randint(1, 5), rng.randint(1, 3), rng.randint(1, 3), 8
        row = 8 * rng.randint(max(Hq, Hk), 8)
        sample = L * row + 8 * rng.choice([0, 0, 1, 5, 20])
        at = 8 * rng.randint(-B * sample // 8, B * sample // 8)

        def cells(start, H):
            return {start + b * sample + l * row + 8 * h
                    for b in range(B) for l in range(L) for h in range(H)}
        want = bool(cells(0, Hq) & cells(at, Hk))
        p, st = A["q"] + (1 << 20), (sample, row, D)
        r = rotary(B=B, L=L, Hq=Hq, Hk=Hk, D=D, q=p, q_out=p, k=p + 2 * at, k_out=p + 2 * at, qs=st,
                   qos=st, ks=st, kos=st, widths=[0])
        assert (r == S.SEGQ_ERR_SHAPE) == want, (B, L, Hq, Hk, row, sample, at, S.segquant_last_error())
        both[want] += 1
    assert min(both) > 200


@pytest.mark.parametrize("B,L", [(1 << 28, 2), (2, 1 << 28)])
def test_overlap_of_many_samples_or_tokens_is_found_at_once(B, L):
    """Two columns of one matrix whose rows are not evenly spaced: the two share
    only bytes of the last sample and token, or none, and the host says so
    without a walk over all of them."""
    n, far = max(B, L), 24 * max(B, L) + 8  # elements between the two long runs
    st = (24, far, 8) if B == n else (far, 24, 8)
    at = 1 << 44
    end = 2 * (far + 24 * (n - 1))  # bytes from the first row to the last
    began = time.perf_counter()
    for off, status in [(-end, S.SEGQ_ERR_SHAPE), (-end - 16, S.SEGQ_ERR_HIP),
                        (16, S.SEGQ_ERR_HIP), (end, S.SEGQ_ERR_SHAPE)]:
        got = rotary(B=B, L=L, D=8, Hq=1, Hk=1, widths=[0], q=at, q_out=at, k=at + off,
                     k_out=at + off, qs=st, qos=st, ks=st, kos=st)
        assert got == status, (off, S.segquant_last_error())
    assert time.perf_counter() - began < 5.0


def test_frequencies():
    f = S.segquant_rotary_frequencies([16, 0, 48], 1000.0)
    want = [1000.0 ** (-2 * j / 16) for j in range(8)] + [1000.0 ** (-2 * j / 48) for j in range(24)]
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor(want, dtype=torch.float64),
                                                       rtol=1e-15, atol=0)
    assert S.segquant_rotary_frequencies([0]).numel() == 0
    for widths, theta in (([15, 1], 1e4), ([8], 1e4), ([16], 0.0), ([16], float("inf")),
                          ([16] * 9, 1e4)):
        with pytest.raises(S.SegQuantError):
            S.segquant_rotary_frequencies(widths, theta)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(n):
    return torch.zeros(n, dtype=torch.uint8)


W = (u8(1024), u8(256))


@pytest.mark.parametrize("fn,text", [
    (lambda: S.segquant_quantize_mxfp4(torch.zeros(4, 64)), "bfloat16"),
    (lambda: S.segquant_quantize_mxfp4(bf(4, 60)), "64"),
    (lambda: S.segquant_quantize_mxfp4(bf(4, 64), out=(u8(512), u8(256))), "codes"),
    (lambda: S.segquant_quantize_mxfp4(bf(64, 4).t()), "unit stride"),
    (lambda: S.segquant_quantize_mxfp4(bf(4, 64)), "on a GPU"),
    (lambda: S.segquant_quantize_weight_mxfp4(bf(64, 16)), "float32"),
    (lambda: S.segquant_unpack_mxfp4(W, 4, 128), "codes|scales|on a GPU"),
    (lambda: S.segquant_gemm_mxfp4(None, W, 16), "exactly one"),
    (lambda: S.segquant_gemm_mxfp4(bf(4, 64), W, 16, xq=W), "exactly one"),
    (lambda: S.segquant_gemm_mxfp4(None, W, 16, xq=W), "required"),
    (lambda: S.segquant_gemm_mxfp4(bf(4, 64), W, 16, K=128), "with M"),
    (lambda: S.segquant_gemm_mxfp4(bf(4, 64), W, 32), "w codes"),
    (lambda: S.segquant_gemm_mxfp4(bf(4, 64), W, 16, out=bf(4, 32)), "out"),
    (lambda: S.segquant_gemm_mxfp4(bf(4, 64), (W[0], u8(512)[::2]), 16), "contiguous"),
    (lambda: S.segquant_gemm_mxfp4(bf(4, 64), W, 16), "on a GPU"),
    (lambda: S.segquant_rmsnorm_quantize(bf(1, 4, 64), x_out=True), r"\[M\]\[K\]"),
    (lambda: S.segquant_rmsnorm_quantize(bf(4, 64), gamma=bf(64), x_out=True), "gamma"),
    (lambda: S.segquant_rmsnorm_quantize(bf(4, 64), mx_out=(u8(4), u8(4))), "mx_out codes"),
    (lambda: S.segquant_rmsnorm_quantize(bf(4, 60), mx_out=True), "64"),
    (lambda: S.segquant_rmsnorm_quantize(bf(4, 64), branch=bf(4, 32), x_out=True), "branch"),
    (lambda: S.segquant_rmsnorm_quantize(bf(4, 64), x_out=True), "on a GPU"),
])
def test_binding_refusals(fn, text):
    with pytest.raises(ValueError, match=text):
        fn()


@pytest.mark.parametrize("kw,text", [
    (dict(q=bf(2, 10, 256)), r"\[heads\]"), (dict(q=torch.zeros(2, 10, 4, 64)), "bfloat16"),
    (dict(k=bf(2, 9, 2, 64)), "k must be"), (dict(k=bf(2, 10, 64)), "k must be"),
    (dict(k_gamma=torch.zeros(64)), "without k"), (dict(q_gamma=torch.zeros(32)), "q_gamma"),
    (dict(positions=torch.zeros(10, 2)), "positions"), (dict(positions=torch.zeros(3, 10, 2, dtype=torch.int32)), "positions"),
    (dict(positions=torch.zeros(10, 3, dtype=torch.int32)[:, :2]), "contiguous"),
    (dict(freq=torch.zeros(32)), "freq"), (dict(freq=torch.zeros(16, dtype=torch.float64)), "freq"),
    (dict(q=bf(2, 10, 64, 4).transpose(2, 3)), "unit stride"), (dict(q_out=bf(2, 10, 4, 32)), "q_out"),
    (dict(), "on a GPU"),
])
def test_rotary_binding_refusals(kw, text):
    args = dict(q=bf(2, 10, 4, 64), k=None, positions=torch.zeros(10, 2, dtype=torch.int32),
                freq=torch.zeros(32, dtype=torch.float64), widths=[32, 32])
    args.update(kw)
    with pytest.raises(ValueError, match=text):
        S.segquant_qk_rotary(**args)
