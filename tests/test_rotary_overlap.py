"""Which tensors of segquant_qk_rotary overlap, without a GPU: through the C ABI with
fake device addresses, against sets of elements."""
import ctypes
import random
import time

import numpy as np
import pytest

import segmented_dual_scale_amd as S
from test_abi import _gpu_present

pytestmark = pytest.mark.skipif(_gpu_present(), reason="fake device pointers: CPU-only tests")

I3 = ctypes.c_int64 * 3
Q, POS, FREQ = 1 << 40, 1 << 30, 1 << 31


def rotary(B, L, Hq, Hk, D, q, qs, q_out, qos, k=None, ks=None, k_out=None, kos=None):
    w = np.array([0], dtype=np.int32)
    st = [None if s is None else I3(*s) for s in (qs, qos, ks, kos)]
    return S.load_library().segquant_qk_rotary(B, L, D, q, Hq, st[0], q_out, st[1], k, Hk, st[2],
                                               k_out, st[3], 1, 1e-6, None, None, POS, 0, 1,
                                               w.ctypes.data, FREQ, 0, None)


def in_place(B, L, Hq, Hk, D, strides, at):
    """q and k in place, k `at` elements behind q."""
    k = Q + 2 * at
    return rotary(B, L, Hq, Hk, D, Q, strides, Q, strides, k, strides, k, strides)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("B,L,H,D,tokens", [(2, 10, 4, 64, 13), (3, 77, 24, 64, 80), (1, 9, 2, 128, 9)])
def test_q_and_k_of_each_head_side_by_side(B, L, H, D, tokens, heads_first):
    """[B][tokens][H][3][D], L of the tokens taken, or [B][H][tokens][3][D]: q, k and v share no
    element."""
    st = (tokens * H * 3 * D, 3 * D, tokens * 3 * D) if heads_first else (tokens * H * 3 * D, H * 3 * D, 3 * D)
    for at in (D, -D, 2 * D, 3 * D * H * L * 100 + D):
        assert in_place(B, L, H, H, D, st, at) == S.SEGQ_ERR_HIP, S.segquant_last_error()
    for at in (0, 8, D - 8, 3 * D, 3 * D + 8):
        if H * L > 2:
            assert in_place(B, L, H, H, D, st, at) == S.SEGQ_ERR_SHAPE


def test_every_overlap_of_q_and_k_with_heads_apart_is_found():
    rng = random.Random(11)
    both = [0, 0]
    for _ in range(3000):
        B, L, Hq, Hk, D = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3), rng.randint(1, 3), 8
        sizes = dict(b=B, l=L, h=max(Hq, Hk))
        stride, extent = {}, D  # nested in any order, with gaps
        for name in rng.sample("blh", 3):
            stride[name] = extent + 8 * rng.choice([0, 0, 1, 2, 7])
            extent = stride[name] * (sizes[name] - 1) + extent
        st = (stride["b"], stride["l"], stride["h"])
        at = 8 * rng.randint(-extent // 8, extent // 8)

        def cells(start, H):
            return {start + b * st[0] + l * st[1] + h * st[2]
                    for b in range(B) for l in range(L) for h in range(H)}
        want = bool(cells(0, Hq) & cells(at, Hk))
        got = in_place(B, L, Hq, Hk, D, st, at)
        assert (got == S.SEGQ_ERR_SHAPE) == want, (B, L, Hq, Hk, st, at, S.segquant_last_error())
        both[want] += 1
    assert min(both) > 300


def test_every_overlap_of_an_output_with_k():
    """Outputs of the same sample, token and head strides as k, which itself may have
    any strides, its own heads overlapping too."""
    rng = random.Random(12)
    both = [0, 0]
    for _ in range(3000):
        B, L, Hq, Hk, D = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3), rng.randint(1, 9), 8
        sizes = dict(b=B, l=L, h=Hq)
        stride, extent = {}, D
        for name in rng.sample("blh", 3):
            stride[name] = extent + 8 * rng.choice([0, 0, 1, 2, 7])
            extent = stride[name] * (sizes[name] - 1) + extent
        st = (stride["b"], stride["l"], stride["h"])
        reach = extent + 8 * 9 * 12
        at = 8 * rng.randint(-reach // 8, reach // 8)

        def cells(start, H):
            return {start + b * st[0] + l * st[1] + h * st[2]
                    for b in range(B) for l in range(L) for h in range(H)}
        want = bool(cells(0, Hq) & cells(at, Hk))
        far, dense = 1 << 50, (L * Hk * D, Hk * D, D)
        got = rotary(B, L, Hq, Hk, D, far, (L * Hq * D, Hq * D, D), Q, st, Q + 2 * at, st,
                     2 * far, dense)
        assert (got == S.SEGQ_ERR_SHAPE) == want, (B, L, Hq, Hk, st, at, S.segquant_last_error())
        both[want] += 1
    assert min(both) > 300


def test_overlap_of_many_elements_is_found_at_once():
    """2^30 heads of samples, tokens and heads, none evenly spaced."""
    n, H, D, h = 1 << 10, 1 << 9, 8, 24
    l = h * (H - 1) + 24  # the last head of a token leaves 16 elements
    b = l * (n - 1) + h * (H - 1) + 40
    end = b * (n - 1) + l * (n - 1) + h * (H - 1)
    began = time.perf_counter()
    for at, status in [(D, S.SEGQ_ERR_HIP), (2 * D, S.SEGQ_ERR_HIP), (end, S.SEGQ_ERR_SHAPE),
                       (-end, S.SEGQ_ERR_SHAPE), (end + D, S.SEGQ_ERR_HIP),
                       (b * 1000 + l * 999 + h * 511, S.SEGQ_ERR_SHAPE),
                       (b + l + h + D, S.SEGQ_ERR_HIP)]:
        assert in_place(n, n, H, H, D, (b, l, h), at) == status, (at, S.segquant_last_error())
    assert time.perf_counter() - began < 1.0
