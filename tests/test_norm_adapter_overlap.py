"""Outputs that share memory with other operands of segquant_groupnorm_quantize,
segquant_adanorm_quantize and segquant_adapter_add: refused wherever a byte is
shared, accepted side by side, and found in a few steps however many rows."""
import random
import time

import pytest

import segmented_dual_scale_amd as S
from test_abi import _gpu_present
from test_norm_adapter_abi import FAKE2, adanorm, adapter, groupnorm

pytestmark = pytest.mark.skipif(_gpu_present(), reason="fake device pointers: CPU-only tests")

FAR = 1 << 50


def refused(status):
    """The call was refused for an overlap (False: it went on to the launch)."""
    assert status in (S.SEGQ_ERR_SHAPE, S.SEGQ_ERR_HIP), S.segquant_last_error()
    assert (status == S.SEGQ_ERR_SHAPE) == ("overlap" in S.segquant_last_error())
    return status == S.SEGQ_ERR_SHAPE


def elements(at, ld, width, rows):
    return {at + i * ld + k for i in range(rows) for k in range(0, width, 8)}


def test_any_shared_element_is_found():
    rng = random.Random(1)
    both = [0, 0]
    for _ in range(3000):
        M, N = rng.randint(1, 12), 16 * rng.randint(1, 5)
        ld_x, ld_y = 64 + 8 * rng.randint(0, 30), N + 8 * rng.randint(0, 40)
        if rng.random() < 0.3:
            ld_x = ld_y = max(ld_x, ld_y)
        elif rng.random() < 0.3:
            ld_x = rng.randint(1, 3) * max(ld_y, 64)
        at = 8 * rng.randint(-M * ld_x // 8 - 2, M * ld_y // 8 + 2)
        want = bool(elements(at, ld_x, 64, M) & elements(0, ld_y, N, M))
        base = FAKE2 << 8
        got = refused(adapter(M=M, N=N, x=base + 2 * at, ld_x=ld_x, y=base, ld_y=ld_y, base=None,
                              row_offset=FAR, ids=FAR, rank_of=FAR, a=FAR, b=FAR, alpha=FAR))
        assert got == want, (M, N, ld_x, ld_y, at)
        both[want] += 1
    assert min(both) > 500


def test_many_interleaved_rows_take_no_time():
    """Rows of one matrix in every second gap between the other's."""
    start = time.perf_counter()
    M = 1 << 27
    kw = dict(M=M, x=FAKE2 + 128, ld_x=2048, y=FAKE2, ld_y=1024, base=None, work=FAR,
              work_bytes=1 << 45)
    assert not refused(adapter(**kw))
    assert refused(adapter(**{**kw, "x": FAKE2 + 128, "ld_x": 2048 + 8}))
    kw = dict(M=(1 << 31) - 1, h=FAKE2, ld_h=1 << 40, branch=None, gate=None, h_out=None, q=None,
              scale=None, shift=None, x=FAKE2 + 128, ld_xo=3 << 40, row_offset=None, n_req=1)
    assert not refused(adanorm(**kw))
    assert refused(adanorm(**{**kw, "ld_xo": (3 << 40) - 8}))
    # distances of rows are the first one's plus multiples of 200: 64, or 144 - 200
    kw = dict(B=1, Px=(1 << 31) - 1, z=FAKE2, ld_z=1000, q=None, ld_xo=1200, work=FAR,
              work_bytes=1 << 45)
    assert not refused(groupnorm(**kw, x=FAKE2 + 2 * 64))
    assert refused(groupnorm(**kw, x=FAKE2 + 2 * 144))
    assert time.perf_counter() - start < 1.0
