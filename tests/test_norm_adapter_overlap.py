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


# every operand in 4 MiB of its own
A = {name: 0x1000000 + (i << 22) for i, name in enumerate(
    ["z", "gamma", "beta", "scale", "shift", "act", "q", "x", "work", "h", "branch", "gate", "h_out",
     "row_offset", "base", "ids", "rank_of", "a", "b", "alpha", "y"])}
GN = dict({k: A[k] for k in ("z", "gamma", "beta", "scale", "shift", "act", "q", "x")}, B=2, Px=4)
GN2 = dict(GN, Px=10000, work=A["work"], work_bytes=1 << 22)  # two launches
ADA = {k: A[k] for k in ("h", "branch", "gate", "scale", "shift", "gamma", "beta", "act", "q", "x",
                         "h_out", "row_offset")}
ADP = {k: A[k] for k in ("x", "row_offset", "ids", "rank_of", "a", "b", "alpha", "base", "y")}
ADP2 = dict(ADP, M=64, rank=80, work=A["work"], work_bytes=1 << 22)


def test_operands_apart_go_on_to_the_launch():
    assert 0 < S.segquant_groupnorm_workspace_bytes(2, 10000, 64, 8) < 1 << 22
    assert 0 < S.segquant_adapter_workspace_bytes(64, 64, 64, 2, 80) < 1 << 22
    for call, kw in ((groupnorm, GN), (groupnorm, GN2), (adanorm, ADA), (adapter, ADP),
                     (adapter, ADP2)):
        assert not refused(call(**kw))
        assert not refused(call(**kw, layout=1)) if call is not adapter else True


@pytest.mark.parametrize("call,kw,out,operand,last", [
    # the operand's last byte or more before its end: the output starts there
    *[(groupnorm, GN, out, name, size - 16) for out in ("q", "x") for name, size in (
        ("gamma", 256), ("beta", 256), ("scale", 256), ("shift", 256))],
    (groupnorm, GN, "q", "act", 0), (groupnorm, GN, "x", "act", 0),
    (groupnorm, GN, "q", "z", 0), (groupnorm, GN, "q", "z", 8 * 128 - 16),
    (groupnorm, GN, "q", "x", 0), (groupnorm, GN, "x", "q", 8 * 64 - 16),
    *[(groupnorm, GN2, "work", name, 0) for name in ("z", "gamma", "beta", "scale", "shift", "act",
                                                     "q", "x")],
    *[(adanorm, ADA, out, name, size - 16) for out in ("q", "x", "h_out") for name, size in (
        ("gamma", 256), ("beta", 256), ("scale", 256), ("shift", 256), ("gate", 256))],
    *[(adanorm, ADA, out, "row_offset", 0) for out in ("q", "x", "h_out")],
    *[(adanorm, ADA, out, "act", 0) for out in ("q", "x", "h_out")],
    *[(adanorm, ADA, "q", name, 8 * 128 - 16) for name in ("h", "branch", "x", "h_out")],
    (adanorm, ADA, "x", "h_out", 0),
    *[(adapter, ADP, "y", name, size - 16) for name, size in (
        ("a", 2 * 16 * 64 * 2), ("b", 2 * 64 * 16 * 2))],
    *[(adapter, ADP, "y", name, 0) for name in ("row_offset", "ids", "rank_of", "alpha")],
    *[(adapter, ADP2, "work", name, 0) for name in ("x", "row_offset", "ids", "rank_of", "alpha",
                                                    "a", "b", "base", "y")],
])
def test_an_output_on_another_operand(call, kw, out, operand, last):
    kw = {**kw, out: kw[operand] + last}
    assert refused(call(**kw))
    if out != "work" and last > 0:  # one 16-byte step on, it stands behind it
        assert not refused(call(**{**kw, out: kw[out] + 16}))


def test_the_second_plane_of_codes_counts():
    kw = dict(GN, q=A["z"] - 8 * 64)  # the first plane ends where z starts
    assert not refused(groupnorm(**kw, layout=0))
    assert refused(groupnorm(**kw, layout=1))


def test_outputs_side_by_side_with_inputs():
    # codes in the padding of z's rows, x_out beside scale and shift
    assert not refused(groupnorm(**dict(GN, ld_z=128, q=A["z"] + 128, ld_q=256)))
    assert not refused(groupnorm(**dict(GN, scale=A["x"] + 128, ld_xo=128, ld_mod=128)))
    # in place
    assert not refused(groupnorm(**dict(GN, x=A["z"])))
    assert not refused(adanorm(**dict(ADA, h_out=A["h"])))
    assert not refused(adanorm(**dict(ADA, h_out=A["branch"])))
    assert not refused(adapter(**dict(ADP, y=A["base"])))


def test_a_workspace_that_the_call_does_not_use_may_stand_anywhere():
    assert S.segquant_groupnorm_workspace_bytes(2, 4, 64, 8) == 0
    for name in ("z", "x", "q", "scale"):
        assert not refused(groupnorm(**GN, work=A[name] + 64, work_bytes=1 << 20))
    assert S.segquant_adapter_workspace_bytes(8, 64, 64, 2, 16) == 0
    for name in ("x", "y", "a", "base"):
        assert not refused(adapter(**ADP, work=A[name] + 64, work_bytes=1 << 20))
