"""The binding of the norms and adapters on batches and operands at its edges,
without a GPU: what it accepts goes on to the check that operands are on one."""
import pytest
import torch

import segmented_dual_scale_amd as S


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("layout", [S.SEGQ_Q_SIGNED, S.SEGQ_Q_PLANES])
@pytest.mark.parametrize("given", [False, True])
def test_codes_of_no_rows(layout, given):
    shape = (0, 80) if layout == S.SEGQ_Q_SIGNED else (2, 0, 80)
    out = torch.zeros(shape, dtype=torch.int8) if given else None
    scales = torch.zeros(4, 1)
    with pytest.raises(ValueError, match="on a GPU"):
        S.segquant_adanorm_quantize(bf(0, 72), act_scales=scales, layout=layout, out=out)
    with pytest.raises(ValueError, match="on a GPU"):
        S.segquant_groupnorm_quantize(bf(0, 5, 72), 8, act_scales=scales, layout=layout, out=out)
    q, _, ld = S._codes_out(out, 0, 72, layout, torch.device("cpu"), torch.empty)
    assert q.shape == shape and ld == 80


@pytest.mark.parametrize("rows", [1, 3])
def test_planes_that_do_not_follow_each_other(rows):
    q = torch.zeros(2, 4, 64, dtype=torch.int8)[:, :rows]
    if rows == 1:  # a plane of one row: the planes' distance is the row's
        assert S._codes_out(q, 1, 64, S.SEGQ_Q_PLANES, q.device, torch.empty)[2] == 256
    else:
        with pytest.raises(ValueError, match="second plane"):
            S._codes_out(q, rows, 64, S.SEGQ_Q_PLANES, q.device, torch.empty)
