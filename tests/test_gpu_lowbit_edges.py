"""Edges of the low-bit and norm operators: widths below one access, rows that are not finite,
waits that are given up, arguments of another device or layout."""
import numpy as np
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import lowbit as ol
from tests import test_gpu_norm as norm
from tests.test_gpu_norm import BF16, F32, FP, cu, inputs, np64, summed

pytestmark = pytest.mark.gpu

# rows narrower than an access of eight elements: the tensor's end is several rows away from
# the first access that would pass it
NARROW = [(rows, d) for d in range(1, 8) for rows in (2, 3, 10, 1001)]


@pytest.mark.parametrize("rows,d", NARROW)
@pytest.mark.parametrize("dtype,res", [(F32, None), (BF16, None), (BF16, F32), (BF16, BF16),
                                       (F32, F32), (F32, BF16)])
def test_narrow_rows_forward(rows, d, dtype, res):
    norm.test_forward(rows, d, dtype, res)


@pytest.mark.parametrize("rows,d", NARROW)
@pytest.mark.parametrize("dtype,res", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("dres", [False, True])
def test_narrow_rows_backward(rows, d, dtype, res, dres):
    norm.test_backward(rows, d, dtype, res, dres)


@pytest.mark.parametrize("d", [1, 2, 3, 5, 7, 9])
def test_what_follows_a_narrow_tensor_is_left_out_and_left(d):
    """NaN behind every tensor of the call: outputs as without them, and the NaN still there."""
    rows = 11
    x, r, w = inputs(rows, d, F32, F32)
    y0, out0, rstd = m3.add_rmsnorm(*cu(x, w), residual=r.cuda(), want_rstd=True)
    wide = [torch.full((rows + 9, d), float("nan"), device="cuda") for _ in range(4)]
    wide[0][:rows], wide[1][:rows] = x.cuda(), r.cuda()
    m3.add_rmsnorm(wide[0][:rows], w.cuda(), residual=wide[1][:rows], y=wide[2][:rows],
                   residual_out=wide[3][:rows])
    assert torch.equal(wide[2][:rows], y0) and torch.equal(wide[3][:rows], out0)
    assert all(torch.isnan(t[rows:]).all() for t in wide)
    dr0, dw0 = m3.add_rmsnorm_bwd(x.cuda(), out0, w.cuda(), rstd, dres=r.cuda())
    dr = torch.full((rows + 9, d), float("nan"), device="cuda")
    _, dw = m3.add_rmsnorm_bwd(wide[0][:rows], wide[3][:rows], w.cuda(), rstd, dres=wide[1][:rows],
                               dr=dr[:rows])
    assert torch.equal(dr[:rows], dr0) and torch.equal(dw, dw0)
    assert torch.isnan(dr[rows:]).all()
