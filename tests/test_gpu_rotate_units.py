"""The heads' norm with its rotation where a warp takes several units (blocks of a token's heads) and
several slots of heads in each, against the fp64 oracle: the ring of copies wraps, a unit goes from
queries to keys, the position of the next unit is read ahead.  Tolerances as in test_gpu_rotate.py.
"""
import pytest
import torch

from tests.test_gpu_rotate import BF, F32, bwd, check_bwd, check_fwd, fwd, gpu, make

pytestmark = pytest.mark.gpu


# tokens of more heads than all warps together take at once: a warp's next unit is of the same token
@pytest.mark.parametrize("rows,Hq,Hk,N,dtype", [(2, 16384, 0, 256, BF), (3, 40000, 0, 128, BF),
                                                (3, 9000, 6000, 256, F32), (2, 33000, 30000, 128, BF)])
def test_forward_of_more_heads_than_warps(rows, Hq, Hk, N, dtype):
    d = make(rows, Hq, Hk, N, N // 2, dtype, seed=rows + N)
    d["positions"] = torch.tensor([3000, -7, 40][:rows], dtype=torch.int32)
    check_fwd(d, fwd(gpu(d)))


@pytest.mark.parametrize("rows,Hq,Hk,N,dtype,grad", [(3, 20000, 0, 256, BF, BF), (5, 9000, 5300, 256, BF, F32),
                                                     (2, 12000, 7000, 128, F32, F32)])
def test_backward_of_more_heads_than_warps(rows, Hq, Hk, N, dtype, grad):
    d = make(rows, Hq, Hk, N, N // 2, dtype, seed=rows + N, up=dtype)
    d["positions"] = torch.tensor([3000, -7, 40, 901, 5][:rows], dtype=torch.int32)
    check_bwd(d, bwd(gpu(d), grad_dtype=grad), grad)


# tokens of a few slots each, several a warp: 9000 x (9 + 3) heads of 64 are three slots of queries and
# one of keys, in units of all four; 5000 x (5 + 2) of 128 the same; 6000 x 40 heads of 128 are 20 slots
MANY = [(9000, 9, 3, 64, 32), (5000, 5, 2, 128, 64), (6000, 32, 8, 128, 40), (7001, 3, 1, 250, 125)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,Hq,Hk,N,R", MANY)
def test_forward_of_many_tokens(rows, Hq, Hk, N, R, dtype):
    d = make(rows, Hq, Hk, N, R, dtype, seed=rows)
    check_fwd(d, fwd(gpu(d)))


@pytest.mark.parametrize("dtype,up,grad", [(BF, BF, BF), (BF, BF, F32), (BF, F32, BF), (BF, F32, F32),
                                           (F32, F32, F32)])
@pytest.mark.parametrize("rows,Hq,Hk,N,R", MANY[:2])
def test_backward_of_many_tokens(rows, Hq, Hk, N, R, dtype, up, grad):
    d = make(rows, Hq, Hk, N, R, dtype, seed=rows, up=up)
    check_bwd(d, bwd(gpu(d), grad_dtype=grad), grad)


def test_backward_of_many_slots():
    d = make(6000, 32, 8, 128, 40, BF, seed=6, up=BF)
    check_bwd(d, bwd(gpu(d), grad_dtype=BF), BF)


@pytest.mark.parametrize("rows,Hq,Hk", [(1, 1, 1), (700, 3, 2)])
def test_weights_gradients_do_not_depend_on_the_others_type(rows, Hq, Hk):
    """dq_w and dk_w are fp32 whatever dq's type is: the same angles, and at ten values a head, which
    either type moves in pairs, the same order of the sums, so the same bits."""
    d = gpu(make(rows, Hq, Hk, 10, 5, BF, seed=8, up=BF))
    a, b = bwd(d, grad_dtype=BF), bwd(d, grad_dtype=F32)
    for n in ("dq_w", "dk_w"):
        assert torch.equal(a[n], b[n])
    assert torch.equal(a["dq"], b["dq"].to(BF)) and torch.equal(a["dk"], b["dk"].to(BF))
