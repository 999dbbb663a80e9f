"""The gated linear recurrence where its gates are closed, against the fp64 oracle by value.

A gate below 2^-63 counts as that (include/m3ssd.h), so the oracle is given gates held at
sigma(-63 ln 2) = 2^-63 (1 - 2^-63).  The kernels hold the exponential there, which is a power of two,
so the tolerances of test_gpu_glr.py hold as they are.
"""
import math

import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import layer as ly
from tests.gpu_util import np64
from tests.test_gpu_glr import FWD, call, check, check_bwd, fwd_tolerance, gpu, host, make

pytestmark = pytest.mark.gpu
CLOSED = [-40.0, -50.0, -60.0, -70.0, -80.0, -88.0, -104.0, -300.0, -float("inf")]


def held(g, bias):
    """The gate's input in fp64 with the gate held at 2^-63."""
    bias = 0.0 if bias is None else bias.double()
    return torch.clamp(g.double() + bias, min=-63 * math.log(2)) - bias


# whole sequences, few sequences in parts, runs with resets, ends inside a run
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,L,D,kw", [(5, 100, 64, {}), (2, 64, 70, {"bias": False}), (1, 1100, 66, {}),
                                      (3, 100, 64, {"reset": 0.3}), (2, 90, 33, {"lengths": [85, 3]}),
                                      (1, 1300, 40, {"reset": 0.01, "lengths": [1203]})])
def test_closed_gates(b, L, D, kw, dtype):
    d = make(b, L, D, dtype, seed=L + D, **kw)
    g = torch.Generator().manual_seed(b)
    closed = torch.tensor(CLOSED)
    at = torch.randint(0, 2 * len(CLOSED), (b, L, D), generator=g)  # half of the gates are open
    d["r"] = torch.where(at < len(CLOSED), closed[at % len(CLOSED)], d["r"].float()).to(dtype)
    at = torch.randint(0, 4 * len(CLOSED), (b, L, D), generator=g)
    d["i"] = torch.where(at < len(CLOSED), closed[at % len(CLOSED)], d["i"].float()).to(dtype)
    ref = dict(d, r=held(d["r"], d["bias_r"]), i=held(d["i"], d["bias_i"]))
    h = host(ref)
    y, hT = ly.glr_fwd(**{k: h[k] for k in FWD if k in h})
    ty, tT = fwd_tolerance(h, y, hT)
    c = gpu(d)
    gy, gT = call(m3.glr_fwd, c)
    check(gy, y, ty, dtype, "y")
    check(gT, hT, tT, torch.float32, "hT")
    for grad in {torch.float32, dtype}:
        got = call(m3.glr_bwd, c, gy, c["dy"], dhT=c["dhT"], grad_dtype=grad)
        check_bwd(ref, np64(gy), got, grad)
