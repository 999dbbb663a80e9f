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


@pytest.mark.parametrize("b,L,kw", [(3, 70, {}), (1, 1100, {}), (3, 70, {"reset": 0.2})])
def test_rates_that_leave_nothing_of_the_state(b, L, kw):
    """Rates from where no gate leaves any of the state, a = 0, up to infinity: y is iota x, g is dy
    (dhT joins at the last token), nothing of the gradient reaches r, the rate or h0."""
    D = 64
    d = make(b, L, D, torch.float32, seed=4, bias=False, **kw)
    d["rate"] = torch.tensor([1e21, 1e25, 1e30, 1e37, 2.9e37, 1e38, 3e38, float("inf")]).repeat(D // 8)
    d["r"][:, ::3] = -float("inf")
    c = gpu(d)
    y, hT = call(m3.glr_fwd, c)
    h = host(d)
    iota = ly.sigmoid(h["i"])
    ry = iota * h["x"]
    rel = 2 * (3 * abs(h["i"]) + 16 + 40 + 4) * 2.0 ** -24  # u's bound, and two products
    check(y, ry, rel * abs(ry), torch.float32, "y")
    assert torch.equal(hT, y[:, -1])
    got = call(m3.glr_bwd, c, y, c["dy"], dhT=c["dhT"])
    g = h["dy"].copy()
    g[:, -1] += h["dhT"]
    check(got["dx"], g * iota, rel * abs(g * iota), torch.float32, "dx")
    di = g * ry * (1 - iota)
    check(got["di"], di, 2 * rel * abs(di), torch.float32, "di")
    for k in ("dr", "drate", "dbias_r", "dh0"):
        assert (got[k] == 0).all(), k
    y1, h1 = m3.glr_step(c["h0"].clone(), c["x"][:, 0], c["r"][:, 0], c["i"][:, 0], c["rate"])
    assert torch.equal(y1, y[:, 0]) and torch.equal(h1, y1)
