"""The gated linear recurrence cut into parts of many runs, against the fp64 oracle: the rings of copies
of the parts' maps and of the walk wrap, forward and backward.  Tolerances as in test_gpu_glr.py; the
oracle is given some of the channels, which do not depend on one another.

26 items (sequences x groups of 64 channels) leave 11 CTAs, 88 parts, a sequence on 148 SMs: of 5000
tokens 64 each in bf16, eight runs, four for each of the two warps that make a part's map backward; of
fp32 60, 15 runs.
"""
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import layer as ly
from tests.gpu_util import np64
from tests.test_gpu_glr import FWD, call, check, check_bwd, fwd_tolerance, gpu, host, make

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
PER_CHANNEL = ("x", "r", "i", "dy", "rate", "bias_r", "bias_i", "h0", "dhT")


def run(d, channels, grad_dtype):
    c = gpu(d)
    y, hT = call(m3.glr_fwd, c)
    got = call(m3.glr_bwd, c, y, c["dy"], dhT=c["dhT"], grad_dtype=grad_dtype)
    some = {k: v[..., channels] if k in PER_CHANNEL else v for k, v in d.items()}
    h = host(some)
    ry, rT = ly.glr_fwd(**{k: h[k] for k in FWD if k in h})
    ty, tT = fwd_tolerance(h, ry, rT)
    check(y[..., channels], ry, ty, y.dtype, "y")
    check(hT[..., channels], rT, tT, torch.float32, "hT")
    check_bwd(some, np64(y[..., channels]), {k: v[..., channels] for k, v in got.items()}, grad_dtype)
    assert all(torch.isfinite(v).all() for v in got.values())


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_runs_a_part(dtype):
    run(make(13, 5000, 65, dtype, seed=1), [0, 33, 64], torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_resets_and_ends_in_many_runs_a_part(dtype):
    lengths = [5000, 0, 1, 4999, 64, 63, 2500, 129, 4800, 4001, 3333, 777, 4937]
    run(make(13, 5000, 72, dtype, seed=2, reset=0.004, lengths=lengths), [7, 63, 71], dtype)


# groups of 64 channels, the last one whole or not, rows in 16-byte, 4-byte and element copies
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [768, 769, 770])
def test_two_sequences_of_many_channels(D, dtype):
    run(make(2, 4096, D, dtype, seed=D, reset=0.002), [0, 1, 63, 64, 400, 767, D - 1], dtype)
