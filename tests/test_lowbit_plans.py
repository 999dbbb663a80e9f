"""What the low-bit and norm entry points decide on the host, from sizes alone (CPU)."""
import ctypes
import math
import random

import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from tests import test_gpu_lowbit_edges, test_gpu_mx


@pytest.fixture(scope="module")
def lib():
    return m3.load()


def whole(lib, rows, d, row, column):
    n, out = m3.NormDims(rows, d, m3.F32, m3.F32, 1e-6, 0), ctypes.c_int32(-1)
    assert lib.m3ssd_test_norm_access(ctypes.byref(n), row, column, ctypes.byref(out)) == m3.OK
    return out.value


@pytest.mark.parametrize("d", [*range(1, 18), 33, 1049, 16377])
def test_norm_accesses_stay_inside_the_tensor(lib, d):
    """Every access of eight elements that a row of an odd width lies in: whole only where all
    eight are the tensor's, and whole wherever they are."""
    for rows in (1, 2, 3, 4, 7, 8, 9, 10, 17, 25):
        for row in range(rows):
            shift = row * d % 8
            for c in range(-shift, d, 8):
                first = row * d + c
                assert first >= 0
                assert whole(lib, rows, d, row, c) == (first + 8 <= rows * d), (rows, row, c)


def test_norm_access_arguments(lib):
    n, out = ctypes.byref(m3.NormDims(4, 9, m3.F32, m3.F32, 1e-6, 0)), ctypes.c_int32()
    f, r = lib.m3ssd_test_norm_access, ctypes.byref(out)
    for row, column in ((-1, 0), (4, 0), (0, -8), (0, 9)):
        assert f(n, row, column, r) == m3.ERR_INVALID_ARG
    assert f(n, 0, 0, None) == m3.ERR_INVALID_ARG
    assert f(ctypes.byref(m3.NormDims(4, 0, 0, 0, 0, 0)), 0, 0, r) == m3.ERR_INVALID_ARG


def test_a_workspace_is_memory_of_the_call_s_device():
    dev = torch.device("cuda", 0)
    assert m3._workspace(None, 0, dev) == (None, None, 0)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        m3._workspace(torch.empty(64, dtype=torch.uint8), 64, dev)
    # the binding refuses before anything is launched
    with pytest.raises(ValueError, match="workspace must be"):
        m3._workspace(torch.empty(64, dtype=torch.uint8, device="meta"), 64, dev)


def shapes_of(test):
    return next(m.args[1] for m in test.pytestmark
                if m.name == "parametrize" and m.args[0] == "M,N,K")


def test_every_plan_of_the_product_is_tested():
    """The plans that shapes of every size take on 148 SMs are those of the GPU tests' shapes:
    every tile whole and in each of its parts, K over each size of cluster."""
    shapes = [s for t in (test_gpu_mx.test_gemm_matches_fp64, test_gpu_mx.test_gemm_parts_of_tiles,
                          test_gpu_mx.test_gemm_many_tiles, test_gpu_mx.test_gemm_long_k,
                          test_gpu_lowbit_edges.test_gemm_plans) for s in shapes_of(t)]
    tested = {fmt: {m3.gemm_mx_plan(*s, fmt, 148) for s in shapes} for fmt in ("mxfp4", "mxfp8")}
    whole = {(0, bn, part) for bn in (256, 192, 128) for part in (0, 64, 128) if part < bn}
    over_k = {(s, 16, 0) for s in (1, 2, 4, 8)} | {(s, 128, 0) for s in (2, 4, 8)}
    rng = random.Random(7)
    size = lambda a, b: round(math.exp(rng.uniform(math.log(a), math.log(b))))  # noqa: E731
    for fmt, plans in tested.items():
        assert plans == (whole | over_k) - {(0, 128, 128)}, plans ^ (whole | over_k)
        for _ in range(20000):
            s = size(1, 60000), size(1, 20000), size(1, 16384)
            assert m3.gemm_mx_plan(*s, fmt, 148) in plans, s


def test_the_plan_s_arguments(lib):
    out = [ctypes.byref(ctypes.c_int32()) for _ in range(3)]
    f = lib.m3ssd_test_gemm_mx_plan
    for bad in ((2, 1, 1, 1, 148), (0, 0, 1, 1, 148), (0, 1, 0, 1, 148), (0, 1, 1, 0, 148),
                (0, 1, 1, 1, 0)):
        assert f(*bad, *out) == m3.ERR_INVALID_ARG
    assert f(0, 1, 1, 1, 148, None, *out[1:]) == m3.ERR_INVALID_ARG
    assert f(0, 2 ** 31, 1, 1, 148, *out) == m3.ERR_UNSUPPORTED
