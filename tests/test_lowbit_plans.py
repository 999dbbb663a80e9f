"""What the low-bit and norm entry points decide on the host, from sizes alone (CPU)."""
import ctypes

import pytest
import torch

import selective_state_space_m3ssd_b200 as m3


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
