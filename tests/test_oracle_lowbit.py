"""Pins of the low-bit and norm oracle (CPU): the code tables and ties by hand, the
scale rule at its borders, storage round trips, and the norm's gradient against
central differences."""
import numpy as np
import pytest

from oracle import lowbit as ol


def test_code_tables_and_ties():
    # e4m3 has 127 finite magnitudes up to 448, the smallest 2^-9; e2m1 ties go to the even code
    assert len(ol.E4M3) == 127 and ol.E4M3[-1] == 448.0 and ol.E4M3[1] == 2.0 ** -9
    assert np.all(np.diff(ol.E4M3) > 0)
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 9.0])
    np.testing.assert_array_equal(ol.E2M1[ol.round_to_grid(v, ol.E2M1)],
                                  [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0])
    v = np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 440.0])  # steps of 2, 2^-9 and 32
    np.testing.assert_array_equal(ol.E4M3[ol.round_to_grid(v, ol.E4M3)],
                                  [16.0, 20.0, 0.0, 2.0 ** -8, 448.0])


@pytest.mark.parametrize("fmt,top", [("mxfp4", 6.0), ("mxfp8", 448.0)])
def test_scale_is_the_least_that_fits(fmt, top):
    for amax, E in ((top, 0), (np.nextafter(top, 1e9), 1), (top / 2, -1),
                    (top * 2.0 ** 90, 90), (top * 2.0 ** -127, -127), (1e-44, -127), (0.0, -127)):
        x = np.zeros((1, 32))
        x[0, 5] = -amax
        _, s = ol.mx_encode(x, fmt)
        assert s[0, 0] == E + 127, (amax, E)


@pytest.mark.parametrize("fmt,half", [("mxfp4", 0.25), ("mxfp8", 2.0 ** -4)])
def test_storage_round_trip(fmt, half):
    g = np.random.default_rng(3)
    x = g.standard_normal((131, 200)) * np.exp(g.standard_normal((131, 1)))
    codes, scales = ol.mx_encode(x, fmt)
    back = ol.mx_load(*ol.mx_store(codes, scales, fmt), 131, 200, fmt)
    unit = np.repeat(2.0 ** (scales.astype(float) - 127), 32, -1)[:, :200]
    floor = 0.25 if fmt == "mxfp4" else 2.0 ** -10
    assert np.all(np.abs(back - x) <= np.maximum(half * np.abs(x), floor * unit))


def test_nonfinite_blocks_and_rows():
    x = np.ones((1, 96))
    x[0, 40], x[0, 70] = np.nan, np.inf
    codes, scales = ol.mx_encode(x, "mxfp8")
    assert list(scales[0]) == [127 - 8, 255, 255, 0]
    back = ol.mx_load(*ol.mx_store(codes, scales, "mxfp8"), 1, 96, "mxfp8")
    assert np.all(back[0, :32] == 1) and np.all(np.isnan(back[0, 32:]))


def test_norm_gradient_against_differences():
    g = np.random.default_rng(5)
    r, w, dy, dres = (g.standard_normal(s) for s in ((3, 7), 7, (3, 7), (3, 7)))
    eps = 0.1  # large enough to matter
    loss = lambda r, w: (ol.rmsnorm(r, w, eps)[0] * dy).sum() + (r * dres).sum()  # noqa: E731
    dr, dw = ol.rmsnorm_bwd(dy, r, w, ol.rmsnorm(r, w, eps)[1], dres)
    h = 1e-6  # central differences: h^2 truncation, 1e-16 / h rounding
    for i in np.ndindex(3, 7):
        e = np.zeros((3, 7))
        e[i] = h
        assert abs((loss(r + e, w) - loss(r - e, w)) / (2 * h) - dr[i]) < 1e-7
    for i in range(7):
        e = np.zeros(7)
        e[i] = h
        assert abs((loss(r, w + e) - loss(r, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_state_form():
    g = np.random.default_rng(6)
    h = g.standard_normal((4, 5, 64)) * np.exp(2 * g.standard_normal((4, 5, 1)))
    h[1, 2] = 0.0
    h[2, 3] *= 1e-40
    codes, s = ol.state_encode(h)
    back = ol.state_decode(codes, s)
    assert s[1, 2] == 0 and s[2, 3] == 0 and not back[2, 3].any()
    big = s > 0
    assert np.all((np.abs(back - h) <= np.maximum(2.0 ** -4 * np.abs(h), 2.0 ** -10 * s[..., None])
                   * (1 + 1e-12))[big])
    # a decay alone moves only the scale
    c2, s2 = ol.state_encode(0.9 * back)
    np.testing.assert_array_equal(c2, codes)
    np.testing.assert_allclose(s2[big], 0.9 * s[big], rtol=1e-12)
