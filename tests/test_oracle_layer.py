"""The oracle of the operators around the scan, pinned without its own code: closed forms,
differences, and what must not change a result (no GPU)."""
import numpy as np
import pytest

from oracle import layer as ly


def inputs(b=2, L=9, D=3, seed=0):
    g = np.random.default_rng(seed)
    f = lambda *s: g.standard_normal(s)  # noqa: E731
    return dict(x=f(b, L, D), r=1.5 * f(b, L, D), i=f(b, L, D), rate=f(D) - 2, bias_r=f(D),
                bias_i=f(D), h0=f(b, D))


def test_constant_gates_give_the_geometric_series():
    """r, i and x constant: h_t = a^t h0 + u (1 - a^t) / (1 - a)."""
    L, D = 12, 4
    rate = np.linspace(-4, 1, D)
    x, r, i = (np.full((1, L, D), v) for v in (0.7, 0.3, -0.4))
    y, hT = ly.glr_fwd(x, r, i, rate, c=2.0, h0=np.ones((1, D)))
    k = 2.0 * np.log1p(np.exp(rate))
    a = np.exp(-k / (1 + np.exp(-0.3)))
    u = np.sqrt(1 - a * a) * 0.7 / (1 + np.exp(0.4))
    for t in range(L):
        np.testing.assert_allclose(y[0, t], a ** (t + 1) + u * (1 - a ** (t + 1)) / (1 - a), rtol=1e-12)
    np.testing.assert_array_equal(hT[0], y[0, -1])


def test_a_reset_is_a_new_sequence_and_lengths_cut():
    d = inputs()
    reset = np.zeros((2, 9), bool)
    reset[0, 4] = True
    d["x"][0, 2] = np.inf  # nothing from before the reset may come through
    y, _ = ly.glr_fwd(**d, reset=reset)
    tail = {k: (v[:1, 4:] if v.ndim == 3 else v) for k, v in d.items() if k != "h0"}
    big = dict(tail, r=tail["r"].copy())
    z, _ = ly.glr_fwd(**big, reset=reset[:1, 4:])
    np.testing.assert_allclose(y[0, 4:], z[0], rtol=1e-13)
    d = inputs()
    y, hT = ly.glr_fwd(**d, lengths=[9, 5])
    z, zT = ly.glr_fwd(**{k: (v[1:, :5] if v.ndim == 3 else v[1:] if k == "h0" else v)
                          for k, v in d.items()})
    np.testing.assert_array_equal(y[1, :5], z[0])
    np.testing.assert_array_equal(hT[1], zT[0])
    assert not y[1, 5:].any()
    _, hT = ly.glr_fwd(**d, lengths=[0, -3])
    np.testing.assert_array_equal(hT, d["h0"])


@pytest.mark.parametrize("reset,lengths", [(False, None), (True, None), (True, [9, 4])])
def test_glr_gradients_are_the_differences(reset, lengths):
    """With y the unrounded state, every gradient is the central difference of the loss
    sum(dy y) + sum(dhT hT): step 1e-5, error about 1e-10 and the loss's rounding / 1e-5."""
    d = inputs(seed=3)
    g = np.random.default_rng(4)
    cut = g.random((2, 9)) < 0.3 if reset else None
    y, hT = ly.glr_fwd(**d, reset=cut, lengths=lengths)
    dy, dhT = g.standard_normal(y.shape), g.standard_normal(hT.shape)
    o = ly.glr_bwd(**{k: d[k] for k in d}, y=y, dy=dy, dhT=dhT, reset=cut, lengths=lengths)
    loss = lambda e: sum(np.sum(p * q) for p, q in  # noqa: E731
                         zip((dy, dhT), ly.glr_fwd(**e, reset=cut, lengths=lengths)))
    names = {"x": "dx", "r": "dr", "i": "di", "rate": "drate", "bias_r": "dbias_r",
             "bias_i": "dbias_i", "h0": "dh0"}
    if lengths is not None:  # rows behind the end: y is 0 there whatever dy is
        assert not o["dx"][1, 4:].any()
    for k, n in names.items():
        for _ in range(12):
            at = tuple(g.integers(0, m) for m in d[k].shape)
            lo, hi = dict(d), dict(d)
            lo[k], hi[k] = d[k].copy(), d[k].copy()
            lo[k][at] -= 1e-5
            hi[k][at] += 1e-5
            diff = (loss(hi) - loss(lo)) / 2e-5
            assert abs(diff - o[n][at]) <= 1e-7 * (1 + abs(diff)), (k, at)


def test_gates_at_their_ends():
    """An open recurrence gate without a rate keeps the state; a closed one too."""
    x = np.ones((1, 3, 1))
    for r, rate in ((-800.0, 0.0), (0.0, -800.0)):
        y, _ = ly.glr_fwd(x, x * r, x, np.array([rate]), h0=np.array([[2.0]]))
        np.testing.assert_allclose(y, 2.0, atol=1e-12)
        o = ly.glr_bwd(x, x * r, x, np.array([rate - 0.0]), y, np.ones_like(y), h0=np.array([[2.0]]))
        assert np.isfinite(o["dr"]).all() and np.abs(o["dr"]).max() < 1e-12


def test_rotation_is_a_matrix_and_keeps_the_norm():
    """One pair, weight 1: the output has mean square 1 and is turned counter-clockwise."""
    u = np.array([[[3.0, 4.0]]])
    o = ly.norm_rotate(u, None, [2], [np.pi / 4], 0.0)
    r = np.sqrt(12.5)
    np.testing.assert_allclose(o[0, 0], [-4 / r, 3 / r], rtol=1e-12)
    v = ly.norm_rotate(np.ones((1, 1, 4)), np.array([1.0, 2, 3, 4]), [5], [0.3], 0.0)[0, 0]
    np.testing.assert_allclose(v, [np.cos(1.5) - 2 * np.sin(1.5), np.sin(1.5) + 2 * np.cos(1.5), 3, 4],
                               rtol=1e-12)
    np.testing.assert_allclose(ly.norm_rotate(np.ones((1, 1, 4)), None, None, None, 3.0), 0.5)


def test_scores_depend_on_the_distance_alone():
    g = np.random.default_rng(0)
    q, k = g.standard_normal((2, 1, 1, 8))
    f = 10000.0 ** (-np.arange(4) / 4)
    dots = [np.sum(ly.norm_rotate(q, None, [p + 7], f, 0.0) * ly.norm_rotate(k, None, [p], f, 0.0))
            for p in (0, 11, -30, 100000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)


def test_norm_rotate_gradients_are_the_differences():
    g = np.random.default_rng(1)
    u, w, d = g.standard_normal((3, 2, 10)), g.standard_normal(10), g.standard_normal((3, 2, 10))
    pos, f = [4, 0, -9], np.array([1.0, 0.25, 0.1])
    du, dw = ly.norm_rotate_bwd(u, w, d, pos, f, 1e-3)
    loss = lambda a, b: np.sum(d * ly.norm_rotate(a, b, pos, f, 1e-3))  # noqa: E731
    for at in np.ndindex(u.shape):
        e = np.zeros_like(u)
        e[at] = 1e-5
        assert abs((loss(u + e, w) - loss(u - e, w)) / 2e-5 - du[at]) < 1e-8
    for j in range(10):
        e = np.zeros(10)
        e[j] = 1e-5
        assert abs((loss(u, w + e) - loss(u, w - e)) / 2e-5 - dw[j]) < 1e-8


def test_w4_layout_and_values():
    """A byte at a time: row 9, column 128 + 32 * 2 + 8 * 3 + 5 of 17 rows x 300 columns."""
    tiled = np.zeros(2 * 3 * 1024, np.uint8)
    tiled[1024 + 512 + 64 * 1 + 16 * 3 + 4 * 2 + 2] = 0xb4
    c = ly.w4_codes(tiled, 17, 300)
    assert c[9, 128 + 64 + 24 + 5] == 11 and c[9, 128 + 64 + 24 + 4] == 4 and c.sum() == 15
    w = ly.w4_weights(c, np.full((3, 17), 0.5), None, 128)
    assert w[9, 221] == 1.5 and w[0, 0] == -4
    w = ly.w4_weights(c, np.full((10, 17), 2.0), np.full((10, 17), 3), 32)
    assert w[9, 220] == 2 and w[0, 0] == -6


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 128])
def test_w4_quantisation_is_within_half_a_step(zeros, group):
    """Scales rounded to bf16 (2^-9 up or down) let the ends clip by 15 * 2^-9 of a step."""
    w = np.random.default_rng(0).standard_normal((5, 200)).astype(np.float32)
    w[2, :128] = 0
    bf = lambda a: (np.asarray(a, np.float32).view(np.uint32) + 0x7fff +  # noqa: E731
                    (np.asarray(a, np.float32).view(np.uint32) >> 16 & 1) & 0xffff0000).view(np.float32)
    c, s, z = ly.w4_quant(w, group, zeros, bf)
    err = np.abs(ly.w4_weights(c, s, z, group) - w)
    step = s.astype(np.float64)[np.arange(200) // group].T
    assert (err <= step * (0.5 + 15 / 512)).all() and not err[2, :128].any()
