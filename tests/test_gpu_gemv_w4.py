"""4-bit weights in groups: the conversions bit for bit, and their product with a few tokens
against fp64.

Tolerance of the product: every product x (code - zero) is exact, sums run in fp32 in any order, at
most two roundings a term with the scaling: K 2^-23 of the sum of magnitudes; fp32 tokens enter
as three exact parts, which triples the terms.  Outputs add half a step of their type.
"""
import numpy as np
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import layer as ly
from tests.gpu_util import np64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().float().numpy()


def weights(N, K, group, zeros, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = -(-K // group)
    codes = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
    scales = K ** -0.5 * torch.exp(0.5 * torch.randn(N, n, generator=g))
    z = torch.randint(0, 16, (N, n), generator=g, dtype=torch.uint8) if zeros else None
    W = m3.W4Tensor.from_codes(codes.cuda(), scales.cuda(), None if z is None else z.cuda(), group=group)
    w = ly.w4_weights(codes.numpy(), np64(W.scales), None if z is None else z.numpy().T, group)
    return W, w


def check(out, x, w, K):
    ref, mag = np64(x) @ w.T, np.abs(np64(x)) @ np.abs(w.T)
    tol = 3 * K * 2.0 ** -23 * mag
    bad = ~(np.abs(np64(out) - ref) <= tol + HALF[out.dtype] * (np.abs(ref) + tol) + 1e-37)
    assert not bad.any(), (float(np.abs(np64(out) - ref).max()), np.argwhere(bad)[:4])


# sizes around tiles of 16 x 128, one and several pieces of K, few and many rows (parts of K 1 to 8)
SHAPES = [(1, 1), (16, 128), (15, 127), (17, 129), (100, 32), (40, 1000), (333, 2049), (6464, 1024), (8, 16384),
          (1024, 5000), (20000, 257), (9480, 640), (40000, 96)]


@pytest.mark.parametrize("group", [32, 64, 128, 384])
@pytest.mark.parametrize("N,K", SHAPES)
def test_product(N, K, group):
    for M, dt, zeros, out in ((1, BF, False, BF), (3, F32, True, F32), (8, BF, True, F32)):
        W, w = weights(N, K, group, zeros, seed=N + K)
        x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(dt).cuda()
        check(m3.gemv_w4(x, W, out_dtype=out), x, w, K)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M", range(1, 17))
def test_every_number_of_tokens(M, dt):
    for (N, K, group, zeros) in ((50, 700, 64, True), (300, 3000, 128, False)):
        W, w = weights(N, K, group, zeros, seed=M)
        g = torch.Generator().manual_seed(M)
        x = (torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))).to(dt).cuda()
        check(m3.gemv_w4(x, W), x, w, K)


@pytest.mark.parametrize("M,N,K,group,zeros,dt", [
    (1, 33, 9000, 32, True, BF), (1, 300, 8191, 128, False, BF), (2, 2500, 3100, 256, True, F32),
    (8, 7, 1024, 64, True, BF), (8, 300, 9000, 32, False, BF), (8, 40000, 1000, 64, True, BF),
    (9, 2500, 1111, 128, True, BF), (16, 300, 9000, 32, True, BF), (16, 40000, 640, 128, False, BF),
    (5, 1234, 1030, 32, True, F32), (8, 2500, 4100, 64, True, F32), (16, 2500, 4100, 32, False, F32),
    (16, 7, 9000, 64, True, F32), (16, 3000, 100, 32, True, F32), (9, 333, 90, 32, False, F32),
    (12, 3000, 300, 64, True, BF)])
def test_many_bytes_of_tokens(M, N, K, group, zeros, dt):
    # from 12 KB of tokens on a CTA has all of an SM's warps: parts of K for all of them and for none,
    # several pieces of the tokens and one; and less than that of many columns
    W, w = weights(N, K, group, zeros, seed=N + K)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(dt).cuda()
    check(m3.gemv_w4(x, W, out_dtype=F32), x, w, K)


@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_of_any_stride_and_alignment(dt):
    N, K, M = 70, 333, 5
    W, w = weights(N, K, 32, True)
    for off, width in ((0, 333), (1, 340), (8, 352), (3, 337)):
        buf = torch.full((M, width + off), float("nan"), device="cuda", dtype=dt)
        x = buf[:, off:off + K]
        x.copy_(torch.randn(M, K))
        out = torch.full((M, N + off + 3), 7.0, device="cuda", dtype=dt)
        got = m3.gemv_w4(x, W, out=out[:, off:off + N])
        check(got, x, w, K)
        assert (out[:, :off] == 7).all() and (out[:, off + N:] == 7).all()


def test_values_that_are_not_finite_stay_with_their_token():
    W, w = weights(40, 300, 64, False)
    for dt in (BF, F32):
        for bad in (float("inf"), float("nan")):
            x = torch.randn(4, 300).to(dt).cuda()
            clean = m3.gemv_w4(x, W)
            x[2, 17] = bad
            out = m3.gemv_w4(x, W)
            assert not torch.isfinite(out[2]).any()
            assert torch.equal(out[[0, 1, 3]], clean[[0, 1, 3]])
    big = torch.full((1, 300), 3e38, device="cuda")  # the largest fp32 values have exact parts too
    one = m3.W4Tensor.from_codes(torch.full((1, 300), 8, dtype=torch.uint8).cuda(),
                                 torch.ones(1, 3).cuda())
    one.codes[0] = 0x89  # column 0: 9 - 8, column 1: 8 - 8
    assert float(m3.gemv_w4(big, one)[0, 0]) == float(torch.tensor(3e38))
    tiny = big * 0 + 1e-41  # and the smallest
    assert float(m3.gemv_w4(tiny, one)[0, 0]) in (float(tiny[0, 0]), 0.0)


def test_padding_is_not_looked_at():
    """Codes of rows and columns that are not there may be anything."""
    N, K = 37, 333
    W, w = weights(N, K, 128, True)
    x = torch.randn(2, K).bfloat16().cuda()
    a = m3.gemv_w4(x, W)
    codes = ly.w4_codes(W.codes.cpu().numpy(), N, K)
    full = torch.randint(0, 16, (48, 384), dtype=torch.uint8)
    full[:N, :K] = torch.from_numpy(codes.astype(np.uint8))
    V = m3.W4Tensor.from_codes(full.cuda(), torch.ones(48, 3).cuda())
    W.codes.copy_(V.codes)
    assert torch.equal(a, m3.gemv_w4(x, W))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (16, 128, 128), (37, 333, 32), (50, 1000, 64),
                                       (9, 700, 256)])
def test_quantisation_bit_for_bit(N, K, group, zeros, dt):
    g = torch.Generator().manual_seed(N)
    w = (torch.randn(N, K, generator=g) * torch.exp(torch.randn(N, 1, generator=g))).to(dt)
    w[N // 2, :min(K, 40)] = 0
    if N > 8:
        w[3], w[4, 0], w[5, K // 2] = w[3].abs(), float("nan"), float("inf")
        w[6] *= 1e-38
        w[7] = -w[7].abs() * (1e37 if dt == F32 else 1)
    q = m3.w4_quant(w.cuda(), group, zeros=zeros)
    codes, scales, zs = ly.w4_quant(w.float().numpy(), group, zeros, bf16)
    got = ly.w4_codes(q.codes.cpu().numpy(), N, K)
    np.testing.assert_array_equal(np64(q.scales), scales.astype(np.float64))
    fin = np.isfinite(scales)[np.arange(K) // group].T  # codes of a NaN group are free
    np.testing.assert_array_equal(got[fin], codes[fin])
    if zeros:
        np.testing.assert_array_equal(q.zeros.cpu().numpy()[np.isfinite(scales)], zs[np.isfinite(scales)])
    ref = ly.w4_weights(got, scales, None if zs is None else q.zeros.cpu().numpy(), group)
    for out in (F32, BF):
        back = m3.w4_dequant(q, out)
        exact = torch.from_numpy(ref).float().to(out)
        assert torch.equal(torch.nan_to_num(back.cpu(), nan=-77.0), torch.nan_to_num(exact, nan=-77.0))
    # rows with a stride, into storage given
    buf = torch.zeros(N, K + 3, dtype=dt)
    buf[:, 2:2 + K] = w
    o = m3.W4Tensor.empty(N, K, group, zeros, device="cuda")
    assert m3.w4_quant(buf.cuda()[:, 2:2 + K], group, zeros=zeros, out=o) is o
    assert torch.equal(o.codes, q.codes) and torch.equal(o.scales.view(torch.int16), q.scales.view(torch.int16))


def test_same_bits_again_and_in_a_graph():
    W, w = weights(5000, 2000, 64, True)
    x = torch.randn(7, 2000).bfloat16().cuda()
    a, out = m3.gemv_w4(x, W), torch.empty(7, 5000, dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            m3.gemv_w4(x, W, out=out)
    for _ in range(2):
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out)


def test_refusals_and_empty_calls():
    W, _ = weights(20, 64, 64, False)
    with pytest.raises(m3.M3SSDError) as e:
        m3.gemv_w4(torch.zeros(17, 64, device="cuda"), W)
    assert e.value.status == m3.ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        m3.gemv_w4(torch.zeros(2, 65, device="cuda"), W)
    with pytest.raises(ValueError):
        m3.gemv_w4(torch.zeros(2, 64), W)
    assert m3.gemv_w4(torch.zeros(0, 64, device="cuda"), W).shape == (0, 20)
    V = m3.W4Tensor.empty(0, 64, 64, device="cuda")
    assert m3.gemv_w4(torch.zeros(3, 64, device="cuda"), V).shape == (3, 0)


def test_small_fp32_tokens():
    """A token's value counts whole from 2^-110 on, below to the multiple of 2^-133 under it: a row of
    W with one column that is not zero leaves one product a part, three parts that add up with one
    rounding of fp32 each (2^-24 of the sum), into multiples of 2^-149 (2^-6 of them before the last
    product: half of 2^-143 each)."""
    K, at = 200, 150
    g = torch.Generator().manual_seed(5)
    e = -torch.arange(90, 150).double()
    x = (1 + torch.rand(60, generator=g, dtype=torch.float64)).mul(torch.exp2(e)).float()
    want = torch.where(x.double() < 2.0 ** -110, torch.floor(x.double() * 2.0 ** 133) * 2.0 ** -133, x.double())
    for code, value in ((15, 7.0), (9, 1.0), (0, -8.0)):
        codes = torch.full((1, K), 8, dtype=torch.uint8)
        codes[0, at] = code
        W = m3.W4Tensor.from_codes(codes.cuda(), torch.ones(1, 2).cuda())
        for lo in range(0, 60, 15):
            t = torch.zeros(15, K)
            t[:, at] = x[lo:lo + 15]
            got = m3.gemv_w4(t.cuda(), W)[:, 0].cpu().double()
            ref = value * want[lo:lo + 15]
            assert (abs(got - ref) <= 3 * 2.0 ** -24 * abs(ref) + 3 * 2.0 ** -144).all(), (code, lo)
            assert (got[(t[:, at] < 2.0 ** -133)] == 0).all()
