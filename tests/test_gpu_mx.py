"""Microscaled quantisation and the product of microscaled operands, against the fp64
oracle.  Quantisation has one right answer (a power-of-two scale read off the largest
magnitude, an exact product with it, one rounding): codes, scales and padding are compared
byte for byte.  The product is of exact held values: each output may differ by its bf16
rounding (half a step, 2^-8 relative) plus fp32 accumulation, K 2^-23 sum |a w|."""
import numpy as np
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import lowbit as ol

pytestmark = pytest.mark.gpu


def values(rows, cols, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    return x.to(dtype)


def same_storage(t, x64, fmt):
    codes, tiles = ol.mx_store(*ol.mx_encode(x64, fmt), fmt)
    np.testing.assert_array_equal(t.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(t.scales.cpu().numpy(), tiles)


def fresh(fmt, rows, cols):
    """Storage full of a wrong pattern, so that unwritten padding shows."""
    t = m3.MXTensor.empty(fmt, rows, cols, "cuda")
    t.codes.fill_(0x5A)
    t.scales.fill_(0xA5)
    return t


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 33), (5, 128), (128, 256), (129, 1049),
                                       (333, 100), (1000, 24)])
def test_quant_and_back(fmt, dtype, rows, cols):
    x = values(rows, cols, rows + cols, dtype)
    t = m3.mx_quant(x.cuda(), fmt, out=fresh(fmt, rows, cols))
    back = m3.mx_dequant(t, dtype=torch.float32)
    back16 = m3.mx_dequant(t)
    torch.cuda.synchronize()
    same_storage(t, x.double().numpy(), fmt)
    ref = ol.mx_load(t.codes.cpu().numpy(), t.scales.cpu().numpy(), rows, cols, fmt)
    np.testing.assert_array_equal(back.cpu().double().numpy(), ref)
    np.testing.assert_array_equal(back16.float().cpu().numpy(),
                                  torch.from_numpy(ref).to(torch.bfloat16).float().numpy())


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_quant_extremes(fmt):
    """Ties, borders of the scale, subnormal, largest, zero, NaN and infinite values."""
    top = 6.0 if fmt == "mxfp4" else 448.0
    x = torch.zeros(40, 64)
    for i, amax in enumerate((top, float(np.nextafter(np.float32(top), np.float32(1e9))), top / 2,
                              1e-45, 1.1754944e-38, float(np.finfo(np.float32).max), 2.0 ** -127 * top,
                              2.0 ** -126 * top)):
        x[i, :32] = amax * torch.linspace(-1, 1, 32)
        x[i, 7] = -amax
    grid = torch.tensor(ol.GRID[fmt], dtype=torch.float32)
    mid = (grid[1:] + grid[:-1]) / 2  # every tie, beside the largest value
    for i in range((len(mid) + 30) // 31):
        part = mid[31 * i:31 * i + 31]
        x[10 + i, :len(part)] = part
        x[10 + i, 31] = -top
    x[30, 3], x[31, 40], x[32, 5] = float("nan"), float("inf"), float("-inf")
    x[30, 4] = 5.0
    t = m3.mx_quant(x.cuda(), fmt, out=fresh(fmt, 40, 64))
    back = m3.mx_dequant(t, dtype=torch.float32).cpu()
    same_storage(t, x.double().numpy(), fmt)
    for r, c in ((30, 0), (31, 32), (32, 0)):
        assert torch.isnan(back[r, c:c + 32]).all()
    assert torch.isfinite(back[31, :32]).all()
    # row 5: FLT_MAX = (2 - 2^-23) 2^127 rounds to the code 4 (256) at 2^126 (2^120), which is
    # 2^128, past fp32
    finite = torch.isfinite(back).all(-1)
    assert finite[:5].all() and not finite[5] and finite[6:30].all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_strided_and_unaligned_rows(fmt):
    base = values(67, 300, 8, torch.bfloat16).cuda()
    for view in (base[:, :200], base[:, 8:208], base[:, 3:203], base[:, 1:]):
        t = m3.mx_quant(view, fmt, out=fresh(fmt, *view.shape))
        same_storage(t, view.double().cpu().numpy(), fmt)
        wide = torch.full((67, 310), 7.0, dtype=torch.bfloat16, device="cuda")
        for off in (0, 5):
            out = wide[:, off:off + view.shape[1]]
            m3.mx_dequant(t, dtype=torch.bfloat16, out=out)
            assert torch.equal(out, m3.mx_dequant(t))
            assert torch.all(wide[:, :off] == 7) and torch.all(wide[:, off + view.shape[1]:] == 7)
            wide.fill_(7)


def operands(M, N, K, fmt, seed):
    A, W = values(M, K, seed).cuda(), values(N, K, seed + 1).cuda() / K ** 0.5
    return m3.mx_quant(A, fmt), m3.mx_quant(W, "mxfp4")


def held(t, rows=None):
    v = m3.mx_dequant(t, dtype=torch.float32)
    return (v if rows is None else v[rows]).double()


def check(D, A, W, rows=None):
    a, w = held(A, rows), held(W)
    got = (D if rows is None else D[rows]).double()
    ref = a @ w.t()
    bound = 2.0 ** -8 * ref.abs() + A.cols * 2.0 ** -23 * (a.abs() @ w.abs().t()) + 1e-30
    worst = ((got - ref).abs() / bound).max().item()
    assert worst <= 1, worst


SHAPES = [(1, 8, 32), (1, 1, 1), (5, 24, 100), (16, 128, 128), (16, 300, 1024), (17, 129, 257),
          (33, 520, 384), (64, 200, 640), (65, 64, 96), (127, 255, 64), (128, 256, 512),
          (129, 257, 1032), (300, 520, 200), (1000, 808, 768),
          # every tile the host chooses from, aligned and ragged: 128 x 192 (two), 128 x 256 (two),
          # 128 x 192 (two; 128 x 128 above)
          (300, 6464, 160), (299, 6463, 96), (4096, 1024, 160), (4001, 1001, 224),
          (3001, 2000, 160), (2000, 3001, 96)]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_matches_fp64(fmt, M, N, K):
    A, W = operands(M, N, K, fmt, M + N + K)
    D = m3.gemm_mx(A, W)
    torch.cuda.synchronize()
    assert m3.device_wait_timeouts() == 0
    check(D, A, W)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M", [13, 333])
def test_gemm_strided_and_unaligned_outputs(fmt, M):
    N = 300
    A, W = operands(M, N, 416, fmt, 4)
    for ld, off in ((N + 12, 0), (N + 13, 0), (N + 12, 3), (N + 12, 8)):
        big = torch.full((M + 2, ld + off), 7.0, dtype=torch.bfloat16, device="cuda")
        out = big[:M, off:off + N]
        m3.gemm_mx(A, W, out=out)
        torch.cuda.synchronize()
        check(out, A, W)
        assert torch.all(big[:M, :off] == 7) and torch.all(big[:M, off + N:] == 7)
        assert torch.all(big[M:] == 7)  # rows behind the last


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_gemm_block_shapes_sampled(fmt):
    """in_proj and out_proj at model size, on sampled rows."""
    for M, N, K in ((8200, 6464, 1024), (20011, 1024, 2048)):
        A, W = operands(M, N, K, fmt, 9)
        D = m3.gemm_mx(A, W)
        rows = torch.tensor([0, 1, 127, 128, 4095, M // 2, M - 1]).cuda()
        check(D, A, W, rows)
    assert m3.device_wait_timeouts() == 0


# whole rounds of tiles and a rest in parts: 64 and 128 columns of 192 and of 256, aligned and
# ragged
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M,N,K", [(18992, 1032, 160), (19131, 963, 288), (13829, 1537, 96),
                                   (19126, 578, 160), (20657, 577, 288), (20011, 1024, 96)])
def test_gemm_parts_of_tiles(fmt, M, N, K):
    A, W = operands(M, N, K, fmt, M + N + K)
    big = torch.full((M + 1, N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    m3.gemm_mx(A, W, out=big[:M, :N])
    check(big[:M, :N], A, W)
    assert torch.all(big[M:] == 7) and torch.all(big[:, N:] == 7)
    assert torch.equal(m3.gemm_mx(A, W), big[:M, :N])
    assert m3.device_wait_timeouts() == 0


# many tiles and a long K: whole tiles and parts of 64 and 128 columns, columns and rows that end
# inside them
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M,N,K", [(16384, 1024, 2048), (20011, 1024, 2048), (13000, 1537, 1500),
                                   (4090, 4000, 4096), (4001, 4099, 4200), (19000, 1000, 2304)])
def test_gemm_many_tiles(fmt, M, N, K):
    A, W = operands(M, N, K, fmt, M + N + K)
    big = torch.full((M + 1, N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    m3.gemm_mx(A, W, out=big[:M, :N])
    check(big[:M, :N], A, W)
    assert torch.all(big[M:] == 7) and torch.all(big[:, N:] == 7)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(m3.gemm_mx(A, W))
    torch.cuda.synchronize()
    assert all(torch.equal(o, big[:M, :N]) for o in outs)
    assert m3.device_wait_timeouts() == 0


# few tokens or few tiles and a long K: K over two, four and eight CTAs, at up to 16 tokens and
# beyond, whole and ragged
LONG_K = [(1, 129, 8192), (13, 4000, 3000), (7, 8200, 4160), (16, 8192, 8192), (3, 20000, 1000),
          (17, 130, 6400), (100, 520, 8200), (129, 255, 4224), (130, 4100, 8200),
          (257, 2000, 5000), (333, 1030, 2600)]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M,N,K", LONG_K)
def test_gemm_long_k(fmt, M, N, K):
    """Against fp64; the same bits from every run; other columns and rows of an output are
    left; runs that overlap on two streams do not disturb one another."""
    A, W = operands(M, N, K, fmt, M + N + K)
    D = m3.gemm_mx(A, W)
    check(D, A, W)
    for ld, off in ((N + 8, 0), (N + 5, 3)):
        big = torch.full((M + 1, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        m3.gemm_mx(A, W, out=big[:M, off:off + N])
        assert torch.equal(big[:M, off:off + N], D)
        big[:M, off:off + N] = 7
        assert torch.all(big == 7)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(m3.gemm_mx(A, W))
    torch.cuda.synchronize()
    assert all(torch.equal(o, D) for o in outs)
    assert m3.device_wait_timeouts() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M", [16, 100])
def test_gemm_long_k_captured(fmt, M):
    """Products with K over a cluster in two captured graphs, replayed on two streams on new
    values; a NaN block stays in its row and column."""
    x, w = values(M, 8192, 6).cuda(), m3.mx_quant(values(200, 8192, 7).cuda(), "mxfp4")
    def run():
        return m3.gemm_mx(m3.mx_quant(x, fmt), w)
    run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    x.mul_(0.75)
    x[2, 5000] = float("nan")
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for (g, _), side in zip(graphs, streams):
        with torch.cuda.stream(side):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    nan = torch.isnan(want)
    assert nan[2].all() and int(nan.sum()) == 200
    for _, out in graphs:
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert m3.device_wait_timeouts() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M", [3, 200])
def test_gemm_nan_blocks_stay_in_their_rows(fmt, M):
    A = values(M, 160, 1)
    W = values(90, 160, 2)
    A[2, 70], W[50, 10] = float("nan"), float("inf")
    D = m3.gemm_mx(m3.mx_quant(A.cuda(), fmt), m3.mx_quant(W.cuda(), "mxfp4")).cpu()
    nan = torch.isnan(D)
    assert nan[2].all() and nan[:, 50].all()
    nan[2], nan[:, 50] = False, False
    assert not nan.any()


def test_empty_sides():
    W = m3.mx_quant(values(40, 64, 1).cuda(), "mxfp4")
    A = m3.mx_quant(values(0, 64, 1).cuda(), "mxfp8")
    assert m3.gemm_mx(A, W).shape == (0, 40)
    assert m3.mx_dequant(A).shape == (0, 64)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_captured_and_on_another_stream(fmt):
    """Quantise, multiply and read back captured into two graphs and replayed on new inputs,
    also on a side stream; the same bits as the eager calls."""
    x, w = values(70, 256, 3).cuda(), m3.mx_quant(values(96, 256, 4).cuda(), "mxfp4")
    few = values(9, 256, 5).cuda()
    def run():
        return m3.gemm_mx(m3.mx_quant(x, fmt), w), m3.gemm_mx(m3.mx_quant(few, fmt), w)
    run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run()
        graphs.append((g, outs))
    x.mul_(-1.5)
    few.add_(0.25)
    want = [o.clone() for o in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for g, _ in graphs:
            g.replay()
        eager = run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for outs in [o for _, o in graphs] + [eager]:
        for got, ref in zip(outs, want):
            assert torch.equal(got, ref)
