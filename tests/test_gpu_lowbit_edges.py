"""Edges of the low-bit and norm operators: widths below one access, rows that are not finite,
waits that are given up, arguments of another device or layout."""
import numpy as np
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from oracle import lowbit as ol
from tests import test_gpu_mx as mx
from tests import test_gpu_norm as norm
from tests import test_gpu_step_q8 as step_q8
from tests.test_gpu_norm import BF16, F32, FP, cu, inputs, np64, summed

pytestmark = pytest.mark.gpu

# rows narrower than an access of eight elements: the tensor's end is several rows away from
# the first access that would pass it
NARROW = [(rows, d) for d in range(1, 8) for rows in (2, 3, 10, 1001)]


@pytest.mark.parametrize("rows,d", NARROW)
@pytest.mark.parametrize("dtype,res", [(F32, None), (BF16, None), (BF16, F32), (BF16, BF16),
                                       (F32, F32), (F32, BF16)])
def test_narrow_rows_forward(rows, d, dtype, res):
    norm.test_forward(rows, d, dtype, res)


@pytest.mark.parametrize("rows,d", NARROW)
@pytest.mark.parametrize("dtype,res", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("dres", [False, True])
def test_narrow_rows_backward(rows, d, dtype, res, dres):
    norm.test_backward(rows, d, dtype, res, dres)


@pytest.mark.parametrize("d", [1, 2, 3, 5, 7, 9])
def test_what_follows_a_narrow_tensor_is_left_out_and_left(d):
    """NaN behind every tensor of the call: outputs as without them, and the NaN still there."""
    rows = 11
    x, r, w = inputs(rows, d, F32, F32)
    y0, out0, rstd = m3.add_rmsnorm(*cu(x, w), residual=r.cuda(), want_rstd=True)
    wide = [torch.full((rows + 9, d), float("nan"), device="cuda") for _ in range(4)]
    wide[0][:rows], wide[1][:rows] = x.cuda(), r.cuda()
    m3.add_rmsnorm(wide[0][:rows], w.cuda(), residual=wide[1][:rows], y=wide[2][:rows],
                   residual_out=wide[3][:rows])
    assert torch.equal(wide[2][:rows], y0) and torch.equal(wide[3][:rows], out0)
    assert all(torch.isnan(t[rows:]).all() for t in wide)
    dr0, dw0 = m3.add_rmsnorm_bwd(x.cuda(), out0, w.cuda(), rstd, dres=r.cuda())
    dr = torch.full((rows + 9, d), float("nan"), device="cuda")
    _, dw = m3.add_rmsnorm_bwd(wide[0][:rows], wide[3][:rows], w.cuda(), rstd, dres=wide[1][:rows],
                               dr=dr[:rows])
    assert torch.equal(dr[:rows], dr0) and torch.equal(dw, dw0)
    assert torch.isnan(dr[rows:]).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("d", [5, 96, 100, 300, 1000, 1049, 4097])
@pytest.mark.parametrize("dtype,res", [(F32, None), (BF16, F32)])
def test_quantised_rows_that_are_not_finite(d, fmt, dtype, res):
    """Rows with a NaN, an infinity, or of zeros with eps 0 (rstd infinite): the bytes that
    quantising their y gives, so byte 255 in every block with a column and 0 in the padding's."""
    rows = 9
    x, r, w = inputs(rows, d, dtype, res)
    x[1, 0], x[4, d - 1], x[6] = float("nan"), float("inf"), 0
    if r is not None:
        r[6] = 0
    xc, wc, rc = cu(x, w, r)
    q = m3.add_rmsnorm(xc, wc, residual=rc, eps=0.0, fmt=fmt)[0]
    y = m3.add_rmsnorm(xc, wc, residual=rc, eps=0.0)[0]
    assert torch.isnan(y[[1, 6]]).all() and torch.isnan(y[4, d - 1])
    u = m3.mx_quant(y, fmt)
    bad = [1, 4, 6]
    assert torch.equal(q.codes[[1, 6]], u.codes[[1, 6]])
    blocks, kp = (d + 31) // 32, q.scales.numel() // 128 * 32
    tiles = q.scales.view(-1, 32, 4, 4)[:, :, 0, :].permute(1, 0, 2).reshape(32, kp // 32)
    other = u.scales.view(-1, 32, 4, 4)[:, :, 0, :].permute(1, 0, 2).reshape(32, kp // 32)
    assert torch.equal(tiles[bad], other[bad])
    assert torch.all(tiles[[1, 6], :blocks] == 255) and tiles[4, blocks - 1] == 255
    assert torch.all(tiles[:, blocks:] == 0) and torch.all(tiles[rows:] == 0)
    assert torch.all(q.codes[:, (d + 1) // 2 if fmt == "mxfp4" else d:] == 0)


LANES = [1, 0x0000ffff, 0xaaaaaaaa, 0xffffffff]


# one tile a CTA and several, whole and in parts; K in one CTA and over a cluster, tokens as the
# narrow side and not
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M,N,K", [(300, 520, 384), (20011, 1024, 256), (4096, 6464, 96),
                                   (16, 8192, 256), (16, 1024, 8192), (100, 520, 8192)])
def test_waits_that_some_lanes_give_up_end_the_product(fmt, M, N, K):
    """The warps leave together, the launch is reported, and the next one is right."""
    g = torch.Generator().manual_seed(M)
    A = m3.mx_quant(torch.randn(M, K, generator=g).cuda(), fmt)
    W = m3.mx_quant((torch.randn(N, K, generator=g) / K ** 0.5).cuda(), "mxfp4")
    want = m3.gemm_mx(A, W)
    assert m3.device_wait_timeouts() == 0
    for lanes in LANES:
        m3.give_up_next_waits_for_tests(lanes)
        m3.gemm_mx(A, W)  # outputs undefined
        assert m3.device_wait_timeouts() >= 1
        assert torch.equal(m3.gemm_mx(A, W), want)
        assert m3.device_wait_timeouts() == 0


# one tile a CTA and several; the pairs of row blocks too; aligned outputs and not
@pytest.mark.parametrize("M,N,K", [(300, 520, 72), (16384, 1024, 256), (37888, 256, 128),
                                   (75000, 250, 64), (3000, 2001, 128)])
def test_waits_that_some_lanes_give_up_end_the_bf16_product(M, N, K):
    g = torch.Generator().manual_seed(M)
    A = torch.randn(M, K, generator=g).bfloat16().cuda()
    W = (torch.randn(N, K, generator=g) / K ** 0.5).bfloat16().cuda()
    want = m3.gemm_bf16(A, W)
    assert m3.device_wait_timeouts() == 0
    for lanes in LANES:
        m3.give_up_next_waits_for_tests(lanes)
        m3.gemm_bf16(A, W)  # outputs undefined
        assert m3.device_wait_timeouts() >= 1
        assert torch.equal(m3.gemm_bf16(A, W), want)
        assert m3.device_wait_timeouts() == 0


def step_inputs(b, H, P, N, G, dtype, seed=0):
    """x_t, logdecay, beta, gamma, B, C, theta, D and a quantised cache."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = [n(b, H, P).to(dtype), -torch.rand(b, H, generator=g), n(b, H), n(b, H),
         n(b, G, N).to(dtype), n(b, G, N).to(dtype), n(b, H, N // 2), n(H)]
    cache = m3.quant_cache({"angle": n(b, H, N // 2).cuda(), "ssm": n(b, H, N, P).cuda(),
                            "x_prev": n(b, H, P).cuda(), "b_prev": n(b, G, N).cuda()})
    return [t.cuda() for t in a], cache


# one round a CTA, and two
@pytest.mark.parametrize("b,H,G", [(10, 32, 1), (40, 32, 4)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_step_whose_wait_some_lanes_give_up_writes_nothing(b, H, G, dtype):
    a, cache = step_inputs(b, H, 64, 128, G, dtype)
    want_cache = {k: torch.empty_like(v) for k, v in cache.items()}
    want = m3.step_q8(cache, *a, cache_out=want_cache)
    assert m3.device_wait_timeouts() == 0
    for lanes in LANES:
        out = {k: torch.full_like(v, 77) for k, v in cache.items()}
        y = torch.full_like(a[0], 77)
        m3.give_up_next_waits_for_tests(lanes)
        m3.step_q8(cache, *a, cache_out=out, y_t=y)
        assert m3.device_wait_timeouts() >= 1
        for t in (y, *out.values()):
            assert torch.all(t == 77)
        m3.step_q8(cache, *a, cache_out=out, y_t=y)  # the same step again
        assert m3.device_wait_timeouts() == 0
        assert torch.equal(y, want)
        assert all(torch.equal(out[k], want_cache[k]) for k in out)


# both kernels of N = 128, P = 64, and the general one with whole accesses and without
@pytest.mark.parametrize("b,H,P,N", [(2, 4, 64, 128), (10, 32, 64, 128), (3, 4, 64, 64),
                                     (3, 4, 75, 32)])
def test_a_step_holds_tiny_rows_as_quant_state_does(b, H, P, N):
    """A state that decays below 2^-100 a row: scale 0 and codes 0 (or -0), as quant_state
    writes the same values."""
    a, _ = step_inputs(b, H, P, N, 1, F32)
    g = torch.Generator().manual_seed(5)
    ssm = torch.randn(b, H, N, P, generator=g).cuda()
    up = torch.full((b, H, N, 1), 2.0 ** -99, device="cuda")
    up[:, :, ::3], up[:, :, 1::3] = 2.0 ** -104, 2.0 ** -130
    zero = torch.zeros(b, 1, N, device="cuda")
    cache = m3.quant_cache({"angle": torch.zeros(b, H, N // 2, device="cuda"), "ssm": ssm,
                            "x_prev": torch.zeros(b, H, P, device="cuda"), "b_prev": zero})
    cache["scale"] *= up[..., 0]
    held = m3.dequant_state(cache["ssm"], cache["scale"])
    codes, scale = m3.quant_state(held)
    m3.step_q8(cache, a[0], torch.zeros(b, H, device="cuda"), None, torch.zeros(b, H, device="cuda"),
               zero, zero)
    tiny = held.abs().amax(-1) < 2.0 ** -100
    assert tiny[:, :, ::3].all() and tiny[:, :, 1::3].all() and not tiny.all()
    assert torch.equal(cache["scale"] == 0, tiny) and torch.equal(scale == 0, tiny)
    assert torch.all(cache["ssm"][tiny] & 127 == 0) and torch.all(codes[tiny] & 127 == 0)
    assert torch.equal(m3.dequant_state(cache["ssm"], cache["scale"])[tiny],
                       torch.zeros_like(held)[tiny])


def test_a_workspace_elsewhere_is_refused():
    """Host memory, and memory with holes: before any launch."""
    dy, r, w = cu(*inputs(6, 40, F32, F32))
    rstd = torch.ones(6, device="cuda")
    need = m3.add_rmsnorm_bwd_workspace_size(m3.NormDims(6, 40, m3.F32, m3.F32, 0.0, 0))
    want = m3.add_rmsnorm_bwd(dy, r, w, rstd)
    for bad in (torch.empty(2 * need, dtype=torch.uint8),
                torch.empty(4 * need, dtype=torch.uint8, device="cuda")[::2],
                torch.empty(1, dtype=torch.uint8, device="cuda").expand(2 * need)):
        with pytest.raises(ValueError, match="workspace must be"):
            m3.add_rmsnorm_bwd(dy, r, w, rstd, workspace=bad)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    got = m3.add_rmsnorm_bwd(dy, r, w, rstd, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x = torch.randn(1, 70, 2, 64, device="cuda", dtype=BF16)
    bc, f = torch.randn(1, 70, 1, 128, device="cuda", dtype=BF16), torch.randn(1, 70, 2, device="cuda")
    for call in (lambda ws: m3.fwd(x, -f.abs(), f, f, bc, bc, workspace=ws),
                 lambda ws: m3.bwd(x, -f.abs(), f, f, bc, bc, dY=x, workspace=ws)):
        call(None)
        with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
            call(torch.empty(1 << 24, dtype=torch.uint8))


@pytest.mark.parametrize("b,H,P,N", [(2, 4, 64, 128), (12, 32, 64, 128), (3, 4, 64, 64),
                                     (2, 3, 12, 10)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_angles_of_the_whole_range(b, H, P, N, dtype):
    """Old angles and theta up to 1e5 with sums up to 1e5, all multiples of 2^-6: the fp32 sum
    is exact, and so is x - k fp32(2 pi) or x - k fp32(pi / 2) (k below 2^16, multiples of
    2^-21 or 2^-23 near or below pi).  The second term's rounding is 2^-23 at most and what two
    terms leave of 2 pi or pi / 2 below 1e-9 for such k: within the 4 2^-23 that the step's
    tolerances allow an angle."""
    inp, cache = step_q8.make(b, H, 1, N, P, dtype)
    g = torch.Generator().manual_seed(11)
    at = lambda *s: torch.round((torch.rand(*s, generator=g) * 2 - 1) * 1e5 * 64) / 64  # noqa: E731
    old, new = at(b, H, N // 2), at(b, H, N // 2)
    theta = new - old
    far = theta.abs() > 1e5
    theta[far] = old[far].sign() * 0.25
    old.view(-1)[:4] = torch.tensor([1e5, -1e5, 99999.0, 0.0])
    theta.view(-1)[:4] = torch.tensor([-1e5, 1e5, 1.0, -99999.984375])
    assert (old.double() + theta.double()).abs().max() <= 1e5 + 1
    cache["angle"], inp["theta"] = old, theta
    args = [None if inp[k] is None else inp[k].cuda() for k in step_q8.ORDER]
    cd = step_q8.to_cuda(cache)
    out = {k: torch.full_like(v, 77) for k, v in cd.items()}
    y = m3.step_q8(cd, *args, cache_out=out)
    step_q8.check(inp, cache, y, out, dtype == "bf16")


# what no other shape of the tests takes: the tiles left over in parts of 128 columns of 192, and
# 4-bit A with K over four CTAs beyond 16 tokens
PLANS = [(32006, 262, 38), (32006, 264, 200), (1785, 14959, 380), (269, 528, 4373),
         (269, 529, 4400)]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M,N,K", PLANS)
def test_gemm_plans(fmt, M, N, K):
    mx.test_gemm_parts_of_tiles(fmt, M, N, K)
