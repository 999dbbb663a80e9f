"""Calls of the gated linear recurrence, the heads' norm with rotation and the 4-bit products that
their documentation allows and that come about in use: two at once, graphs replayed in turn, the same
tensor twice, values that are not finite across the parts of a long sequence and beside other tokens of
a large product."""
import pytest
import torch

import selective_state_space_m3ssd_b200 as m3
from tests.test_gpu_gemv_w4 import check as check_product, weights
from tests.test_gpu_glr import call, gpu, make, run_fwd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def work(seed):
    """A recurrence in parts and back, a rotation and back, a product: a thunk of their outputs."""
    d = gpu(make(1, 900, 130, BF, seed=seed, reset=0.01))
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(500, h, 64, generator=g).bfloat16().cuda() for h in (6, 2))
    w = (0.5 + torch.rand(2, 64, generator=g)).cuda()
    at = dict(positions=torch.arange(500, dtype=torch.int32).cuda(), freqs=(0.9 ** torch.arange(32.0)).cuda())
    W, _ = weights(1000, 1500, 64, True, seed=seed)
    x = torch.randn(8, 1500, generator=g).bfloat16().cuda()

    def run():
        y, hT = call(m3.glr_fwd, d)
        out = [y, hT, *call(m3.glr_bwd, d, y, d["dy"], dhT=d["dhT"]).values()]
        o = m3.norm_rotate(q, k, w[0], w[1], **at)
        out += [*o, *m3.norm_rotate_bwd(q, k, w[0], w[1], *o, **at).values()]
        return out + [m3.gemv_w4(x, W)]
    return run, (d, x, q)


def test_two_streams_at_once():
    jobs = [work(s)[0] for s in (1, 2)]
    want = [j() for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(jobs[k]())
    torch.cuda.synchronize()
    for k in range(2):
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k]))


def test_graphs_replayed_in_turn_follow_their_inputs():
    runs, inputs = zip(*(work(s) for s in (3, 4)))
    for r in runs:
        r()
    graphs, outs = [], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(r())
        graphs.append(g)
    for turn in range(3):
        for d, x, q in inputs:  # the inputs change where they lie
            d["x"].mul_(-1), x.mul_(0.5), q.mul_(-2)
        want = [r() for r in runs]
        for k in (1, 0):
            for o in outs[k]:
                o.fill_(float("nan"))
        graphs[turn % 2].replay()
        graphs[1 - turn % 2].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_same_tensor_as_several_inputs(dtype):
    d = make(2, 70, 66, dtype, seed=5)
    d["r"] = d["i"] = d["x"]
    y, hT = run_fwd(d)
    c = gpu(d)
    c["r"] = c["i"] = c["x"]
    y2, hT2 = call(m3.glr_fwd, c)
    assert torch.equal(y, y2) and torch.equal(hT, hT2)
    g = call(m3.glr_bwd, gpu(d), y, c["dy"], dhT=c["dhT"])
    g2 = call(m3.glr_bwd, c, y, c["dy"], dhT=c["dhT"])
    assert all(torch.equal(g[k], g2[k]) for k in g)
    u = torch.randn(40, 3, 64).to(dtype).cuda()
    a, b = m3.norm_rotate(u, u)
    assert torch.equal(a, b) and torch.equal(a, m3.norm_rotate(u)[0])
    g = m3.norm_rotate_bwd(u, u, None, None, a, a)
    assert torch.equal(g["dq"], g["dk"]) and torch.equal(g["dq_w"], g["dk_w"])


def test_parts_and_values_that_are_not_finite():
    """A token or start that is not a number reaches to the next reset, over the parts, and no other
    channel or sequence; what lies behind a sequence's end is not looked at."""
    for bad in (float("nan"), float("inf")):
        d = make(1, 1300, 64, F32, seed=6, reset=0.0, lengths=[1200])
        clean = gpu(d)
        y0, h0 = call(m3.glr_fwd, clean)
        d["h0"][0, 3] = bad
        for k in ("x", "r", "i", "dy"):
            d[k][0, 1200:] = bad
        y, hT = call(m3.glr_fwd, gpu(d))
        assert not torch.isfinite(y[0, 0, 3]) and not torch.isfinite(hT[0, 3])
        keep = [c for c in range(64) if c != 3]
        assert torch.equal(y[..., keep], y0[..., keep]) and torch.equal(hT[:, keep], h0[:, keep])
        d["reset"][0, 700] = True
        c = gpu(d)
        y, hT = call(m3.glr_fwd, c)
        assert torch.isfinite(y[0, 700:]).all() and torch.isfinite(hT).all()
        c["dhT"][0, 5], c["dy"][0, 690, 7] = bad, bad
        c["h0"][0, 3] = 0
        y, hT = call(m3.glr_fwd, c)
        ok = torch.isfinite(call(m3.glr_bwd, c, y, c["dy"], dhT=c["dhT"])["dx"])[0]
        assert not ok[700:1200, 5].any() and ok[:700, 5].all() and ok[1200:].all()
        assert not ok[:691, 7].any() and ok[691:, 7].all()
        assert ok[:, [c for c in range(64) if c not in (5, 7)]].all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_large_products_keep_tokens_apart(dt):
    M, N, K = 5, 300, 5000
    W, w = weights(N, K, 32, True, seed=7)
    buf = torch.randn(M, K + 5, generator=torch.Generator().manual_seed(7)).to(dt).cuda()
    x = buf[:, 3:3 + K]  # rows that start inside a word
    out = torch.full((M, N + 7), 5.0, device="cuda", dtype=BF)
    check_product(m3.gemv_w4(x, W, out=out[:, 2:2 + N]), x, w, K)
    assert (out[:, :2] == 5).all() and (out[:, 2 + N:] == 5).all()
    clean = m3.gemv_w4(x, W, out_dtype=F32)
    for bad in (float("nan"), float("-inf")):
        x[3, 4999] = bad
        got = m3.gemv_w4(x, W, out_dtype=F32)
        assert torch.equal(got[[0, 1, 2, 4]], clean[[0, 1, 2, 4]])
        assert not torch.isfinite(got[3]).any()

