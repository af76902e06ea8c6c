"""The 8-bit block-scaled entry points on the GPU against 64-bit evaluations of
their definitions (tests/fp8_util.py derives the bounds)."""
import numpy as np
import pytest
import torch

from tests import fp8_util as R
from tests.gpu_util import random_topk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import moe_routing_expert_fp32_b200 as m
    m.lib()
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def bits(t):
    return t.contiguous().view(torch.uint8)


# ----------------------------------------------------------------- quantise
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("B,M,K,block_rows", [
    (1, 1, 16, 1), (1, 5, 128, 1), (1, 77, 144, 1), (1, 3, 7168, 1), (3, 33, 400, 1),
    (1, 1, 16, 128), (1, 128, 128, 128), (2, 200, 272, 128), (3, 7, 1040, 128)])
def test_quantize_bit_exact(moe, B, M, K, block_rows, pow2):
    g = gen(B * 1000 + M + K)
    x = torch.randn(B, M, K, generator=g, device="cuda")
    x = (x * torch.exp(3 * torch.randn(B, M, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    x[0, 0, :8] = 0
    x[-1, -1] = 0  # a row (and, for one-row weights, a block) of zeros
    q, s = moe.quantize_fp8(x, block_rows=block_rows, pow2_scales=pow2)
    qr, sr = R.quantize_ref(x, block_rows, pow2)
    assert torch.equal(s.view(sr.shape), sr)
    assert torch.equal(q.float(), qr)


def test_quantize_extremes(moe):
    """The type's largest and smallest values, a block that is exactly at a power
    of two, ties, and blocks with an infinity or a NaN."""
    x = torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
    x[0] = torch.finfo(torch.bfloat16).max
    x[1, 3] = 2.0 ** -133  # the smallest bf16 subnormals
    x[2, :128] = 448.0
    x[2, 1:20] = torch.arange(1, 20, device="cuda") * 0.5 + 16.0
    x[3, 200] = float("inf")
    x[3, 201] = 3.0
    x[4, 5] = float("nan")
    x[5, 0] = 7.0 * 2.0 ** 20
    for pow2 in (False, True):
        q, s = moe.quantize_fp8(x, pow2_scales=pow2)
        qr, sr = R.quantize_ref(x[None], 1, pow2)
        qr, sr = qr[0], sr[0]
        fin = torch.isfinite(sr)
        assert torch.equal(s[fin], sr[fin]) and fin.sum() == 10
        assert torch.isinf(s[3, 1]) and torch.isnan(s[4, 0])
        keep = fin.repeat_interleave(128, 1)
        assert torch.equal(q.float()[keep], qr[keep])
        assert torch.isnan(q.float()[3, 200]) and q.float()[3, 201] == 0
        assert torch.isnan(q.float()[4, 5])


def test_quantize_into_buffers_and_shapes(moe):
    x = torch.randn(2, 3, 272, device="cuda").to(torch.bfloat16)
    q, s = moe.quantize_fp8(x)
    assert q.shape == (2, 3, 272) and s.shape == (2, 3, 3)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    assert moe.quantize_fp8(x, q=q2, scale=s2)[0] is q2
    assert torch.equal(bits(q), bits(q2)) and torch.equal(s, s2)
    e, es = moe.quantize_fp8(x[:, :0])
    assert e.shape == (2, 0, 272) and es.shape == (2, 0, 3)


# ----------------------------------------------------------------- dispatch
@pytest.mark.parametrize("N,K,E,d,pow2", [(1, 1, 1, 16, False), (128, 8, 256, 7168, False),
                                          (33, 16, 1024, 144, True), (1500, 4, 7, 400, False)])
def test_dispatch_fp8(moe, N, K, E, d, pow2):
    g = gen(N + d)
    x = torch.randn(N, d, generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.from_numpy(random_topk(N, K, E, np.random.default_rng(N), 0.7 if E > K else 0)).cuda()
    counts, offsets, perm, pos, xq, xs = moe.dispatch_fp8(idx, x, E, pow2_scales=pow2)
    c0, o0, p0, q0, _ = moe.dispatch(idx, x, E)
    assert torch.equal(counts, c0) and torch.equal(offsets, o0)
    assert torch.equal(perm, p0) and torch.equal(pos, q0)
    qr, sr = R.quantize_ref(x[None], 1, pow2)
    tok = (perm // K).long()
    assert torch.equal(xq.float(), qr[0][tok]) and torch.equal(xs, sr[0][tok])


@pytest.mark.parametrize("E", [1, 37, 256, 1000, 1024])
@pytest.mark.parametrize("N,K", [(1, 1), (31, 1), (1024, 1), (1025, 1), (341, 7), (1024, 8),
                                 (2731, 3), (8192, 2), (4681, 14), (8192, 8), (65537, 1)])
def test_dispatch_fp8_sort(moe, N, K, E):
    """The sort behind the dispatch is the stable one, around the sizes where it
    changes its form, with skewed and with bad indices, and as often as it runs."""
    g = gen(N + K + E)
    idx = (torch.rand(N, K, generator=g, device="cuda") ** 3 * E).to(torch.int32).clamp(max=E - 1)
    if E > 1:
        idx[N // 2:, 0] = 1  # a long run of one expert
    bad = torch.rand(N, K, generator=g, device="cuda") < 0.02
    x = torch.randn(N, 16, generator=g, device="cuda").to(torch.bfloat16)
    xq0, xs0 = moe.quantize_fp8(x)
    ws = moe.workspace(moe.lib().moe_dispatch_workspace_size(N, K, E))
    for i in (idx, torch.where(bad, torch.full_like(idx, E), idx),
              torch.full_like(idx, E - 1), idx):
        flat = i.reshape(-1).long()
        live = (flat < E).nonzero().squeeze(1)
        order = live[torch.sort(flat[live], stable=True).indices]
        n = torch.bincount(flat[live], minlength=E)
        p_ref = torch.full_like(flat, -1)
        p_ref[order] = torch.arange(len(order), device="cuda")
        counts, offsets, perm, pos, xq, xs = moe.dispatch_fp8(i, x, E, ws=ws)
        assert moe.get_status(ws) == (-7 if len(live) < N * K else 0)
        assert torch.equal(counts.long(), n)
        assert torch.equal(offsets[1:].long(), n.cumsum(0)) and int(offsets[0]) == 0
        assert torch.equal(perm[:len(order)].long(), order)
        assert torch.equal(pos.long(), p_ref)
        assert torch.equal(bits(xq[:len(order)]), bits(xq0[order // K]))
        assert torch.equal(xs[:len(order)], xs0[order // K])


def test_dispatch_fp8_leaves_out_bad_indices(moe):
    """A slot with an expert outside [0, E) is recorded and left out; rows behind
    the last kept slot stay as they were."""
    N, K, E, d = 40, 2, 8, 256
    idx = torch.randint(0, E, (N, K), dtype=torch.int32, device="cuda")
    idx[3, 1], idx[17, 0] = E, -1
    x = torch.randn(N, d, device="cuda").to(torch.bfloat16)
    ws = moe.workspace(moe.lib().moe_dispatch_workspace_size(N, K, E))
    counts, offsets, perm, pos, xq, xs = moe.dispatch_fp8(idx, x, E, ws=ws)
    assert moe.get_status(ws) == -7
    S = int(offsets[-1])
    assert S == N * K - 2 and int(counts.sum()) == S
    qr, _ = R.quantize_ref(x[None], 1, False)
    assert torch.equal(xq.float()[:S], qr[0][(perm[:S] // K).long()])


# ------------------------------------------------------------------- linear
@pytest.mark.parametrize("M,K,N", [
    (1, 16, 8), (1, 7168, 2048), (2, 128, 128), (16, 2048, 1000), (17, 144, 136), (31, 272, 264),
    (33, 1040, 24), (100, 512, 384), (128, 1024, 256), (129, 400, 520), (300, 2048, 1160),
    (1000, 1296, 640), (5, 7168, 8), (40, 4096, 136), (3, 1040, 72),
    (4, 8192, 2056), (4, 8208, 520), (1, 32784, 40), (2, 7152, 5000), (3000, 400, 4232), (2048, 1040, 2312)])
def test_linear_fp8(moe, M, K, N):
    g = gen(M + K + N)
    xq, xs = R.rand_rows(g, M, K)
    w, ws = R.rand_weights(g, 1, N, K)
    y = moe.linear_fp8(xq, xs, w[0], ws[0])
    ref, bound = R.product(xq, xs, w[0], ws[0])
    R.assert_within(y, ref, bound, "plain")
    res = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)
    ref, bound = R.product(xq, xs, w[0], ws[0], res)
    z = moe.linear_fp8(xq, xs, w[0], ws[0], residual=res)
    R.assert_within(z, ref, bound, "residual")
    buf = res.clone()
    moe.linear_fp8(xq, xs, w[0], ws[0], residual=buf, out=buf)
    assert torch.equal(bits(buf), bits(z))


def test_linear_fp8_exact_values(moe):
    """Small integers times power-of-two scales: every sum is exact, so the
    result is, whatever the order."""
    g = gen(4)
    M, K, N = 70, 656, 328
    xi = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float()
    wi = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float()
    xs = torch.exp2(torch.randint(-2, 1, (M, 6), generator=g, device="cuda").float())
    ws = torch.exp2(torch.randint(-2, 1, (3, 6), generator=g, device="cuda").float())
    xq, wq = xi.to(torch.float8_e4m3fn), wi.to(torch.float8_e4m3fn)
    y = moe.linear_fp8(xq, xs, wq, ws)
    ref = (R.deq_rows(xq, xs) @ R.deq_weights(wq, ws).t()).float().to(torch.bfloat16)
    assert torch.equal(y, ref)


def test_linear_fp8_nonfinite_rows_stay_in_their_rows(moe):
    g = gen(9)
    x = torch.randn(40, 512, generator=g, device="cuda").to(torch.bfloat16)
    w, ws = R.rand_weights(g, 1, 256, 512)
    clean = moe.linear_fp8(*moe.quantize_fp8(x), w[0], ws[0])
    x[3, 100], x[20, 511] = float("nan"), float("inf")
    y = moe.linear_fp8(*moe.quantize_fp8(x), w[0], ws[0])
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[3] = bad[20] = True
    assert torch.isnan(y[bad]).all()
    assert torch.equal(bits(y[~bad]), bits(clean[~bad]))


def test_linear_fp8_more_than_2_31_elements(moe):
    """Rows, scales and outputs whose offsets pass 32 bits: the first and the
    last rows of 340000 x 6400 against the same rows alone."""
    g = gen(2)
    M, K, N = 340000, 6400, 6400
    row_q, row_s = R.rand_rows(g, 1000, K)
    xq = row_q.view(torch.uint8).repeat(M // 1000, 1).view(torch.float8_e4m3fn)
    xs = row_s.repeat(M // 1000, 1)
    assert xq.numel() > 2 ** 31
    w, ws = R.rand_weights(g, 1, N, K)
    y = moe.linear_fp8(xq, xs, w[0], ws[0])
    assert y.numel() > 2 ** 31
    part = moe.linear_fp8(row_q, row_s, w[0], ws[0])
    for a in (0, M // 2 // 1000 * 1000, M - 1000):
        d = (y[a:a + 1000].double() - part.double()).abs()
        # the same operator on the same rows: at most one bf16 rounding apart
        assert (d <= 2 * R.BF16_HALF * part.double().abs() + 1e-4).all()
    del xq, xs, y
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ grouped
SEGMENTS = {
    "one_each": [1, 1, 1, 1],
    "empty_ends": [0, 5, 0, 0, 40, 0],
    "all_on_one": [0, 0, 300, 0],
    "ragged": [16, 17, 0, 33, 129, 128, 127, 1],
    "tiles": [64, 256, 257, 31],
    "none": [0, 0, 0],
    "large": [700, 300, 130, 513, 0],
}


def offsets_of(counts, tail=0):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return torch.from_numpy(off).cuda(), int(off[-1]) + tail


@pytest.mark.parametrize("K,N", [(128, 128), (144, 264), (1040, 40), (512, 640)])
@pytest.mark.parametrize("name", list(SEGMENTS))
def test_grouped_linear_fp8(moe, name, K, N):
    counts = SEGMENTS[name]
    E = len(counts)
    off, S = offsets_of(counts, tail=9)
    g = gen(S + K + N)
    xq, xs = R.rand_rows(g, S, K)
    w, ws = R.rand_weights(g, E, N, K)
    out = torch.full((S, N), 7.25, dtype=torch.bfloat16, device="cuda")
    wk = moe.workspace(moe.lib().moe_grouped_linear_fp8_workspace_size(S, K, E, N))
    moe.grouped_linear_fp8(xq, xs, off, w, ws, out=out, ws=wk)
    assert moe.get_status(wk) == 0
    assert (out[S - 9:] == 7.25).all()  # behind the last segment: as they were
    a = 0
    for e, n in enumerate(counts):
        if n:
            ref, bound = R.product(xq[a:a + n], xs[a:a + n], w[e], ws[e])
            R.assert_within(out[a:a + n], ref, bound, f"expert {e}")
        a += n


def test_grouped_many_experts(moe):
    """1024 segments, most of them empty; and more rows than 128 per segment."""
    rng = np.random.default_rng(3)
    for E, S, K, N in ((1024, 300, 128, 72), (3, 1500, 256, 136)):
        counts = rng.multinomial(S, rng.dirichlet(np.ones(E)))
        off, _ = offsets_of(counts)
        g = gen(E)
        xq, xs = R.rand_rows(g, S, K)
        w, ws = R.rand_weights(g, E, N, K)
        y = moe.grouped_linear_fp8(xq, xs, off, w, ws)
        for e in np.nonzero(counts)[0]:
            a, b = int(off[e]), int(off[e + 1])
            ref, bound = R.product(xq[a:b], xs[a:b], w[e], ws[e])
            R.assert_within(y[a:b], ref, bound, f"expert {e}")


@pytest.mark.parametrize("bad", [[0, 5, 3, 20, 20], [0, 5, 30, 20, 20], [1, 5, 10, 20, 20],
                                 [0, -4, 10, 20, 20]])
def test_grouped_bad_offsets_are_recorded(moe, bad):
    """Segments that run backwards or leave [0, S] are left out and reported;
    the good ones are computed, and nothing out of range is written."""
    S, K, N = 20, 256, 136
    g = gen(1)
    xq, xs = R.rand_rows(g, S, K)
    w, ws = R.rand_weights(g, 4, N, K)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    out = torch.full((S, N), -3.0, dtype=torch.bfloat16, device="cuda")
    wk = moe.workspace(256)
    moe.grouped_linear_fp8(xq, xs, off, w, ws, out=out, ws=wk)
    assert moe.get_status(wk) == -7
    written = torch.zeros(S, dtype=torch.bool, device="cuda")
    for e in range(4):
        a, b = bad[e], bad[e + 1]
        if 0 <= a <= b <= S and not (e == 0 and a != 0):
            written[a:b] = True
            last = [k for k in range(4) if 0 <= bad[k] <= bad[k + 1] <= S and
                    bad[k] < b and bad[k + 1] > a and not (k == 0 and bad[k] != 0)]
            if last == [e] and b > a:  # rows of no other kept segment
                ref, bound = R.product(xq[a:b], xs[a:b], w[e], ws[e])
                R.assert_within(out[a:b], ref, bound, f"expert {e}")
    assert (out[~written] == -3.0).all()


# ---------------------------------------------------------------- expert MLP
@pytest.mark.parametrize("K,N", [(2048, 128), (256, 1024)])
def test_grouped_fp8_overlapping_segments(moe, K, N):
    """Segments behind one that runs backwards may overlap, more tiles than rows: the
    error is recorded, nothing outside the rows is written, and the next call is
    as always (with K split over a cluster too)."""
    E, S = 8, 100
    off = torch.tensor([0, 100] * 4 + [0], dtype=torch.int32, device="cuda")
    g = gen(31)
    xq, xs = R.rand_rows(g, S, K)
    w, ws = R.rand_weights(g, E, N, K)
    buf = torch.full((S + 64, N), 3.0, dtype=torch.bfloat16, device="cuda")
    wk = moe.workspace(moe.lib().moe_grouped_linear_fp8_workspace_size(S, K, E, N))
    moe.grouped_linear_fp8(xq, xs, off, w, ws, out=buf[32:32 + S], ws=wk)
    assert moe.get_status(wk) == -7
    assert (buf[:32] == 3).all() and (buf[32 + S:] == 3).all()
    off = torch.tensor([0] + [100] * 8, dtype=torch.int32, device="cuda")
    y = moe.grouped_linear_fp8(xq, xs, off, w, ws, ws=wk)
    assert moe.get_status(wk) == 0
    ref, bound = R.product(xq, xs, w[0], ws[0])
    R.assert_within(y, ref, bound)


def make_ffn(g, E, d, F, S, pow2):
    xq, xs = R.rand_rows(g, S, d, pow2)
    w1, w1s = R.rand_weights(g, E, F, d)
    w3, w3s = R.rand_weights(g, E, F, d)
    w2, w2s = R.rand_weights(g, E, d, F)
    return xq, xs, (w1, w1s, w3, w3s, w2, w2s)


@pytest.mark.parametrize("act,beta,lbeta", [("silu", 1.0, 0.0), ("situ", 4.0, 8.0),
                                            ("situ", 0.0, 0.0)])
@pytest.mark.parametrize("d,F,pow2", [(256, 128, False), (272, 400, True), (128, 16, False),
                                      (1040, 528, True)])
@pytest.mark.parametrize("name", ["empty_ends", "ragged", "tiles", "large"])
def test_expert_ffn_fp8(moe, name, d, F, pow2, act, beta, lbeta):
    counts = SEGMENTS[name]
    E = len(counts)
    off, S = offsets_of(counts, tail=3)
    g = gen(S + d + F)
    xq, xs, w = make_ffn(g, E, d, F, S, pow2)
    y = torch.full((S, d), 5.5, dtype=torch.bfloat16, device="cuda")
    wk = moe.workspace(moe.lib().moe_expert_ffn_fp8_workspace_size(S, d, E, F))
    moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig(act, beta, lbeta), pow2_scales=pow2, y=y,
                       ws=wk)
    assert moe.get_status(wk) == 0
    assert (y[S - 3:] == 5.5).all()
    a = 0
    for e, n in enumerate(counts):
        if n:
            ref, bound = R.ffn(xq[a:a + n], xs[a:a + n], *[t[e] for t in w], act, beta or 1.0,
                               lbeta, pow2)
            R.assert_within(y[a:a + n], ref, bound, f"expert {e}")
        a += n


def test_expert_ffn_fp8_large_gates(moe):
    """Gates far into the activation's tails: silu(-200) is 0, silu(200) = 200,
    SiTU saturates; no NaN appears."""
    g = gen(8)
    xq, xs, w = make_ffn(g, 2, 256, 256, 60, False)
    w = (w[0], w[1] * 100, *w[2:])
    off = torch.tensor([0, 20, 60], dtype=torch.int32, device="cuda")
    for act, beta, lbeta in (("silu", 1.0, 0.0), ("situ", 4.0, 8.0)):
        y = moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig(act, beta, lbeta))
        for e, (a, b) in enumerate(((0, 20), (20, 60))):
            ref, bound = R.ffn(xq[a:b], xs[a:b], *[t[e] for t in w], act, beta, lbeta, False)
            R.assert_within(y[a:b], ref, bound, f"{act} expert {e}")


@pytest.mark.parametrize("counts", [[20, 9], [300, 200]])
@pytest.mark.parametrize("act,beta,lbeta", [("silu", 1.0, 0.0), ("situ", 4.0, 8.0),
                                            ("situ", 2.0, 0.0), ("situ", -1.0, 0.5)])
def test_expert_ffn_fp8_argument_sizes(moe, act, beta, lbeta, counts):
    """The activation from arguments where tanh is its argument, over the border of
    its series, to where it is 1, in the kernels of few and of many rows."""
    off, S = offsets_of(counts)
    g = gen(21)
    xq, xs, w = make_ffn(g, 2, 256, 256, S, False)
    for by in (1e-5, 0.01, 0.08, 0.5, 8.0):
        v = (w[0], w[1] * by, w[2], w[3] * by, *w[4:])
        y = moe.expert_ffn_fp8(xq, xs, off, *v, moe.ActConfig(act, beta, lbeta))
        a = 0
        for e, n in enumerate(counts):
            ref, bound = R.ffn(xq[a:a + n], xs[a:a + n], *[t[e] for t in v], act, beta, lbeta,
                               False)
            R.assert_within(y[a:a + n], ref, bound, f"x {by}, expert {e}")
            a += n


# ---------------------------------------------------------- the run together
def layer_inputs(moe, N=100, d_r=256, d_e=256, E=16, F=128, K=4, seed=3):
    g = gen(seed)
    x = torch.randn(N, d_r, generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn(E, d_r, generator=g, device="cuda") * 0.05
    bias = torch.randn(E, generator=g, device="cuda") * 0.01
    raw = [torch.randn(E, *s, generator=g, device="cuda").mul_(0.05).to(torch.bfloat16)
           for s in ((F, d_e), (F, d_e), (d_e, F))]
    q = [moe.quantize_fp8(t, block_rows=128) for t in raw]
    cfg = moe.RouteConfig(E, 4, 2, K, 2.5)
    return x, W, bias, cfg, raw, [t for pair in q for t in pair]


def test_layer_equals_its_steps_and_follows_bf16(moe):
    """forward_fp8 is route -> dispatch_fp8 -> expert_ffn_fp8 -> combine bit for
    bit, and near the bf16 layer on the weights it was quantised from."""
    x, W, bias, cfg, raw, q = layer_inputs(moe)
    act = moe.ActConfig("silu")
    idx = torch.empty(100, 4, dtype=torch.int32, device="cuda")
    tw = torch.empty(100, 4, device="cuda")
    out = moe.forward_fp8(x, W, bias, cfg, *q, act, topk_idx=idx, topk_w=tw)
    i2, w2 = moe.route(x, W, bias, cfg)
    assert torch.equal(idx, i2) and torch.equal(tw, w2)
    counts, off, perm, pos, xq, xs = moe.dispatch_fp8(i2, x, 16)
    y = moe.expert_ffn_fp8(xq, xs, off, *q, act)
    assert torch.equal(bits(out), bits(moe.combine(y, pos, w2)))
    ref = moe.forward(x, W, bias, cfg, *raw, act).double()
    # each of x, w1, w3, h, w2 is rounded by at most 2^-4 relative, uniformly: a
    # deviation of 2^-4 / sqrt(3) / ~1.4 = 2.6 %.  g and u carry two of them
    # each, y two more beside h: sqrt(2 * 2 + 1 + 1) of 2.6 % is 6.4 %; twice that
    rel = ((out.double() - ref).norm() / ref.norm()).item()
    assert rel < 0.13, rel


def test_layer_latent_input_and_pow2(moe):
    x, W, bias, cfg, raw, q = layer_inputs(moe, d_r=512, d_e=272, F=144, seed=5)
    xe = torch.randn(100, 272, device="cuda").to(torch.bfloat16)
    act = moe.ActConfig("situ", 4.0, 8.0)
    out = moe.forward_fp8(x, W, bias, cfg, *q, act, x_e=xe, pow2_scales=True)
    i2, w2 = moe.route(x, W, bias, cfg)
    _, off, _, pos, xq, xs = moe.dispatch_fp8(i2, xe, 16, pow2_scales=True)
    y = moe.expert_ffn_fp8(xq, xs, off, *q, act, pow2_scales=True)
    assert torch.equal(bits(out), bits(moe.combine(y, pos, w2)))


def test_fp8_calls_on_a_side_stream_and_in_a_graph(moe):
    """The layer on another stream, captured, and replayed on new inputs, with
    two graphs that share one workspace."""
    x, W, bias, cfg, raw, q = layer_inputs(moe, seed=7)
    act = moe.ActConfig("silu")
    want = moe.forward_fp8(x, W, bias, cfg, *q, act).clone()
    want_neg = moe.forward_fp8(-x, W, bias, cfg, *q, act).clone()
    ws = moe.workspace(moe.forward_fp8_workspace_size(100, 256, 256, cfg, 128))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = moe.forward_fp8(x, W, bias, cfg, *q, act, ws=ws)
    s.synchronize()
    assert torch.equal(bits(side), bits(want))
    bufs = [(x.clone(), torch.empty_like(want)) for _ in range(2)]
    graphs = []
    for xi, oi in bufs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            moe.forward_fp8(xi, W, bias, cfg, *q, act, ws=ws, out=oi)
        graphs.append(gr)
    bufs[1][0].copy_(-x)
    for _ in range(2):
        for (xi, oi), gr in zip(bufs, graphs):
            oi.zero_()
            gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(bufs[0][1]), bits(want))
    assert torch.equal(bits(bufs[1][1]), bits(want_neg))
    assert moe.get_status(ws) == 0


def test_fp8_results_repeat(moe):
    """The same call twice gives the same bits."""
    g = gen(6)
    off, S = offsets_of([300, 1, 0, 77])
    xq, xs, w = make_ffn(g, 4, 512, 384, S, False)
    a = moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig("silu"))
    for _ in range(3):
        assert torch.equal(bits(a), bits(moe.expert_ffn_fp8(xq, xs, off, *w,
                                                            moe.ActConfig("silu"))))
    y = moe.linear_fp8(xq[:1], xs[:1], w[0][0], w[1][0])
    for _ in range(3):
        assert torch.equal(bits(y), bits(moe.linear_fp8(xq[:1], xs[:1], w[0][0], w[1][0])))


@pytest.mark.parametrize("M,K,N", [(8, 2048, 1024), (64, 512, 512), (2048, 512, 4096)])
def test_wait_probe_stops_the_8_bit_linear(moe, M, K, N):
    """The same in the cluster-split decode kernel and both widths of the large one."""
    g = gen(12)
    xq, xs = R.rand_rows(g, M, K)
    w, ws = R.rand_weights(g, 1, N, K)
    good = moe.linear_fp8(xq, xs, w[0], ws[0])
    wk = moe.workspace(256)
    y = torch.full((M, N), 2.0, dtype=torch.bfloat16, device="cuda")
    prev = moe.set_wait_probe(True)
    try:
        moe.linear_fp8(xq, xs, w[0], ws[0], out=y, ws=wk)
        assert moe.get_status(wk) == -6
    finally:
        moe.set_wait_probe(prev)
    assert (y == 2.0).all()
    moe.linear_fp8(xq, xs, w[0], ws[0], out=y, ws=wk)
    assert moe.get_status(wk) == 0 and torch.equal(bits(y), bits(good))


def test_fp8_calls_back_to_back_and_on_two_streams(moe):
    """Dependent calls without a synchronisation between them (each kernel is a
    programmatic dependent of the one before), and independent ones at once on
    two streams, each with its own workspace."""
    g = gen(13)
    S, E, d, F = 700, 6, 256, 128
    off, _ = offsets_of([100, 0, 300, 1, 99, 200])
    xq, xs, w = make_ffn(g, E, d, F, S, False)
    act = moe.ActConfig("silu")
    y = moe.expert_ffn_fp8(xq, xs, off, *w, act)
    torch.cuda.synchronize()
    chain = [y]
    for _ in range(4):  # the output, quantised, is the next input
        q, s = moe.quantize_fp8(chain[-1])
        chain.append(moe.expert_ffn_fp8(q, s, off, *w, act))
    torch.cuda.synchronize()
    for a, b in zip(chain, chain[1:]):
        torch.cuda.synchronize()
        q, s = moe.quantize_fp8(a)
        torch.cuda.synchronize()
        assert torch.equal(bits(b), bits(moe.expert_ffn_fp8(q, s, off, *w, act)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for st, o in zip(streams, outs):
            with torch.cuda.stream(st):
                o.append(moe.expert_ffn_fp8(xq, xs, off, *w, act))
    torch.cuda.synchronize()
    for o in outs:
        for t in o:
            assert torch.equal(bits(t), bits(y))


def test_linear_fp8_views_and_offsets_into_buffers(moe):
    """Row slices of larger tensors: contiguous, 16-byte aligned, not at the start
    of their allocation; the rows around the output stay as they were."""
    g = gen(14)
    xq, xs = R.rand_rows(g, 90, 272)
    w, ws = R.rand_weights(g, 3, 200, 272)
    out = torch.full((120, 200), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.linear_fp8(xq[7:77], xs[7:77], w[1], ws[1], out=out[20:90])
    ref, bound = R.product(xq[7:77], xs[7:77], w[1], ws[1])
    R.assert_within(out[20:90], ref, bound)
    assert (out[:20] == 9).all() and (out[90:] == 9).all()
    with pytest.raises(ValueError):
        moe.linear_fp8(xq[::2], xs[::2], w[1], ws[1])
    with pytest.raises(ValueError):
        moe.linear_fp8(xq, xs, w[1], ws[1][:, :2])


@pytest.mark.parametrize("counts", [[3, 2, 0, 1], [300, 40, 0, 200], [900, 40, 300, 200]])
def test_wait_probe_stops_the_8_bit_kernels(moe, counts):
    """The bounded wait that the diagnostics hook makes run out: an error status,
    outputs unwritten, and the next call as always."""
    off, S = offsets_of(counts)
    g = gen(11)
    xq, xs, w = make_ffn(g, 4, 256, 128, S, False)
    good = moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig("silu"))
    wk = moe.workspace(moe.lib().moe_expert_ffn_fp8_workspace_size(S, 256, 4, 128))
    y = torch.full((S, 256), 2.0, dtype=torch.bfloat16, device="cuda")
    prev = moe.set_wait_probe(True)
    try:
        moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig("silu"), y=y, ws=wk)
        assert moe.get_status(wk) == -6
    finally:
        moe.set_wait_probe(prev)
    assert (y == 2.0).all()
    moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig("silu"), y=y, ws=wk)
    assert moe.get_status(wk) == 0 and torch.equal(bits(y), bits(good))


def test_refusals_of_arguments(moe):
    """A flag that has no truth value, and more experts than the sort takes (before
    anything is allocated for them)."""
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="pow2_scales"):
        moe.quantize_fp8(x, pow2_scales=torch.ones(2))
    with pytest.raises(ValueError, match="pow2_scales"):
        moe.dispatch_fp8(idx, x, 8, pow2_scales=torch.ones(2))
    for E in (1025, 2 ** 31 - 1):
        with pytest.raises(moe.MoeError):
            moe.dispatch_fp8(idx, x, E)
