"""The 8-bit products, the MLP and the layer at the ends of their ranges: many
experts, empty and bad segments among many, offsets past 32 bits, no rows at all;
against 64 bits (tests/fp8_util.py derives the bounds)."""
import numpy as np
import pytest
import torch

from tests import fp8_util as R

pytestmark = pytest.mark.gpu

BEFORE = -3.0  # what outputs hold before a call


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import moe_routing_expert_fp32_b200 as m
    m.lib()
    return m


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def bits(t):
    return t.contiguous().view(torch.uint8)


def segments(E, mean, seed):
    """Ragged segments of about `mean` rows, empty ones at both ends and between."""
    rng = np.random.default_rng(seed)
    n = rng.integers(0, 2 * mean + 1, E)
    n[rng.random(E) < 0.1] = 0
    n[[0, 1, E - 1]] = 0
    n[2], n[E - 2] = mean, max(1, mean)
    off = np.concatenate([[0], np.cumsum(n)])
    return off.astype(np.int32)


def some_of(experts):
    """All of them, or of many both ends and every so many between."""
    n = len(experts)
    return experts if n <= 120 else [*experts[:30], *experts[30:-30:n // 60], *experts[-30:]]


def raw_weights(g, E, N, K):
    """Random e4m3 bytes (magnitudes up to 240, no NaN), for weights too large to draw."""
    q = torch.randint(0, 2 ** 31 - 1, (E * N * K // 4,), generator=g, device="cuda",
                      dtype=torch.int32)
    q.bitwise_and_(0x77777777)
    q = q.view(torch.uint8).view(torch.float8_e4m3fn).view(E, N, K)
    s = torch.rand(E, -(-N // 128), -(-K // 128), generator=g, device="cuda") + 0.5
    return q, s * 1e-4


def grouped_ref(xq, xs, off, w, ws, skip=()):
    """(y, bound) of the kept segments' rows; rows of none are 0 and infinite."""
    S, N = xq.shape[0], w.shape[1]
    y = torch.zeros(S, N, dtype=torch.float64, device="cuda")
    b = torch.full((S, N), float("inf"), dtype=torch.float64, device="cuda")
    for e in range(len(off) - 1):
        a, z = int(off[e]), int(off[e + 1])
        if a < z and e not in skip:
            y[a:z], b[a:z] = R.product(xq[a:z], xs[a:z], w[e], ws[e])
    return y, b


# ------------------------------------------------------------- many experts
# K, N, mean: the decode kernel, units of 128 columns, units of 256
@pytest.mark.parametrize("K,N,mean", [(144, 264, 1), (144, 264, 70), (1040, 512, 70)])
@pytest.mark.parametrize("E", [128, 129, 256, 384, 639, 640, 1024])
def test_grouped_many_segments(moe, E, K, N, mean):
    off = segments(E, mean, E)
    S = int(off[-1]) + 5
    g = gen(E + N)
    xq, xs = R.rand_rows(g, S, K)
    w, ws = R.rand_weights(g, E, N, K)
    out = torch.full((S, N), BEFORE, dtype=torch.bfloat16, device="cuda")
    wk = moe.workspace(256)
    moe.grouped_linear_fp8(xq, xs, torch.from_numpy(off).cuda(), w, ws, out=out, ws=wk)
    assert moe.get_status(wk) == 0
    assert (out[S - 5:] == BEFORE).all()
    ref, bound = grouped_ref(xq, xs, off, w, ws)
    R.assert_within(out[:S - 5], ref[:S - 5], bound[:S - 5])


@pytest.mark.parametrize("mean,act", [(1, "silu"), (70, "situ")])
@pytest.mark.parametrize("E,d,F", [(129, 272, 144), (256, 272, 144), (384, 528, 400),
                                   (640, 272, 144), (1024, 144, 80)])
def test_expert_ffn_many_segments(moe, E, d, F, mean, act):
    """The tile list of more than 128 segments in both gate/up kernels, and in the
    down kernels, which build it before the kernel in front of them has ended."""
    off = segments(E, mean, E + 1)
    S = int(off[-1]) + 3
    g = gen(E + d)
    xq, xs = R.rand_rows(g, S, d)
    w = [t for n, k in ((F, d), (F, d), (d, F)) for t in R.rand_weights(g, E, n, k)]
    beta, lbeta = (4.0, 8.0) if act == "situ" else (1.0, 0.0)
    y = torch.full((S, d), BEFORE, dtype=torch.bfloat16, device="cuda")
    wk = moe.workspace(moe.lib().moe_expert_ffn_fp8_workspace_size(S, d, E, F))
    moe.expert_ffn_fp8(xq, xs, torch.from_numpy(off).cuda(), *w,
                       moe.ActConfig(act, beta, lbeta), y=y, ws=wk)
    assert moe.get_status(wk) == 0
    assert (y[S - 3:] == BEFORE).all()
    for e in some_of(np.nonzero(np.diff(off))[0]):
        a, z = int(off[e]), int(off[e + 1])
        ref, bound = R.ffn(xq[a:z], xs[a:z], *[t[e] for t in w], act, beta, lbeta, False)
        R.assert_within(y[a:z], ref, bound, f"expert {e}")


@pytest.mark.parametrize("K,N,mean", [(144, 264, 1), (144, 264, 70), (1040, 512, 70)])
@pytest.mark.parametrize("E", [129, 256, 640, 700])
@pytest.mark.parametrize("kind", ["past the end", "negative", "backwards", "first"])
def test_grouped_bad_segment_among_many(moe, kind, E, K, N, mean):
    """One bad offset among more than 128 segments: the segments that it ends and
    begins are left out and recorded, the others are computed, nothing else is
    written."""
    off = segments(E, mean, E + 2)
    S = int(off[-1]) + 5
    at = {"past the end": E // 2, "negative": E - 3, "backwards": 131 if E > 131 else 100,
          "first": 0}[kind]
    while kind == "backwards" and not off[at - 1] < off[at] < off[at + 1]:
        at += 1
    skip = {at - 1, at}
    if kind == "backwards":  # from its own start on: segment at - 1 is empty of rows
        bad = int(off[at - 1]) - 1
        skip = {at - 1}
    else:
        bad = {"past the end": S + 3, "negative": -7, "first": 2}[kind]
    good = off.copy()
    off[at] = bad
    g = gen(E + N + at)
    xq, xs = R.rand_rows(g, S, K)
    w, ws = R.rand_weights(g, E, N, K)
    buf = torch.full((S + 64, N), BEFORE, dtype=torch.bfloat16, device="cuda")
    out = buf[32:32 + S]
    wk = moe.workspace(256)
    moe.grouped_linear_fp8(xq, xs, torch.from_numpy(off).cuda(), w, ws, out=out, ws=wk)
    assert moe.get_status(wk) == -7
    assert (buf[:32] == BEFORE).all() and (buf[32 + S:] == BEFORE).all()
    ref, bound = grouped_ref(xq, xs, off, w, ws, skip)
    if kind == "backwards":  # the row that segments at - 2 and at both hold may be either's
        bound[bad] = float("inf")
    kept = torch.isfinite(bound).all(1)
    assert kept.any()
    R.assert_within(out[kept], ref[kept], bound[kept])
    none = torch.ones(S, dtype=torch.bool, device="cuda")
    for e in range(E):
        if e not in skip:
            none[int(off[e]):int(off[e + 1])] = False
    assert (out[none] == BEFORE).all()
    off = good
    moe.grouped_linear_fp8(xq, xs, torch.from_numpy(off).cuda(), w, ws, out=out, ws=wk)
    assert moe.get_status(wk) == 0
    ref, bound = grouped_ref(xq, xs, off, w, ws)
    R.assert_within(out[:S - 5], ref[:S - 5], bound[:S - 5])


@pytest.mark.parametrize("E,mean", [(129, 1), (256, 70), (700, 1)])
def test_expert_ffn_bad_segment_among_many(moe, E, mean):
    """The same through the MLP: both products leave the segments out."""
    d, F = 272, 144
    off = segments(E, mean, E + 3)
    S = int(off[-1]) + 3
    at = E - 4
    off[at] = S + 9
    g = gen(E)
    xq, xs = R.rand_rows(g, S, d)
    w = [t for n, k in ((F, d), (F, d), (d, F)) for t in R.rand_weights(g, E, n, k)]
    buf = torch.full((S + 64, d), BEFORE, dtype=torch.bfloat16, device="cuda")
    y = buf[32:32 + S]
    wk = moe.workspace(moe.lib().moe_expert_ffn_fp8_workspace_size(S, d, E, F))
    moe.expert_ffn_fp8(xq, xs, torch.from_numpy(off).cuda(), *w, moe.ActConfig("silu"), y=y,
                       ws=wk)
    assert moe.get_status(wk) == -7
    none = torch.ones(S + 64, dtype=torch.bool, device="cuda")
    for e in range(E):
        a, z = int(off[e]), int(off[e + 1])
        if a < z and e not in (at - 1, at):
            none[32 + a:32 + z] = False
    for e in some_of([e for e in range(E) if off[e] < off[e + 1] and e not in (at - 1, at)]):
        a, z = int(off[e]), int(off[e + 1])
        ref, bound = R.ffn(xq[a:z], xs[a:z], *[t[e] for t in w], "silu", 1.0, 0.0, False)
        R.assert_within(y[a:z], ref, bound, f"expert {e}")
    assert (buf[none] == BEFORE).all()


# ------------------------------------------------------- offsets past 32 bits
def test_quantize_past_2_32_elements(moe):
    M, K = 700001, 6400
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.randn(1, K, generator=gen(1), device="cuda"))
    x.mul_(torch.linspace(0.5, 2.0, M, device="cuda")[:, None].to(torch.bfloat16))
    assert x.numel() > 2 ** 32
    for block_rows in (1, 128):
        q, s = moe.quantize_fp8(x, block_rows=block_rows)
        n = M // 128 * 128  # the last, partial block of rows among those compared
        for a, z in ((0, 256), (n // 2 // 128 * 128, n // 2 // 128 * 128 + 256), (n - 128, M)):
            qr, sr = R.quantize_ref(x[None, a:z], block_rows, False)
            assert torch.equal(q[a:z].float(), qr[0])
            assert torch.equal(s[a // block_rows:-(-z // block_rows)], sr[0])


def test_dispatch_past_2_32_elements(moe):
    N, K, E, d = 90000, 8, 16, 6400
    g = gen(2)
    x = torch.randn(N, d, generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.randint(0, E, (N, K), generator=g, device="cuda", dtype=torch.int32)
    counts, off, perm, pos, xq, xs = moe.dispatch_fp8(idx, x, E)
    assert xq.numel() > 2 ** 32
    flat = idx.reshape(-1).long()
    assert torch.equal(perm.long(), torch.sort(flat, stable=True).indices)
    assert torch.equal(counts.long(), torch.bincount(flat, minlength=E))
    for a in (0, N * K // 2, N * K - 500):
        qr, sr = R.quantize_ref(x[(perm[a:a + 500] // K).long()][None], 1, False)
        assert torch.equal(xq[a:a + 500].float(), qr[0]) and torch.equal(xs[a:a + 500], sr[0])


def test_linear_past_2_32_elements(moe):
    """Rows and outputs of more than 2^32 elements."""
    g = gen(3)
    M, K, N = 700000, 6400, 6400
    row_q, row_s = R.rand_rows(g, 1000, K)
    xq = row_q.view(torch.uint8).repeat(M // 1000, 1).view(torch.float8_e4m3fn)
    xs = row_s.repeat(M // 1000, 1)
    w, ws = R.rand_weights(g, 1, N, K)
    y = moe.linear_fp8(xq, xs, w[0], ws[0])
    assert xq.numel() > 2 ** 32 and y.numel() > 2 ** 32
    ref, bound = R.product(row_q, row_s, w[0], ws[0])
    for a in (0, M // 2, M - 1000):
        R.assert_within(y[a:a + 1000], ref, bound, f"row {a}")


@pytest.mark.parametrize("rows", [3, 200])
def test_grouped_weights_past_2_32_elements(moe, rows):
    E, N, K = 70, 8192, 8192
    w, ws = raw_weights(gen(4), E, N, K)
    assert w.numel() > 2 ** 32
    n = np.zeros(E, dtype=np.int64)
    n[[0, 31, 32, 33, 63, 64, 69]] = rows  # on both sides of 2^31 and of 2^32
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    xq, xs = R.rand_rows(gen(5), int(off[-1]), K)
    y = moe.grouped_linear_fp8(xq, xs, torch.from_numpy(off).cuda(), w, ws)
    ref, bound = grouped_ref(xq, xs, off, w, ws)
    R.assert_within(y, ref, bound)


@pytest.mark.parametrize("rows", [3, 200])
def test_expert_ffn_weights_past_2_32_elements(moe, rows):
    E, F, d = 260, 2064, 8192
    w1, w1s = raw_weights(gen(6), E, F, d)
    w3, w3s = raw_weights(gen(7), E, F, d)
    w2, w2s = raw_weights(gen(8), E, d, F)
    assert w1.numel() > 2 ** 32
    n = np.zeros(E, dtype=np.int64)
    n[[0, 126, 127, 128, 253, 254, 259]] = rows
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    xq, xs = R.rand_rows(gen(9), int(off[-1]), d)
    w = (w1, w1s, w3, w3s, w2, w2s)
    y = moe.expert_ffn_fp8(xq, xs, torch.from_numpy(off).cuda(), *w, moe.ActConfig("silu"))
    for e in np.nonzero(n)[0]:
        a, z = int(off[e]), int(off[e + 1])
        ref, bound = R.ffn(xq[a:z], xs[a:z], *[t[e] for t in w], "silu", 1.0, 0.0, False)
        R.assert_within(y[a:z], ref, bound, f"expert {e}")


def test_expert_ffn_rows_of_h_past_2_32_elements(moe):
    S, d, F, E = 2100000, 128, 2064, 2
    assert S * F > 2 ** 32
    row_q, row_s = R.rand_rows(gen(10), 1000, d)
    xq = row_q.view(torch.uint8).repeat(S // 1000, 1).view(torch.float8_e4m3fn)
    xs = row_s.repeat(S // 1000, 1)
    g = gen(11)
    w = [t for n, k in ((F, d), (F, d), (d, F)) for t in R.rand_weights(g, E, n, k)]
    off = torch.tensor([0, 1000000, S], dtype=torch.int32, device="cuda")
    y = moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig("situ", 4.0, 8.0))
    for a, e in ((0, 0), (999000, 0), (1000000, 1), (S - 1000, 1)):
        ref, bound = R.ffn(row_q, row_s, *[t[e] for t in w], "situ", 4.0, 8.0, False)
        R.assert_within(y[a:a + 1000], ref, bound, f"row {a}")


# ------------------------------------------------------------------ the layer
LAYERS = {
    # N, E, groups, kept groups, top_k, d_r, d_e, F, activation, pow2
    "one token": (1, 16, 4, 2, 4, 256, 256, 128, "silu", False),
    "no group step": (65, 384, 1, 1, 8, 512, 512, 144, "silu", True),
    "eight groups": (300, 256, 8, 4, 8, 256, 256, 128, "silu", False),
    "many slots": (9000, 384, 1, 1, 8, 256, 144, 80, "situ", True),
    "few experts": (3000, 8, 1, 1, 2, 256, 272, 400, "situ", False),
    "most experts": (40, 1024, 1, 1, 16, 128, 128, 16, "silu", False),
}


@pytest.mark.parametrize("name", list(LAYERS))
def test_layer_by_its_definition(moe, name):
    """forward_fp8 is its steps bit for bit, and each step follows the definition:
    the rows bit for bit, the MLP within its bound, the sum over k in fp32."""
    N, E, groups, keep, K, d_r, d_e, F, act, pow2 = LAYERS[name]
    g = gen(N + E)
    x = torch.randn(N, d_r, generator=g, device="cuda").to(torch.bfloat16)
    xe = x if d_e == d_r else torch.randn(N, d_e, generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn(E, d_r, generator=g, device="cuda") * 0.05
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    w = [t for n, k in ((F, d_e), (F, d_e), (d_e, F)) for t in R.rand_weights(g, E, n, k)]
    cfg = moe.RouteConfig(E, groups, keep, K, 2.5)
    beta, lbeta = (4.0, 8.0) if act == "situ" else (1.0, 0.0)
    a = moe.ActConfig(act, beta, lbeta)
    ws = moe.workspace(moe.forward_fp8_workspace_size(N, d_r, d_e, cfg, F))
    idx = torch.empty(N, K, dtype=torch.int32, device="cuda")
    tw = torch.empty(N, K, device="cuda")
    out = moe.forward_fp8(x, W, bias, cfg, *w, a, x_e=None if d_e == d_r else xe,
                          pow2_scales=pow2, ws=ws, topk_idx=idx, topk_w=tw)
    assert moe.get_status(ws) == 0
    i2, t2 = moe.route(x, W, bias, cfg)
    assert torch.equal(idx, i2) and torch.equal(tw, t2)
    counts, off, perm, pos, xq, xs = moe.dispatch_fp8(idx, xe, E, pow2_scales=pow2)
    y = moe.expert_ffn_fp8(xq, xs, off, *w, a, pow2_scales=pow2)
    assert torch.equal(bits(out), bits(moe.combine(y, pos, tw)))
    assert torch.equal(perm.long(), torch.sort(idx.reshape(-1).long(), stable=True).indices)
    qr, sr = R.quantize_ref(xe[None], 1, pow2)
    tok = (perm // K).long()
    assert torch.equal(xq.float(), qr[0][tok]) and torch.equal(xs, sr[0][tok])
    o = off.tolist()
    some = [e for e in range(E) if o[e] < o[e + 1]]
    for e in some[:6] + some[-6:]:
        r = slice(o[e], o[e + 1])
        ref, bound = R.ffn(xq[r], xs[r], *[t[e] for t in w], act, beta, lbeta, pow2)
        R.assert_within(y[r], ref, bound, f"expert {e}")
    terms = y.double()[pos.view(N, K).long()] * tw.double()[..., None]
    # K products and K sums in fp32, one rounding to bf16
    err = (2 * K) * R.U * terms.abs().sum(1)
    ref = terms.sum(1)
    R.assert_within(out, ref, err + R.BF16_HALF * (ref.abs() + err), "sum over k")


# -------------------------------------------------------------------- no rows
def test_calls_without_rows(moe):
    bf, f8, f32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
    e = lambda *s, dtype=bf: torch.empty(*s, dtype=dtype, device="cuda")
    g = gen(12)
    q, s = moe.quantize_fp8(e(0, 256))
    assert q.shape == (0, 256) and s.shape == (0, 2)
    q, s = moe.quantize_fp8(e(3, 0, 256), block_rows=128)
    assert q.shape == (3, 0, 256) and s.shape == (3, 0, 2)
    counts, off, perm, pos, xq, xs = moe.dispatch_fp8(e(0, 2, dtype=torch.int32), e(0, 256), 8)
    assert (counts == 0).all() and (off == 0).all() and off.shape == (9,)
    assert perm.numel() == pos.numel() == 0 and xq.shape == (0, 256) and xs.shape == (0, 2)
    w = [t for n, k in ((128, 256), (128, 256), (256, 128)) for t in R.rand_weights(g, 8, n, k)]
    assert moe.linear_fp8(xq, xs, w[0][0], w[1][0]).shape == (0, 128)
    assert moe.grouped_linear_fp8(xq, xs, off, w[0], w[1]).shape == (0, 128)
    assert moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig("silu")).shape == (0, 256)
    cfg = moe.RouteConfig(8, 1, 1, 2, 1.0)
    W = torch.zeros(8, 256, device="cuda")
    wk = moe.workspace(moe.forward_fp8_workspace_size(0, 256, 256, cfg, 128))
    assert moe.forward_fp8(e(0, 256), W, None, cfg, *w, moe.ActConfig("silu"), ws=wk).shape == (0, 256)
    assert moe.get_status(wk) == 0
    # rows, but none of them in a segment
    xq, xs = R.rand_rows(g, 5, 256)
    off = torch.zeros(9, dtype=torch.int32, device="cuda")
    y = torch.full((5, 256), BEFORE, dtype=bf, device="cuda")
    moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig("silu"), y=y)
    assert (y == BEFORE).all()


# --------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("counts", [[3, 2, 17, 30], [70, 1, 129, 300], [900, 40, 300, 260]])
def test_nonfinite_rows_stay_in_their_rows(moe, counts):
    """NaN and infinities in some rows, the last of a segment and the first of the
    next among them: every other row has the bits that it has without them, in the
    grouped product and through the MLP, whose h shares a scale per row only."""
    d, F, E = 272, 400, len(counts)
    o = np.concatenate([[0], np.cumsum(counts)])
    off = torch.from_numpy(o.astype(np.int32)).cuda()
    S = int(o[-1])
    g = gen(S)
    x = torch.randn(S, d, generator=g, device="cuda").to(torch.bfloat16)
    w = [t for n, k in ((F, d), (F, d), (d, F)) for t in R.rand_weights(g, E, n, k)]
    calls = [lambda q, s: moe.grouped_linear_fp8(q, s, off, w[0], w[1]),
             lambda q, s: moe.expert_ffn_fp8(q, s, off, *w, moe.ActConfig("silu")),
             lambda q, s: moe.expert_ffn_fp8(q, s, off, *w, moe.ActConfig("situ", 4.0, 8.0))]
    clean = [c(*moe.quantize_fp8(x)) for c in calls]
    bad = torch.zeros(S, dtype=torch.bool, device="cuda")
    for i, r in enumerate([0, int(o[1]) - 1, int(o[1]), int(o[2]), S - 1]):
        bad[r] = True
        x[r, (37 * i) % d] = float("nan") if i % 2 else float("inf")
    for c, was in zip(calls, clean):
        y = c(*moe.quantize_fp8(x))
        assert torch.isnan(y[bad]).all() and not torch.isnan(was).any()
        assert torch.equal(bits(y[~bad]), bits(was[~bad]))


@pytest.mark.parametrize("rows", [3, 300])
def test_nonfinite_weights_stay_with_their_expert(moe, rows):
    d, F, E = 272, 400, 3
    off = torch.arange(0, (E + 1) * rows, rows, dtype=torch.int32, device="cuda")
    g = gen(rows)
    xq, xs = R.rand_rows(g, E * rows, d)
    w = [t for n, k in ((F, d), (F, d), (d, F)) for t in R.rand_weights(g, E, n, k)]
    was = moe.grouped_linear_fp8(xq, xs, off, w[0], w[1])
    ffn = moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig("silu"))
    w[0].view(torch.uint8)[1, 255, 3] = 0x7f  # NaN in one weight row of expert 1
    y = moe.grouped_linear_fp8(xq, xs, off, w[0], w[1])
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[rows:2 * rows, 255] = True
    assert torch.isnan(y[hit]).all() and torch.equal(bits(y[~hit]), bits(was[~hit]))
    z = moe.expert_ffn_fp8(xq, xs, off, *w, moe.ActConfig("silu"))
    mine = slice(rows, 2 * rows)
    assert torch.isnan(z[mine]).all()
    z[mine], ffn[mine] = 0, 0
    assert torch.equal(bits(z), bits(ffn))
