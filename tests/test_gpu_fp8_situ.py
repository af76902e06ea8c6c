"""SiTU of the 8-bit expert MLP over the range of its two parameters, against 64 bits."""
import numpy as np
import pytest
import torch

from tests import fp8_util as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import moe_routing_expert_fp32_b200 as m
    m.lib()
    return m


def tanh_part(v, b):
    return b * torch.tanh(v / b) if b else v


def ffn(xq, xs, w1, w1s, w3, w3s, w2, w2s, beta, lbeta, steps=0.0):
    """(y, bound) of the MLP on one expert's rows, as fp8_util.ffn, with a slope that
    holds for any beta: the derivative of beta tanh(g/beta) sigmoid(g) is
    sech^2(g/beta) s + beta tanh(g/beta) s (1 - s), s = sigmoid(g); the first term is
    at most 1 and |beta tanh(g/beta)| at most |g|, and |g| s (1 - s) < 0.224.  The
    derivative of lbeta tanh(u/lbeta) is at most 1.  The left factor lies between
    -|beta| and |beta|, and where g is past 1000 beta it moves with its sigmoid alone,
    whose slope is at most 1/4.  What fp32 rounds (R.ACT_REL,
    relative) does not grow with either parameter; steps: what the left factor is off
    by where it is subnormal."""
    x = R.deq_rows(xq, xs)
    W1, W3, W2 = R.deq_weights(w1, w1s), R.deq_weights(w3, w3s), R.deq_weights(w2, w2s)
    c = R.acc_bound(x.shape[1])
    g, u = x @ W1.t(), x @ W3.t()
    eg, eu = c * (x.abs() @ W1.abs().t()), c * (x.abs() @ W3.abs().t())
    left, right = tanh_part(g, beta) / (1 + torch.exp(-g)), tanh_part(u, lbeta)
    h = left * right
    eleft = 1.224 * eg
    if beta:
        far = g.abs() - eg > 1e3 * abs(beta)
        eleft = torch.minimum(eleft, torch.where(far, abs(beta) / 4 * eg, 2 * abs(beta)))
    eh = eleft * (right.abs() + eu) + left.abs() * eu + R.ACT_REL * h.abs()
    eh = eh + steps * right.abs()
    hb, eb = h.view(h.shape[0], -1, R.BLK), eh.view(h.shape[0], -1, R.BLK)
    scales = [R.scale_of((hb.abs() + d * eb).amax(2).float(), False).double() for d in (0, -1, 1)]
    deq = R.e4m3(hb / scales[0][..., None]) * scales[0][..., None]
    dev = torch.stack([
        (R.e4m3((hb + d * eb) * (1 + r * 4 * R.U) / t[..., None]) * t[..., None] - deq).abs()
        for d in (-1, 1) for r in (-1, 1) for t in scales]).amax(0)
    deq, dev = deq.view(h.shape), dev.view(h.shape)
    y = deq @ W2.t()
    err = dev @ W2.abs().t() + R.acc_bound(h.shape[1]) * ((deq.abs() + dev) @ W2.abs().t())
    return y, err + R.BF16_HALF * (y.abs() + err)


def check(moe, counts, beta, lbeta, sizes):
    """sizes: (of g, of u), factors on rows of deviation about 16 * 0.02 a column."""
    beta, lbeta = float(np.float32(beta)), float(np.float32(lbeta))
    g = torch.Generator(device="cuda")
    g.manual_seed(17)
    S, E, d, F = sum(counts), len(counts), 256, 256
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    xq, xs = R.rand_rows(g, S, d)
    w1, w1s = R.rand_weights(g, E, F, d)
    w3, w3s = R.rand_weights(g, E, F, d)
    w2, w2s = R.rand_weights(g, E, d, F)
    for by_g, by_u in sizes:
        v = (w1, w1s * by_g, w3, w3s * by_u, w2, w2s)
        y = moe.expert_ffn_fp8(xq, xs, off, *v, moe.ActConfig("situ", beta, lbeta))
        a = 0
        for e, n in enumerate(counts):
            ref, bound = ffn(xq[a:a + n], xs[a:a + n], *[t[e] for t in v], beta, lbeta)
            R.assert_within(y[a:a + n], ref, bound, f"sizes {by_g} {by_u}, expert {e}")
            a += n


@pytest.mark.parametrize("counts", [[5, 29], [300, 200]])
@pytest.mark.parametrize("beta,lbeta", [(1e20, 1e20), (-1e20, 1e20), (3e38, 3e38), (1e30, 1e10),
                                        (3e38, 0.0), (1e20, 8.0), (4.0, 1e30)])
def test_large_parameters(moe, counts, beta, lbeta):
    """Limits that ordinary arguments never reach: g sigmoid(g) u, whatever the
    product of the two parameters is."""
    check(moe, counts, beta, lbeta, [(1.0, 1.0), (0.01, 20.0), (20.0, 0.01)])


@pytest.mark.parametrize("counts", [[5, 29], [300, 200]])
@pytest.mark.parametrize("beta,lbeta,by", [(1e15, 1e15, 1e15), (1e15, 1e12, 1e15), (1e12, 1e15, 1e14)])
def test_large_parameters_that_are_reached(moe, counts, beta, lbeta, by):
    """Arguments of the size of the limits, on both sides of the series' border."""
    check(moe, counts, beta, lbeta, [(by, by), (0.1 * by, by), (by, 0.1 * by), (10 * by, 10 * by)])


@pytest.mark.parametrize("counts", [[5, 29], [300, 200]])
@pytest.mark.parametrize("beta,lbeta", [(2e-39, 0.0), (-1e-39, 0.0), (1e-39, 1e35)])
def test_subnormal_parameters(moe, counts, beta, lbeta):
    """A limit whose inverse is past fp32, on gates that are zero (h = 0) and on gates
    that it saturates.  beta is on the grid of 2^-149: each of at most four products
    of its size rounds by half a step of that, times u."""
    beta, lbeta = float(np.float32(beta)), float(np.float32(lbeta))
    g = torch.Generator(device="cuda")
    g.manual_seed(23)
    S, E, d, F = sum(counts), len(counts), 256, 256
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    xq, xs = R.rand_rows(g, S, d)
    xq[::7] = 0  # rows whose g and u are 0
    w1, w1s = R.rand_weights(g, E, F, d)
    w1[:, ::5] = 0  # columns whose g is 0
    w3, w3s = R.rand_weights(g, E, F, d)
    w3s = w3s * 1e35
    w2, w2s = R.rand_weights(g, E, d, F)
    y = moe.expert_ffn_fp8(xq, xs, off, w1, w1s, w3, w3s, w2, w2s,
                           moe.ActConfig("situ", beta, lbeta))
    a = 0
    for e, n in enumerate(counts):
        rows = (xq[a:a + n], xs[a:a + n])
        w = (w1[e], w1s[e], w3[e], w3s[e], w2[e], w2s[e])
        ref, bound = ffn(*rows, *w, beta, lbeta, steps=4 * 2.0 ** -150)
        R.assert_within(y[a:a + n], ref, bound, f"expert {e}")
        assert (ref != 0).any() and (y[a:a + n][rows[0].float().eq(0).all(1)] == 0).all()
        a += n
