"""The 8-bit block-scaled format in 64 bits, for the tests of the FP8 entry
points: quantisation by the definition, products, the expert MLP, and bounds
on what fp32 evaluation may differ by.

Bounds.  u = 2^-24 is half a step of fp32, 2^-8 half a step of bf16.  A product
of a K block is a sum of at most 128 exact e4m3 products held in fp32; each of
its additions may truncate, so the block is off by at most 128 * 2u times the
sum of the magnitudes.  The scale product, its multiplication and the addition
over the blocks round once each: (KB + 3) u more.  With A = sum |x| |w| this is
    |y32 - y64| <= ACC * A,  ACC = (256 + KB + 3) u,
and the bf16 result adds 2^-8 (|y64| + ACC A).
"""
import numpy as np
import torch

U = 2.0 ** -24
BF16_HALF = 2.0 ** -8
BLK = 128


def acc_bound(K):
    return (256 + -(-K // BLK) + 3) * U


def e4m3(v):
    """Nearest e4m3 (ties to even, magnitude at most 448; NaN stays), 64-bit in and out."""
    v = v.double()
    _, e = torch.frexp(v.abs())
    step = torch.exp2((e - 1).clamp(-6, 8).double() - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def scale_of(amax, pow2):
    """The fp32 scale of blocks with largest magnitude amax (fp32), as the definition has it."""
    a = amax.cpu().numpy().astype(np.float32)
    with np.errstate(all="ignore"):
        s = np.where(a < np.float32(2.0 ** -100), np.float32(2.0 ** -100), a) / np.float32(448.0)
        s = s.astype(np.float32)
        if pow2:
            m, e = np.frexp(s)
            up = np.ldexp(np.float32(1.0), np.where(m == 0.5, e - 1, e)).astype(np.float32)
            s = np.where(np.isfinite(s), up, s)
    return torch.from_numpy(s).to(amax.device)


def quantize_ref(x, block_rows, pow2):
    """(q as fp32 values, scale) of bf16 x [B, M, K]: fl32 steps of the definition."""
    B, M, K = x.shape
    p = torch.nn.functional.pad(x.float(), (0, -K % BLK, 0, -M % block_rows))
    b = p.view(B, p.shape[1] // block_rows, block_rows, p.shape[2] // BLK, BLK)
    amax = b.abs().amax(dim=(2, 4))
    s = scale_of(amax, pow2)
    inv = torch.from_numpy(np.float32(1.0) / s.cpu().numpy()).to(x.device)
    q = e4m3((b * inv[:, :, None, :, None]))  # the product is rounded to fp32
    q = q.reshape(p.shape)[:, :M, :K].float()
    return q, s


def deq_rows(q, s):
    return q.double() * s.double().repeat_interleave(BLK, -1)[..., :q.shape[-1]]


def deq_weights(q, s):
    s = s.double().repeat_interleave(BLK, -1)[..., :q.shape[-1]]
    return q.double() * s.repeat_interleave(BLK, -2)[..., :q.shape[-2], :]


def product(xq, xs, w, ws, res=None):
    """(y, bound) of one product in 64 bits."""
    x, wt = deq_rows(xq, xs), deq_weights(w, ws)
    y = x @ wt.t()
    err = acc_bound(x.shape[1]) * (x.abs() @ wt.abs().t())
    if res is not None:
        y = y + res.double()
        err = err + U * (y.abs() + err)  # the fp32 addition
    return y, err + BF16_HALF * (y.abs() + err)


# Relative error of the activations' fp32 functions: exp, reciprocal and tanh
# each within a few fp32 steps; e^2x - 1 is used from |x| = 0.125 on, where it is
# 0.22 of e^2x, so e^2x's 2^-22 becomes 1.1e-6 there, twice with two tanh; the
# argument of exp carries |g| u.
ACT_REL = 2.0 ** -18


def act64(g, u, kind, beta, lbeta):
    sig = 1.0 / (1.0 + torch.exp(-g))
    if kind == "silu":
        return g * sig * u
    up = lbeta * torch.tanh(u / lbeta) if lbeta else u
    return beta * torch.tanh(g / beta) * sig * up


def ffn(xq, xs, w1, w1s, w3, w3s, w2, w2s, kind, beta, lbeta, pow2):
    """(y, bound) of the expert MLP on the rows of one expert, 64 bits.

    h carries the errors of g and u through the activation (|d silu| <= 1.1,
    |d (beta tanh(g/beta) sigmoid(g))| <= 1 + beta/4); where that interval
    crosses a rounding border of the 8-bit format, h may land a step away, and
    that step times |w2| is added to the bound."""
    x = deq_rows(xq, xs)
    W1, W3, W2 = deq_weights(w1, w1s), deq_weights(w3, w3s), deq_weights(w2, w2s)
    c = acc_bound(x.shape[1])
    g, u = x @ W1.t(), x @ W3.t()
    eg, eu = c * (x.abs() @ W1.abs().t()), c * (x.abs() @ W3.abs().t())
    h = act64(g, u, kind, beta, lbeta)
    slope = 1.1 if kind == "silu" else 1.0 + abs(beta) / 4
    left = act64(g, torch.ones_like(u), kind, beta, 0.0).abs()
    umag = u.abs() if kind == "silu" or not lbeta else (lbeta * torch.tanh(u / lbeta)).abs()
    eh = slope * eg * (umag + eu) + left * eu + ACT_REL * h.abs()
    F = h.shape[1]
    pad = -F % BLK
    hb = torch.nn.functional.pad(h, (0, pad)).view(h.shape[0], -1, BLK)
    eb = torch.nn.functional.pad(eh, (0, pad)).view(h.shape[0], -1, BLK)
    amax = hb.abs().amax(2)
    lo_a = (hb.abs() - eb).amax(2)
    hi_a = (hb.abs() + eb).amax(2)
    s = scale_of(amax.float(), pow2).double()
    s_lo, s_hi = scale_of(lo_a.float(), pow2).double(), scale_of(hi_a.float(), pow2).double()
    q = e4m3(hb / s[..., None])
    deq = q * s[..., None]
    # the extremes over the interval of h and of the scale
    cand = [e4m3((hb + d * eb) * (1 + r * 4 * U) / t[..., None]) * t[..., None]
            for d in (-1, 1) for r in (-1, 1) for t in (s_lo, s_hi, s)]
    dev = torch.stack([(k - deq).abs() for k in cand]).amax(0)
    deq = deq.reshape(h.shape[0], -1)[:, :F]
    dev = dev.reshape(h.shape[0], -1)[:, :F]
    y = deq @ W2.t()
    err = dev @ W2.abs().t() + acc_bound(F) * ((deq.abs() + dev) @ W2.abs().t())
    return y, err + BF16_HALF * (y.abs() + err)


def rand_rows(g, M, K, pow2=False):
    """Quantised rows of differing sizes (q as e4m3 tensor, scale)."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x = (x * torch.exp(torch.randn(M, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    q, s = quantize_ref(x[None], 1, pow2)
    return q[0].to(torch.float8_e4m3fn), s[0]


def rand_weights(g, E, N, K):
    w = (torch.randn(E, N, K, generator=g, device="cuda") * 107).clamp(-448, 448)
    s = torch.rand(E, -(-N // BLK), -(-K // BLK), generator=g, device="cuda") + 0.5
    return w.to(torch.float8_e4m3fn), s * (0.02 / 107)


def assert_within(got, ref, bound, what=""):
    d = (got.double() - ref).abs()
    over = d > bound
    assert not torch.isnan(got).any(), what
    if over.any():
        i = torch.nonzero(over)[0].tolist()
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} outside, first at {i}: "
                             f"{got[tuple(i)].item()} for {ref[tuple(i)].item()} "
                             f"(bound {bound[tuple(i)].item():.3e})")
