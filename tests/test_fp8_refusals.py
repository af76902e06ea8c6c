"""The 8-bit entry points refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def m():
    from moe_routing_expert_fp32_b200 import build as b
    b.build()
    import moe_routing_expert_fp32_b200 as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def mem():
    buf = (ctypes.c_uint8 * 8192)()
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    return buf, base


@pytest.mark.parametrize("B,M,K,rows,code", [
    (-1, 4, 128, 1, -1), (1, -4, 128, 1, -1), (1, 4, 0, 1, -1), (1, 4, 128, 64, -1),
    (1, 4, 120, 1, -2), (2 ** 40, 4, 128, 1, -2), (1, 2 ** 40, 128, 1, -2),
    (1, 4, 2 ** 30 + 16, 1, -2), (2 ** 31 - 1, 2 ** 31 - 1, 7168, 1, -2), (2 ** 31 - 1, 2 ** 31 - 1, 16, 128, -2),
    (1, 4, 128, 1, -1)])  # the last: null pointers
def test_quantize_refusals(m, B, M, K, rows, code):
    assert m.lib().moe_quantize_fp8(None, B, M, K, rows, 0, None, None, None) == code


def test_quantize_alignment(m, mem):
    _, p = mem
    L = m.lib()
    assert L.moe_quantize_fp8(p + 8, 1, 4, 128, 1, 0, p, p, None) == -3
    assert L.moe_quantize_fp8(p, 1, 4, 128, 1, 0, p + 8, p, None) == -3
    assert L.moe_quantize_fp8(p, 1, 4, 128, 1, 0, p, p + 2, None) == -3


@pytest.mark.parametrize("N,K,E,d,code", [
    (-1, 2, 4, 128, -1), (4, 0, 4, 128, -1), (4, 2, 0, 128, -1), (4, 2, 4, 0, -1),
    (4, 17, 32, 128, -2), (4, 2, 1025, 128, -2), (4, 2, 4, 136, -2),
    (2 ** 31 // 2, 2, 4, 128, -2), (2 ** 62, 16, 32, 128, -2), (4, 2, 4, 128, -1)])
def test_dispatch_refusals(m, N, K, E, d, code):
    n = None
    assert m.lib().moe_dispatch_fp8(n, N, K, E, n, d, 0, n, n, n, n, n, n, n, 0, n) == code


@pytest.mark.parametrize("S,K,E,N,code", [
    (-1, 128, 4, 128, -1), (4, 0, 4, 128, -1), (4, 128, 0, 128, -1), (4, 128, 4, 0, -1),
    (4, 136, 4, 128, -2), (4, 128, 1025, 128, -2), (4, 128, 4, 12, -2),
    (2 ** 31, 128, 4, 128, -2), (4, 2 ** 30 + 16, 4, 128, -2), (4, 128, 4, 2 ** 30 + 8, -2),
    (4, 128, 4, 128, -1)])
def test_grouped_refusals(m, S, K, E, N, code):
    L, n = m.lib(), None
    assert L.moe_grouped_linear_fp8(n, n, n, E, S, K, n, n, N, n, n, 0, n) == code
    size = L.moe_grouped_linear_fp8_workspace_size(S, K, E, N)
    assert (size >= 256) if (S, K, E, N) == (4, 128, 4, 128) else size == 0
    if E == 4 and code == -2:
        assert L.moe_linear_fp8(n, n, S, K, n, n, N, n, n, n, 0, n) == code
        assert L.moe_linear_fp8_workspace_size(S, K, N) == 0


def test_linear_pointers_alignment_and_workspace(m, mem):
    _, p = mem
    L = m.lib()

    def call(xq=p, xs=p, w=p, ws=p, res=None, y=p, wk=p, size=256):
        return L.moe_linear_fp8(xq, xs, 4, 128, w, ws, 128, res, y, wk, size, None)
    for k in ("xq", "xs", "w", "ws", "y"):
        assert call(**{k: None}) == -1, k
    for k in ("xq", "w", "y", "res"):
        assert call(**{k: p + 8}) == -3, k
    for k in ("xs", "ws"):
        assert call(**{k: p + 1}) == -3, k
    assert call(wk=None) == -4 and call(wk=p + 16) == -4 and call(size=255) == -4


def test_expert_ffn_refusals(m, mem):
    _, p = mem
    L = m.lib()
    ok_w = m._Fp8Experts(p, p, p, p, p, p)
    ok_a = m.ActConfig("silu")._c()

    def call(S=4, d=128, E=4, F=128, w=ok_w, act=ok_a, off=p, xq=p, y=p, wk=p, size=1 << 20):
        return L.moe_expert_ffn_fp8(xq, p, off, E, S, d, F,
                                    None if w is None else ctypes.byref(w),
                                    None if act is None else ctypes.byref(act), 0, y, wk, size,
                                    None)
    assert call(d=136) == -2 and call(F=24) == -2 and call(E=1025) == -2 and call(S=2 ** 31) == -2
    assert call(S=-1) == -1 and call(F=0) == -1 and call(d=-128) == -1
    assert call(w=None) == -1 and call(act=None) == -1 and call(off=None) == -1
    assert call(act=m._ActCfg(7, 1.0, 0.0)) == -1
    assert call(xq=None) == -1 and call(y=None) == -1 and call(y=p + 8) == -3
    assert call(w=m._Fp8Experts(p, None, p, p, p, p)) == -1
    assert call(w=m._Fp8Experts(p, p, p + 4, p, p, p)) == -3
    assert call(w=m._Fp8Experts(p, p, p, p, p + 2, p)) == -3
    need = L.moe_expert_ffn_fp8_workspace_size(4, 128, 4, 128)
    assert need >= 256 + 4 * 128 + 4 * 4
    assert call(size=need - 1) == -4
    assert L.moe_expert_ffn_fp8_workspace_size(4, 136, 4, 128) == 0


def test_forward_refusals(m, mem):
    _, p = mem
    L = m.lib()
    ok_w = m._Fp8Experts(p, p, p, p, p, p)
    act = m.ActConfig("silu")._c()

    def call(N=4, d_r=256, d_e=256, F=128, cfg=(16, 4, 2, 4, 2.5), xe=None, W=p, out=p, wk=None):
        c = m.RouteConfig(*cfg)._c()
        return L.moe_forward_fp8(p, xe, N, d_r, d_e, W, None, ctypes.byref(c),
                                 ctypes.byref(ok_w), F, ctypes.byref(act), 0, out, None, None, wk,
                                 1 << 30, None)
    assert call() == -4  # only the workspace is missing
    assert call(N=-1) == -1 and call(d_r=0) == -1 and call(d_e=512) == -1
    assert call(d_r=100, xe=p) == -2 and call(d_e=264, xe=p) == -2 and call(F=24) == -2
    assert call(N=2 ** 61) == -2
    assert call(cfg=(16, 3, 2, 4, 2.5)) == -1 and call(W=None) == -1 and call(out=None) == -1
    assert call(out=p + 8) == -3
    c = m.RouteConfig(16, 4, 2, 4, 2.5)._c()
    assert L.moe_forward_fp8_workspace_size(4, 256, 256, ctypes.byref(c), 24) == 0
    assert L.moe_forward_fp8_workspace_size(4, 256, 256, ctypes.byref(c), 128) > 0


def test_binding_refuses_wrong_tensors(m):
    """Wrong types, shapes, strides and places are refused in Python."""
    import torch
    f8 = torch.float8_e4m3fn
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.quantize_fp8(x)  # not on a GPU
    with pytest.raises(ValueError):
        m.quantize_fp8(x[0], block_rows=128)
    q, s = torch.zeros(4, 256, dtype=f8), torch.zeros(4, 2)
    w, ws = torch.zeros(8, 256, dtype=f8), torch.zeros(1, 2)
    for bad in ((q, s, w, ws), (q.float(), s, w, ws), (q, s[:, :1], w, ws)):
        with pytest.raises(ValueError):
            m.linear_fp8(*bad)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.grouped_linear_fp8(q, s, off, torch.zeros(2, 8, 256, dtype=f8), torch.zeros(2, 1, 2))
