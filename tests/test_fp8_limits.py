"""Sizes whose tiles and units the 8-bit products cannot count are refused on the
host, by every entry point that would come to them, before anything is enqueued."""
import ctypes

import pytest

OK = -8  # every argument taken: the next check is that of the device (there is none here)


@pytest.fixture(scope="module")
def m():
    from moe_routing_expert_fp32_b200 import build as b
    b.build()
    import moe_routing_expert_fp32_b200 as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_uint8 * 1024)()
    yield (ctypes.addressof(buf) + 255) // 256 * 256
    del buf


def fits(S, E, N):
    return (S // 32 + min(S, E)) * -(-N // 128) < 2 ** 31 and (S // 32 + 1) * E < 2 ** 31


HUGE = 1 << 62
TILES = 2 ** 31 // 1024 * 32 - 32  # 1024 segments: the first S whose tiles are not counted


@pytest.mark.parametrize("S,E,N", [
    (TILES - 32, 1024, 16), (TILES - 1, 1024, 16), (TILES, 1024, 16), (2 ** 31 - 1, 32, 16),
    (2 ** 31 - 1, 31, 16), (8000, 4, 2 ** 30), (8192, 4, 2 ** 30), (2 ** 31 - 1, 1, 4096),
    (2 ** 31 - 1, 1, 4224)])
def test_products(m, p, S, E, N, no_device):
    L = m.lib()
    want = OK if fits(S, E, N) else -2
    size = L.moe_grouped_linear_fp8_workspace_size(S, 16, E, N)
    assert (size > 0) == (want == OK)
    assert L.moe_grouped_linear_fp8(p, p, p, E, S, 16, p, p, N, p, p, HUGE, None) == want
    if E == 1:
        assert (L.moe_linear_fp8_workspace_size(S, 16, N) > 0) == (want == OK)
        assert L.moe_linear_fp8(p, p, S, 16, p, p, N, None, p, p, HUGE, None) == want


@pytest.mark.parametrize("S,E,d,F", [
    (TILES - 1, 1024, 16, 16), (TILES, 1024, 16, 16), (8000, 4, 2 ** 30, 16),
    (8192, 4, 2 ** 30, 16), (8192, 4, 16, 2 ** 30), (2 ** 31 - 1, 31, 128, 4096)])
def test_expert_mlp(m, p, S, E, d, F, no_device):
    """The down product's limit too, which the gate/up product does not reach."""
    L = m.lib()
    want = OK if fits(S, E, d) and fits(S, E, F) else -2
    assert (L.moe_expert_ffn_fp8_workspace_size(S, d, E, F) > 0) == (want == OK)
    w, act = m._Fp8Experts(p, p, p, p, p, p), m.ActConfig("silu")._c()
    assert L.moe_expert_ffn_fp8(p, p, p, E, S, d, F, ctypes.byref(w), ctypes.byref(act), 0, p, p,
                                HUGE, None) == want


@pytest.mark.parametrize("N,K,E,d,F", [(TILES // 16 - 1, 16, 1024, 32, 16),
                                       (TILES // 16, 16, 1024, 32, 16),
                                       (4000, 1, 8, 2 ** 30, 16), (7900, 1, 8, 2 ** 30, 16),
                                       (4000, 16, 16, 2 ** 30, 16)])
def test_layer(m, p, N, K, E, d, F, no_device):
    """The layer refuses before its router and its sort run."""
    L = m.lib()
    rows = N <= ROWS // -(-d // 128)
    want = OK if fits(N * K, E, d) and fits(N * K, E, F) and rows else -2
    cfg = m.RouteConfig(E, 1, 1, K, 1.0)._c()
    assert (L.moe_forward_fp8_workspace_size(N, 32, d, ctypes.byref(cfg), F) > 0) == (want == OK)
    w, act = m._Fp8Experts(p, p, p, p, p, p), m.ActConfig("silu")._c()
    assert L.moe_forward_fp8(p, p, N, 32, d, p, None, ctypes.byref(cfg), ctypes.byref(w), F,
                             ctypes.byref(act), 0, p, None, None, p, HUGE, None) == want


ROWS = (2 ** 31 - 1) * 16  # blocks of 128 columns of the rows that are quantised


@pytest.mark.parametrize("N,K,d,want", [
    (2 ** 27, 8, 2 ** 30, -2), (2 ** 27, 8, 128, OK), (ROWS // 2 ** 23, 8, 2 ** 30, OK),
    (ROWS // 2 ** 23 + 1, 8, 2 ** 30, -2), (2 ** 31 - 1, 1, 2048, OK), (2 ** 31 - 1, 1, 2064, -2)])
def test_rows_of_the_dispatch(m, p, N, K, d, want, no_device):
    """A grid that would not cover the rows is refused, as the quantisation's is."""
    L = m.lib()
    assert L.moe_dispatch_fp8(p, N, K, 16, p, d, 0, p, p, p, p, p, p, p, HUGE, None) == want
    assert L.moe_quantize_fp8(p, 1, N, d, 1, 0, p, p, None) == want
    cfg = m.RouteConfig(1024, 1, 1, K, 1.0)._c()
    if want != OK:
        assert L.moe_forward_fp8_workspace_size(N, 32, d, ctypes.byref(cfg), 16) == 0


@pytest.fixture
def no_device(monkeypatch):
    """These calls pass every check of their arguments, so they must not find a GPU."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("runs where there is no GPU")
