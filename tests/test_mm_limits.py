"""Limits of the grouped products, weight gradients and their workspaces,
answered from scalars and pointers alone (nothing is launched)."""
from routed_grouped_gemm_amd import _lib

F = 0x1000                                          # stands for a device pointer; never dereferenced
OK, NULL, SHAPE, UNSUP, WS = (_lib.MOE_OK, _lib.MOE_ERR_NULL, _lib.MOE_ERR_SHAPE, _lib.MOE_ERR_UNSUPPORTED,
                              _lib.MOE_ERR_WORKSPACE)
BF16, F16 = _lib.MOE_T_BF16, _lib.MOE_T_F16


def mm(R=64, N=256, K=128, G=4, src=None, ws=F, ws_bytes=1 << 40, x_rows=None):
    return _lib.load().moe_grouped_mm(F, R if x_rows is None else x_rows, K, src, F, BF16, F, R, N, K, G, 0, F, N, ws,
                                      ws_bytes, None)


def fp8(R=64, N=256, K=128, G=4, src=None, ws=F, ws_bytes=1 << 40, x_rows=None):
    return _lib.load().moe_grouped_mm_fp8(F, F, R if x_rows is None else x_rows, src, F, F, F, R, N, K, G, BF16, F, N,
                                          ws, ws_bytes, None)


def wgrad(R=64, N=256, K=128, G=4, src=None, xs=None, ws=F, ws_bytes=1 << 40, x_rows=None):
    return _lib.load().moe_grouped_wgrad(F, R, N, None, F, R if x_rows is None else x_rows, K, src, xs, BF16, F, R, N,
                                         K, G, 0, F, ws, ws_bytes, None)


def test_rows_past_the_limit():
    """Row counts that 32-bit arithmetic on the device does not hold (a tile more
    than the rows, four bytes a source) are refused, with and without sources."""
    lib = _lib.load()
    most = _lib.MOE_MM_MAX_ROWS
    assert most == 2**29 - 1
    for R in (most + 1, 1 << 30, 2**31 - 64, 2**31 - 1):
        for src in (None, F):
            at = dict(R=R, N=8, K=16, G=1, src=src, x_rows=64 if src else R)
            assert mm(**at) == SHAPE and fp8(**at) == SHAPE, (R, src)
            assert wgrad(**at) == SHAPE and wgrad(xs=F, **at) == SHAPE, (R, src)
        for f in (lib.moe_grouped_mm_workspace_size, lib.moe_grouped_wgrad_workspace_size,
                  lib.moe_grouped_mm_fp8_workspace_size):
            assert f(R, 1, 64, 64) == 0


def test_workspace_is_checked():
    """A call that splits its sums refuses a workspace that is missing, too small
    or not at a multiple of 16 bytes (partial sums go there 16 bytes at a time)."""
    lib = _lib.load()
    few = dict(R=16, G=1, N=1024, K=4096)            # few tiles: split
    need = {mm: lib.moe_grouped_mm_workspace_size(16, 1, 1024, 4096),
            fp8: lib.moe_grouped_mm_fp8_workspace_size(16, 1, 1024, 4096)}
    one = dict(R=16384, G=1, N=256, K=256)
    need[wgrad] = lib.moe_grouped_wgrad_workspace_size(16384, 1, 256, 256)
    for f, at in ((mm, few), (fp8, few), (wgrad, one)):
        assert need[f] > 0
        assert f(ws=None, ws_bytes=need[f], **at) == WS and f(ws_bytes=need[f] - 1, **at) == WS, f.__name__
        assert f(ws=None, ws_bytes=0, **at) == WS
        for odd in (1, 4, 8):
            assert f(ws=F + odd, ws_bytes=need[f] + 16, **at) == SHAPE, (f.__name__, odd)


def test_plans():
    """Pure host functions: a tile height, a split only of few-row tiles, a
    workspace exactly where something is split, and refusals as the calls'."""
    import ctypes as C

    lib = _lib.load()
    rows, parts, part = C.c_int32(), C.c_int32(), C.c_int32()
    out = C.byref(rows), C.byref(parts)
    seen = set()
    for f, size in ((0, lib.moe_grouped_mm_workspace_size), (1, lib.moe_grouped_mm_fp8_workspace_size)):
        for R in (0, 1, 16, 300, 2600, 9000, 100000):
            for G in (1, 8, 40, 2049):
                for N, K in ((8, 16), (264, 528), (2056, 336), (4096, 7168)):
                    assert lib.moe_grouped_mm_plan(R, G, N, K, f, *out) == OK
                    assert rows.value in (32, 64, 128, 256) and parts.value >= 1
                    assert parts.value == 1 or rows.value <= 64
                    assert (size(R, G, N, K) > 0) == (parts.value > 1 and R > 0)
                    seen.add((f, rows.value, parts.value > 1))
        assert {r for g, r, _ in seen if g == f} == {32, 64, 128, 256}
        assert lib.moe_grouped_mm_plan(64, 4, 252, 128, f, *out) == SHAPE
        assert lib.moe_grouped_mm_plan(64, 4, 256, 128, f, None, out[1]) == NULL
        assert lib.moe_grouped_mm_plan(64, 4, 256, 128, f, out[0], None) == NULL
    assert lib.moe_grouped_mm_plan(64, 4, 256, 136, 1, *out) == SHAPE
    for R in (0, 1, 64, 5000, 16384):
        for G in (1, 8, 2049):
            for N, K in ((8, 8), (256, 256), (2816, 2048)):
                assert lib.moe_grouped_wgrad_plan(R, G, N, K, C.byref(part)) == OK
                assert part.value % 64 == 0 and 0 <= part.value < max(R, 1) + 64
                assert (lib.moe_grouped_wgrad_workspace_size(R, G, N, K) > 0) == (part.value > 0)
    assert lib.moe_grouped_wgrad_plan(64, 0, 256, 256, C.byref(part)) == SHAPE
    assert lib.moe_grouped_wgrad_plan(64, 4, 256, 256, None) == NULL
