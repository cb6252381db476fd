"""The plan query of the products with an epilogue answers from sizes alone (no GPU needed)."""
import ctypes as C

from routed_grouped_gemm_amd import _lib

lib = _lib.load()
GATED = _lib.MOE_MM_GATED
OK, NULL, SHAPE, UNSUP = _lib.MOE_OK, _lib.MOE_ERR_NULL, _lib.MOE_ERR_SHAPE, _lib.MOE_ERR_UNSUPPORTED


def plan(*a):
    p = (C.c_int32 * 6)()
    assert lib.moe_grouped_mm_act_plan(*a, p) == OK
    return list(p)


def test_refusals():
    p = (C.c_int32 * 6)()
    call = lib.moe_grouped_mm_act_plan
    assert call(64, 4, 256, 128, 0, None) == NULL
    assert call(64, 4, 256, 128, _lib.MOE_MM_W_KN, p) == UNSUP
    assert call(-1, 4, 256, 128, 0, p) == SHAPE and call(64, 0, 256, 128, 0, p) == SHAPE and call(64, 4, 252, 128, 0, p) == SHAPE
    assert call(64, 4, 264, 128, GATED, p) == SHAPE          # N % 16
    assert call(64, 4, 264, 128, 0, p) == OK and call(0, 1, 8, 8, 0, p) == OK


def test_plans_are_those_of_the_kernels():
    """Tiles that exist, tails of one group only, whole launches split where tiles are of 32 or 64 rows,
    and workspaces that hold the parts."""
    tails = set()
    for R in (0, 1, 40, 300, 2000, 4099, 8256, 20000, 100001):
        for G in (1, 2, 17, 2049):
            for N in (8, 520, 4104, 4160, 16384):
                for K in (8, 136, 4096):
                    for flags in (0, GATED) if N % 16 == 0 else (0,):
                        rows, parts, rr, rp, cr, cp = plan(R, G, N, K, flags)
                        assert rows in (32, 64, 128, 256) and parts >= 1 and (parts == 1 or rows <= 64)
                        for r, n in ((rr, rp), (cr, cp)):
                            assert (r, n) == (0, 0) or (G == 1 and rows >= 128 and r in (32, 64) and n >= 1)
                        if not flags:
                            need = max(parts * R * N if parts > 1 else 0, rp * rows * N if rp > 1 else 0)
                            assert lib.moe_grouped_mm_act_workspace_size(R, G, N, K) >= 4 * need
                            assert lib.moe_grouped_mm_dact_workspace_size(R, G, N, K) >= 4 * need
                        tails |= {rr, cr}
    assert tails == {0, 32, 64}
