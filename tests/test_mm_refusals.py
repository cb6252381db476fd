"""What the grouped products, the block quantisers and the checkpointed
activation refuse, answered from scalars and pointers alone (nothing is
launched: a call that passed its checks would fault on these pointers)."""
import ctypes as C

import pytest

from routed_grouped_gemm_amd import _lib

F = 0x1000                                          # stands for a device pointer; never dereferenced
OK, NULL, SHAPE, UNSUP, WS = (_lib.MOE_OK, _lib.MOE_ERR_NULL, _lib.MOE_ERR_SHAPE, _lib.MOE_ERR_UNSUPPORTED,
                              _lib.MOE_ERR_WORKSPACE)
BF16, F16, F32 = _lib.MOE_T_BF16, _lib.MOE_T_F16, _lib.MOE_T_F32


def test_grouped_mm():
    lib = _lib.load()

    def call(x=F, x_rows=64, ldx=128, src=None, w=F, dtype=BF16, off=F, R=64, N=256, K=128, G=4, flags=0, y=F,
             ldy=256, ws=F, ws_bytes=1 << 40):
        return lib.moe_grouped_mm(x, x_rows, ldx, src, w, dtype, off, R, N, K, G, flags, y, ldy, ws, ws_bytes, None)

    assert call(dtype=F32) == UNSUP and call(dtype=7) == UNSUP
    assert call(flags=_lib.MOE_WGRAD_F32) == UNSUP
    assert call(N=4) == SHAPE and call(N=252) == SHAPE and call(K=132, ldx=136) == SHAPE and call(K=0) == SHAPE
    assert call(N=(1 << 20) + 8, ldy=1 << 21) == SHAPE
    assert call(G=0) == SHAPE and call(G=2050) == SHAPE and call(R=-1) == SHAPE
    assert call(ldx=120) == SHAPE and call(ldx=132) == SHAPE and call(ldx=(1 << 22) + 8) == SHAPE
    assert call(ldy=248) == SHAPE and call(ldy=258) == SHAPE
    assert call(x_rows=63) == SHAPE                 # fewer rows than R_max, and no sources
    assert call(x_rows=0, src=F) == SHAPE
    assert call(x_rows=1 << 24, src=F) == SHAPE     # a gathered array of 4 GiB
    assert call(x=None) == NULL and call(w=None) == NULL and call(off=None) == NULL and call(y=None) == NULL
    assert call(x=F + 8) == SHAPE and call(w=F + 8) == SHAPE and call(y=F + 4) == SHAPE
    assert call(R=0, x=None, x_rows=0, w=None, off=None, y=None) == OK


def test_grouped_wgrad():
    lib = _lib.load()

    def call(dy=F, dy_rows=64, ld_dy=256, dsrc=None, x=F, x_rows=64, ldx=128, xsrc=None, xs=None, dtype=BF16, off=F,
             R=64, N=256, K=128, G=4, flags=0, dw=F, ws=F, ws_bytes=1 << 40):
        return lib.moe_grouped_wgrad(dy, dy_rows, ld_dy, dsrc, x, x_rows, ldx, xsrc, xs, dtype, off, R, N, K, G,
                                     flags, dw, ws, ws_bytes, None)

    assert call(dtype=F32) == UNSUP and call(flags=_lib.MOE_MM_W_KN) == UNSUP
    assert call(xs=F, dtype=F16) == UNSUP           # 8-bit rows are decoded to bf16
    assert call(xs=F, ldx=132) == SHAPE and call(xs=F, x=F + 4) == SHAPE and call(xs=F, x_rows=10) == SHAPE
    assert call(xs=F, x=None) == NULL
    assert call(N=252) == SHAPE and call(K=132, ldx=136) == SHAPE and call(G=0) == SHAPE and call(R=-1) == SHAPE
    assert call(dy_rows=63) == SHAPE and call(x_rows=63) == SHAPE
    assert call(dy_rows=1 << 24, dsrc=F) == SHAPE and call(x_rows=1 << 25, xsrc=F) == SHAPE
    assert call(ld_dy=248) == SHAPE and call(ldx=120) == SHAPE
    assert call(dy=None) == NULL and call(x=None) == NULL and call(off=None) == NULL and call(dw=None) == NULL
    assert call(dw=F + 8, flags=_lib.MOE_WGRAD_F32) == SHAPE and call(dw=F + 4) == SHAPE
    assert call(dy=F + 2) == SHAPE and call(x=F + 8) == SHAPE


def test_workspace_sizes():
    """Pure host functions, defined at every size: 0 where nothing is split or
    the sizes are refused, bounded where a product is."""
    lib = _lib.load()
    for f in (lib.moe_grouped_mm_workspace_size, lib.moe_grouped_wgrad_workspace_size,
              lib.moe_grouped_mm_fp8_workspace_size):
        assert f(0, 4, 256, 128) == 0
        assert f(-1, 4, 256, 128) == 0 and f(64, 0, 256, 128) == 0 and f(64, 4, 250, 128) == 0
        for R in (1, 15, 64, 1000, 16384, 1 << 20):
            for G in (1, 8, 2049):
                for N, K in ((8, 16), (256, 256), (4096, 7168), (1 << 20, 1 << 20)):
                    assert f(R, G, N, K) < 1 << 38, (R, G, N, K)
    assert lib.moe_grouped_mm_workspace_size(16, 1, 1024, 7168) > 0
    assert lib.moe_grouped_mm_workspace_size(16384, 8, 4096, 4096) == 0
    assert lib.moe_grouped_wgrad_workspace_size(16384, 1, 256, 256) > 0
    assert lib.moe_grouped_wgrad_workspace_size(4096, 64, 4096, 4096) == 0


def test_quantisers():
    lib = _lib.load()

    def rows(x=F, dtype=BF16, R=4, K=256, ld=256, q=F, s=F):
        return lib.moe_quantize_block(x, dtype, R, K, ld, None, q, s, None)

    assert rows(dtype=3) == UNSUP
    assert rows(K=252) == SHAPE and rows(K=0) == SHAPE and rows(ld=248) == SHAPE and rows(R=-1) == SHAPE
    assert rows(ld=260) == SHAPE and rows(ld=258, dtype=F32) == SHAPE
    assert rows(x=F + 8) == SHAPE and rows(q=F + 4) == SHAPE
    assert rows(x=None) == NULL and rows(q=None) == NULL and rows(s=None) == NULL
    assert rows(R=0, x=None, q=None, s=None) == OK

    def weights(w=F, dtype=BF16, G=2, N=100, K=256, q=F, s=F):
        return lib.moe_quantize_block_weights(w, dtype, G, N, K, q, s, None)

    assert weights(dtype=-1) == UNSUP
    assert weights(N=0) == SHAPE and weights(K=4) == SHAPE and weights(G=-1) == SHAPE and weights(G=2050) == SHAPE
    assert weights(w=None) == NULL and weights(q=None) == NULL and weights(s=None) == NULL
    assert weights(w=F + 8) == SHAPE
    assert weights(G=0, w=None, q=None, s=None) == OK


def test_grouped_mm_fp8():
    lib = _lib.load()

    def call(x=F, xs=F, x_rows=64, src=None, w=F, ws_=F, off=F, R=64, N=256, K=128, G=4, dtype=BF16, y=F, ldy=256,
             ws=F, ws_bytes=1 << 40):
        return lib.moe_grouped_mm_fp8(x, xs, x_rows, src, w, ws_, off, R, N, K, G, dtype, y, ldy, ws, ws_bytes, None)

    assert call(dtype=F32) == UNSUP
    assert call(K=136) == SHAPE and call(N=252) == SHAPE and call(G=0) == SHAPE and call(ldy=250) == SHAPE
    assert call(x_rows=63) == SHAPE and call(x_rows=1 << 25, src=F) == SHAPE
    for name in ("x", "xs", "w", "ws_", "off", "y"):
        assert call(**{name: None}) == NULL, name
    assert call(x=F + 8) == SHAPE and call(w=F + 8) == SHAPE and call(y=F + 4) == SHAPE
    assert call(R=0, x=None, x_rows=0) == OK


def test_checkpointed_activation():
    lib = _lib.load()

    def fwd(pre=F, dtype=BF16, R=4, I=128, ld=256, epi=None, h=F, q=F, s=F):
        return lib.moe_glu_checkpoint(pre, dtype, R, I, ld, None, None, None if epi is None else C.byref(epi), h, q,
                                      s, None)

    def bwd(q=F, s=F, dh=F, dtype=BF16, R=4, I=128, ld=128, epi=None, dpre=F, h=F, dw=F):
        return lib.moe_glu_checkpoint_backward(q, s, dh, dtype, R, I, ld, None, None,
                                               None if epi is None else C.byref(epi), dpre, h, dw, None)

    assert fwd(dtype=F32) == UNSUP and bwd(dtype=F32) == UNSUP
    assert fwd(I=132, ld=264) == SHAPE and fwd(ld=248) == SHAPE and fwd(ld=260) == SHAPE and fwd(R=-1) == SHAPE
    assert bwd(I=132, ld=136) == SHAPE and bwd(ld=120) == SHAPE and bwd(ld=132) == SHAPE and bwd(R=-1) == SHAPE
    assert fwd(q=None) == NULL and fwd(s=None) == NULL and fwd(pre=None) == NULL and fwd(h=None) == NULL
    assert bwd(q=None) == NULL and bwd(s=None) == NULL and bwd(dh=None) == NULL and bwd(dpre=None) == NULL
    assert fwd(pre=F + 8) == SHAPE and fwd(h=F + 8) == SHAPE and fwd(q=F + 4) == SHAPE
    assert bwd(dh=F + 8) == SHAPE and bwd(dpre=F + 8) == SHAPE and bwd(h=F + 8) == SHAPE and bwd(q=F + 4) == SHAPE
    for f in (fwd, bwd):
        assert f(epi=_lib.moe_epilogue(9, 1.0, 0.0, 0, None, None)) == UNSUP
        assert f(epi=_lib.moe_epilogue(0, 1.0, 0.0, 0, F, None)) == UNSUP           # a bias
        assert f(epi=_lib.moe_epilogue(0, 1.0, 0.0, 0, None, F)) == UNSUP           # a pre-activation copy
        assert f(epi=_lib.moe_epilogue(0, 0.0, 0.0, 0, None, None)) == SHAPE
        assert f(epi=_lib.moe_epilogue(0, 1.0, float("inf"), 0, None, None)) == SHAPE
    assert fwd(R=0, pre=None, h=None, q=None, s=None) == OK
    assert bwd(R=0, q=None, s=None, dh=None, dpre=None, h=None, dw=None) == OK


def test_bindings_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    import routed_grouped_gemm_amd as moe

    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    for f in (lambda: moe.moe_grouped_mm(x, torch.zeros((1, 8, 16), dtype=torch.bfloat16), off),
              lambda: moe.moe_grouped_wgrad(x, x, off),
              lambda: moe.moe_quantize_block(x),
              lambda: moe.moe_quantize_block_weights(x[None]),
              lambda: moe.moe_grouped_mm_fp8(x.byte(), x.float(), x.byte()[None], x.float(), off),
              lambda: moe.moe_glu_checkpoint(x),
              lambda: moe.moe_glu_checkpoint_backward(x.byte(), x.float(), x)):
        with pytest.raises(moe.MoeError):
            f()
