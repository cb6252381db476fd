"""What the layer for a few tokens, the bias gradients and the router's
gradient refuse, answered from scalars and pointers alone (nothing is launched:
a call that passed its checks would fault on these pointers)."""
import ctypes as C

import pytest

from routed_grouped_gemm_amd import _lib

F = 0x1000                                          # stands for a device pointer; never dereferenced
OK, NULL, SHAPE, UNSUP, WS = (_lib.MOE_OK, _lib.MOE_ERR_NULL, _lib.MOE_ERR_SHAPE, _lib.MOE_ERR_UNSUPPORTED,
                              _lib.MOE_ERR_WORKSPACE)
BF16, F16, F32 = _lib.MOE_T_BF16, _lib.MOE_T_F16, _lib.MOE_T_F32


def test_layer_few():
    lib = _lib.load()

    def call(ws=F, ws_bytes=1 << 30, epi=None, **kw):
        a = dict(logits=F, T=4, E_tot=8, k=2, e0=0, E_loc=8, dtype=BF16, x=F, ldx=256, H=256, I=128, flags=0, w1=F, w2=F,
                 out=F, ld_out=256)
        a.update(kw)
        args = _lib.moe_few_args()
        for n, v in a.items():
            setattr(args, n, v)
        if epi is not None:
            args.epi = C.pointer(epi)
        return lib.moe_layer_few(C.byref(args), ws, ws_bytes, None)

    assert lib.moe_layer_few(None, F, 1 << 30, None) == NULL
    assert call(dtype=F32) == UNSUP and call(flags=_lib.MOE_WEIGHT_AT_COMBINE) == UNSUP
    assert call(epi=_lib.moe_epilogue(4, 1.0, 0.0, 0, None, None)) == UNSUP
    assert call(epi=_lib.moe_epilogue(0, 1.0, 0.0, 0, None, F)) == UNSUP            # a pre-activation copy
    assert call(epi=_lib.moe_epilogue(0, 0.0, 0.0, 0, None, None)) == SHAPE
    assert call(epi=_lib.moe_epilogue(0, 1.0, -1.0, 0, None, None)) == SHAPE
    assert call(T=33) == SHAPE and call(T=-1) == SHAPE and call(k=0) == SHAPE and call(k=9) == SHAPE
    assert call(k=33, E_tot=64) == SHAPE and call(k=32, E_tot=64, shared_w1=F, shared_w2=F) == SHAPE
    assert call(E_loc=0) == SHAPE and call(e0=-1) == SHAPE and call(e0=2041) == SHAPE and call(E_tot=2049) == SHAPE
    assert call(H=252, ldx=256) == SHAPE and call(I=132) == SHAPE and call(H=0) == SHAPE and call(I=0) == SHAPE
    assert call(H=264, I=128, ldx=264, ld_out=264, w1_scales=F, w2_scales=F) == SHAPE        # E4M3: multiples of 16
    assert call(H=65536, ldx=65536, ld_out=65536, I=32768) == SHAPE                  # 4 GiB of an expert's weights
    assert call(ldx=248) == SHAPE and call(ldx=260) == SHAPE and call(ld_out=255) == SHAPE
    assert call(residual=F, ld_res=255) == SHAPE
    for n in ("logits", "x", "w1", "w2", "out"):
        assert call(**{n: None}) == NULL, n
    assert call(shared_w1=F) == NULL and call(w1_scales=F) == NULL and call(w2_scales=F) == NULL
    assert call(shared_w1=F, shared_w2=F, w1_scales=F, w2_scales=F) == NULL
    assert call(shared_w1_scales=F) == NULL
    assert call(x=F + 8) == SHAPE and call(w1=F + 8) == SHAPE and call(w2=F + 8) == SHAPE and call(logits=F + 4) == SHAPE
    assert call(out=F + 1) == SHAPE and call(residual=F + 1, ld_res=256) == SHAPE
    assert call(ws_bytes=16) == WS and call(ws=None) == WS and call(ws=F + 8) == SHAPE
    assert call(T=0, logits=None, x=None, out=None, ws=None, ws_bytes=0) == OK
    size = lib.moe_layer_few_workspace_size
    assert size(33, 2, 8, 256, 128, 0) == 0 and size(4, 2, 8, 256, 128, 2) == 0 and size(4, 0, 8, 256, 128, 0) == 0
    assert size(32, 31, 2048, 65536, 65536, 1) < 1 << 28 and size(1, 1, 1, 8, 8, 0) > 0


def test_bias_grad():
    lib = _lib.load()

    def call(dy=F, rows=64, ld=256, src=None, w=None, dtype=BF16, off=F, R=64, N=256, G=4, flags=0, db=F, ws=F,
             ws_bytes=1 << 40):
        return lib.moe_grouped_bias_grad(dy, rows, ld, src, w, dtype, off, R, N, G, flags, db, ws, ws_bytes, None)

    assert call(dtype=F32) == UNSUP and call(flags=_lib.MOE_WGRAD_F32) == UNSUP
    assert call(N=4) == SHAPE and call(N=252) == SHAPE and call(G=0) == SHAPE and call(G=2050) == SHAPE and call(R=-1) == SHAPE
    assert call(rows=63) == SHAPE and call(rows=0, src=F) == SHAPE and call(ld=248) == SHAPE and call(ld=260) == SHAPE
    assert call(rows=1 << 24, src=F) == SHAPE
    assert call(dy=None) == NULL and call(off=None) == NULL and call(db=None) == NULL
    assert call(dy=F + 8) == SHAPE and call(db=F + 8) == SHAPE
    assert call(R=5000, rows=5000, ws_bytes=0) == WS and call(R=5000, rows=5000, ws=F + 8) == SHAPE
    size = lib.moe_grouped_bias_grad_workspace_size
    assert size(16, 4, 256) == 0 and size(5000, 1, 256) > 0 and size(-1, 1, 256) == 0 and size(64, 1, 4) == 0


def test_route_backward():
    lib = _lib.load()

    def call(l=F, T=4, E=8, k=2, flags=0, idx=F, dw=F, rows=8, slot=None, ld=0, pg=None, z=0.0, out=F):
        return lib.moe_route_backward(l, T, E, k, flags, idx, dw, rows, slot, ld, pg, z, out, None)

    assert call(flags=_lib.MOE_MM_W_KN) == UNSUP
    assert call(T=-1) == SHAPE and call(E=0) == SHAPE and call(E=2049) == SHAPE and call(k=0) == SHAPE and call(k=9) == SHAPE
    assert call(k=33, E=64, rows=400) == SHAPE and call(rows=7) == SHAPE and call(rows=-1) == SHAPE
    assert call(slot=F, ld=1) == SHAPE and call(z=float("inf")) == SHAPE and call(z=float("nan")) == SHAPE
    for n in ("l", "idx", "dw", "out"):
        assert call(**{n: None}) == NULL, n
    assert call(l=F + 2) == SHAPE and call(out=F + 2) == SHAPE
    assert call(T=0, l=None, idx=None, dw=None, rows=0, out=None) == OK


def test_bindings_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    import routed_grouped_gemm_amd as moe

    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    w = torch.zeros((1, 16, 16), dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    for f in (lambda: moe.moe_layer_few(x.float(), x, w, w, 1), lambda: moe.moe_grouped_bias_grad(x, off),
              lambda: moe.moe_route_backward(x.float(), off[None], x.float())):
        with pytest.raises(moe.MoeError):
            f()


def test_grouped_mm_act():
    lib = _lib.load()

    def call(x=F, x_rows=64, ldx=128, src=None, w=F, dtype=BF16, off=F, R=64, N=256, K=128, G=4, flags=0, epi=None, rw=None,
             res=None, ld_res=0, y=F, ldy=256, ws=F, ws_bytes=1 << 40):
        return lib.moe_grouped_mm_act(x, x_rows, ldx, src, w, dtype, off, R, N, K, G, flags,
                                      None if epi is None else C.byref(epi), rw, res, ld_res, y, ldy, ws, ws_bytes, None)

    gated = _lib.MOE_MM_GATED
    assert call(dtype=F32) == UNSUP and call(flags=_lib.MOE_WGRAD_F32) == UNSUP
    assert call(flags=gated | _lib.MOE_MM_W_KN) == UNSUP
    assert call(epi=_lib.moe_epilogue(4, 1.0, 0.0, 0, None, None)) == UNSUP
    assert call(epi=_lib.moe_epilogue(-1, 1.0, 0.0, 0, None, None)) == UNSUP
    assert call(epi=_lib.moe_epilogue(0, float("nan"), 0.0, 0, None, None)) == SHAPE
    assert call(epi=_lib.moe_epilogue(0, 1.0, -0.5, 0, None, None)) == SHAPE
    assert call(epi=_lib.moe_epilogue(0, 1.0, 0.0, 0, F + 8, None)) == SHAPE and call(epi=_lib.moe_epilogue(0, 1.0, 0.0, 0, None, F + 8)) == SHAPE
    assert call(N=252) == SHAPE and call(N=264, ldy=264, flags=gated) == SHAPE and call(K=132, ldx=136) == SHAPE
    assert call(N=1 << 16, K=1 << 15, ldx=1 << 15, ldy=1 << 15, flags=gated) == SHAPE       # 4 GiB of a group's weights
    assert call(G=0) == SHAPE and call(G=2050) == SHAPE and call(R=-1) == SHAPE and call(x_rows=63) == SHAPE
    assert call(ldy=248) == SHAPE and call(ldy=258) == SHAPE and call(ldy=120, flags=gated) == SHAPE
    assert call(res=F, ld_res=252) == SHAPE and call(res=F, ld_res=258) == SHAPE and call(res=F + 4, ld_res=256) == SHAPE
    assert call(x=None) == NULL and call(w=None) == NULL and call(off=None) == NULL and call(y=None) == NULL
    assert call(x=F + 8) == SHAPE and call(w=F + 8) == SHAPE and call(y=F + 4) == SHAPE
    assert call(R=16, G=1, K=4096, ldx=4096, ws_bytes=0) == WS and call(R=16, G=1, K=4096, ldx=4096, ws=F + 8) == SHAPE
    assert call(R=0, x=None, x_rows=0, w=None, off=None, y=None) == OK


def test_grouped_mm_dact():
    lib = _lib.load()

    def call(dy=F, rows=64, ld=128, src=None, w=F, dtype=BF16, off=F, R=64, N=256, K=128, G=4, flags=_lib.MOE_MM_GATED,
             epi=None, pre=F, ld_pre=512, rw=None, dpre=F, h=F, dw=F, ws=F, ws_bytes=1 << 40):
        return lib.moe_grouped_mm_dact(dy, rows, ld, src, w, dtype, off, R, N, K, G, flags,
                                       None if epi is None else C.byref(epi), pre, ld_pre, rw, dpre, h, dw, ws, ws_bytes, None)

    assert call(dtype=F32) == UNSUP and call(flags=_lib.MOE_WGRAD_F32) == UNSUP
    assert call(epi=_lib.moe_epilogue(7, 1.0, 0.0, 0, None, None)) == UNSUP
    assert call(epi=_lib.moe_epilogue(0, 1.0, float("nan"), 0, None, None)) == SHAPE
    assert call(N=252, ld_pre=504) == SHAPE and call(K=132, ld=136) == SHAPE and call(G=0) == SHAPE and call(R=-1) == SHAPE
    assert call(ld_pre=508) == SHAPE and call(ld_pre=514) == SHAPE and call(pre=F + 4) == SHAPE
    assert call(rows=63) == SHAPE and call(ld=120) == SHAPE and call(rows=1 << 24, src=F) == SHAPE
    for n in ("dy", "w", "off", "pre", "dpre"):
        assert call(**{n: None}) == NULL, n
    assert call(dy=F + 8) == SHAPE and call(w=F + 8) == SHAPE and call(dpre=F + 8) == SHAPE and call(h=F + 8) == SHAPE
    assert call(ws_bytes=0) == WS and call(ws=F + 8) == SHAPE
    assert call(R=0, dy=None, rows=0, w=None, off=None, pre=None, dpre=None, h=None, dw=None, ws=None, ws_bytes=0) == OK
    for f in (lib.moe_grouped_mm_act_workspace_size, lib.moe_grouped_mm_dact_workspace_size):
        assert f(-1, 4, 256, 128) == 0 and f(64, 0, 256, 128) == 0 and f(64, 4, 250, 128) == 0
