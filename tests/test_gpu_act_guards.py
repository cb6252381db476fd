"""Offsets that do not ascend: nothing is written outside the outputs and the workspace
of the gradients, whose every byte outside is checked."""
import ctypes as C

import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")
lib = moe.lib
GUARD = 4096
FILL = 0x5A


class Guarded:
    """`n` bytes with GUARD filled bytes before and behind."""

    def __init__(self, n):
        self.n = n
        self.all = torch.full((GUARD + n + GUARD,), FILL, dtype=torch.uint8, device="cuda")

    def ptr(self):
        return self.all.data_ptr() + GUARD

    def intact(self):
        return bool((self.all[:GUARD] == FILL).all()) and bool((self.all[GUARD + self.n:] == FILL).all())


# none of these ascend; the last group ends past the rows, another starts before them
def offsets(R):
    return torch.tensor([0, R, 0, R + 4999, -7, R, 2, R], dtype=torch.int32, device="cuda")


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("R,N", [(100, 264), (3000, 264), (30000, 1032), (9000, 8)])
@pytest.mark.parametrize("accumulate", [0, moe.MOE_WGRAD_ACCUMULATE])
def test_bias_gradient(R, N, accumulate):
    banner(f"guards, bias gradient {R} {N} {accumulate}")
    dy = torch.ones((R, N), dtype=torch.bfloat16, device="cuda")
    off = offsets(R)
    nws = int(lib.moe_grouped_bias_grad_workspace_size(R, 7, N))
    db, ws = Guarded(7 * N * 4), Guarded(nws)
    st = lib.moe_grouped_bias_grad(dy.data_ptr(), R, N, None, None, moe.MOE_T_BF16, off.data_ptr(), R, N, 7, accumulate, db.ptr(),
                                   ws.ptr(), nws, stream())
    torch.cuda.synchronize()
    assert st == 0 and db.intact() and ws.intact()


@pytest.mark.parametrize("R,N,K", [(64, 264, 72), (300, 264, 2040), (5000, 264, 72), (20000, 520, 136)])
@pytest.mark.parametrize("gated", [0, moe.MOE_MM_GATED])
@pytest.mark.parametrize("single", [False, True])
def test_products_and_their_gradient(R, N, K, gated, single):
    banner(f"guards, products with an epilogue {R} {N} {K} {gated} {single}")
    G = 1 if single else 7
    off = torch.tensor([-3, R + 77], dtype=torch.int32, device="cuda") if single else offsets(R)
    x = torch.ones((R, K), dtype=torch.bfloat16, device="cuda")
    wide = 2 * N if gated else N
    w = torch.ones((G, wide, K), dtype=torch.bfloat16, device="cuda")
    epi = moe._lib.moe_epilogue(moe.MOE_ACT_SWIGLU, 1.0, 0.0, 0, None, None)
    y, pre = Guarded(R * N * 2), Guarded(R * wide * 2)
    epi.save_pre = pre.ptr()
    nws = int(lib.moe_grouped_mm_act_workspace_size(R, G, wide, K))
    ws = Guarded(nws)
    st = lib.moe_grouped_mm_act(x.data_ptr(), R, K, None, w.data_ptr(), moe.MOE_T_BF16, off.data_ptr(), R, wide, K, G, gated,
                                C.byref(epi), None, None, 0, y.ptr(), N, ws.ptr(), nws, stream())
    torch.cuda.synchronize()
    assert st == 0 and y.intact() and pre.intact() and ws.intact()
    epi.save_pre = None
    kept = torch.ones((R, wide), dtype=torch.bfloat16, device="cuda")
    dpre, h, dw = Guarded(R * wide * 2), Guarded(R * N * 2), Guarded(R * 4)
    nws = int(lib.moe_grouped_mm_dact_workspace_size(R, G, N, K))
    ws = Guarded(nws)
    st = lib.moe_grouped_mm_dact(x.data_ptr(), R, K, None, w.data_ptr(), moe.MOE_T_BF16, off.data_ptr(), R, N, K, G, gated,
                                 C.byref(epi), kept.data_ptr(), wide, None, dpre.ptr(), h.ptr(), dw.ptr(), ws.ptr(), nws, stream())
    torch.cuda.synchronize()
    assert st == 0 and dpre.intact() and h.intact() and dw.intact() and ws.intact()


@pytest.mark.parametrize("T,E,k,E_loc,H,I,shared", [(1, 8, 2, 8, 64, 32, 0), (16, 64, 8, 64, 264, 136, 1), (32, 40, 8, 40, 72, 1032, 0),
                                                    (32, 4, 4, 4, 64, 2568, 1), (32, 2048, 31, 2048, 16, 8, 1)])
def test_few_token_layer(T, E, k, E_loc, H, I, shared):
    """The same check of the layer for a few tokens, and its workspace."""
    banner(f"guards, few layer {T} {E} {k} {H} {I} {shared}")
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.1).to(torch.bfloat16)  # noqa: E731
    logits = torch.randn((T, E), generator=g, device="cuda")
    x, w1, w2, s1, s2 = n(T, H), n(E_loc, 2 * I, H), n(E_loc, H, I), n(1, 2 * I, H), n(1, H, I)
    want = moe.moe_layer_few(logits, x, w1, w2, k, shared=(s1, None, s2, None) if shared else None)
    nws = int(lib.moe_layer_few_workspace_size(T, k, E_loc, H, I, shared))
    out, ws = Guarded(T * H * 2), Guarded(nws)
    a = moe.moe_few_args(logits=logits.data_ptr(), T=T, E_tot=E, k=k, e0=0, E_loc=E_loc, dtype=moe.MOE_T_BF16, x=x.data_ptr(),
                         ldx=H, H=H, I=I, flags=0, w1=w1.data_ptr(), w2=w2.data_ptr(), out=out.ptr(), ld_out=H)
    if shared:
        a.shared_w1, a.shared_w2 = s1.data_ptr(), s2.data_ptr()
    st = lib.moe_layer_few(C.byref(a), ws.ptr(), nws, stream())
    torch.cuda.synchronize()
    assert st == 0 and out.intact() and ws.intact()
    got = out.all[GUARD:GUARD + out.n].view(torch.bfloat16).view(T, H)
    assert torch.equal(got, want)
