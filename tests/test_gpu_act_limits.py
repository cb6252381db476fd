"""The products with an epilogue and the gradients beside them at the ends of their
ranges: arrays past 4 GiB, the most groups, offsets that do not ascend."""
import pytest
import torch

from gpu_util import banner
from test_gpu_mm_act import forward, gradient

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")


@pytest.mark.parametrize("R", [60, 3000])
def test_most_groups(R):
    """2049 groups, most of them empty or of one row."""
    banner(f"2049 groups, {R} rows")
    forward(R, 2049, 24, 40, torch.bfloat16, True, moe.MOE_ACT_SWIGLU, weighted=True, T=50, seed=R)
    forward(R, 2049, 24, 40, torch.float16, False, moe.MOE_ACT_GEGLU, kn=True, seed=R + 1)
    gradient(R, 2049, 24, 40, torch.float16, True, moe.MOE_ACT_SWIGLU, weighted=True, seed=R + 2)


def tail_check(got, want, what):
    """`got` of a call whose last rows are `want`'s call: the same rows of the same
    products; both are within their bounds of the true values elsewhere, here they
    may differ by the order of the sums: two roundings of fp32 sums and one of bf16."""
    d = (got.double() - want.double()).abs()
    assert bool((d <= 2 ** -7 * want.double().abs() + 2 ** -10).all()), what


def test_rows_past_4_gib():
    """290000 rows of 8192 outputs: y and residual of 4.4 GiB, pre and dpre of 8.9; the
    last rows against a call of their own."""
    R, N, K, n = 290000, 8192, 64, 700
    banner(f"{R} rows of {N}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn((1, 2 * N, K), generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    off_n = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    rw = torch.rand(R, generator=g, device="cuda")
    res = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
    res[-n:] = torch.randn((n, N), generator=g, device="cuda")
    y, pre = moe.moe_grouped_mm_act(x, w, off, gated=True, row_w=rw, residual=res, keep_pre=True, out=res.clone())
    y_n, pre_n = moe.moe_grouped_mm_act(x[-n:].contiguous(), w, off_n, gated=True, row_w=rw[-n:].contiguous(),
                                        residual=res[-n:], keep_pre=True)
    tail_check(y[-n:], y_n, "y")
    tail_check(pre[-n:], pre_n, "pre")
    del res, y
    w2 = (torch.randn((1, K, N), generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    pre[-n:] = pre_n
    o = moe.moe_grouped_mm_dact(x, w2, off, pre, row_w=rw)
    o_n = moe.moe_grouped_mm_dact(x[-n:].contiguous(), w2, off_n, pre_n, row_w=rw[-n:].contiguous())
    for k in ("dpre", "h"):
        tail_check(o[k][-n:], o_n[k], k)
    # sums of 8192 terms in another order: fewer than 600 roundings of 2^-24 of |terms| below 8 each
    assert bool(((o["dw"][-n:] - o_n["dw"]).abs() <= 8192 * 8 * 600 * 2.0 ** -24).all())
    del pre, o["h"]
    db = moe.moe_grouped_bias_grad(o["dpre"], torch.tensor([R - n, R], dtype=torch.int32, device="cuda"))
    assert torch.equal(db, moe.moe_grouped_bias_grad(o["dpre"][-n:].contiguous(), off_n)) or bool(
        ((db - o["dpre"][-n:].double().sum(0)).abs() <= 2.0 ** -16 * o["dpre"][-n:].double().abs().sum(0)).all())


def test_route_gradient_past_2_31_logits():
    T, E, n = 1050000, 2048, 40
    banner(f"router gradient {T} x {E}")
    g = torch.Generator(device="cuda").manual_seed(2)
    l = torch.zeros((T, E), device="cuda")
    l[-n:] = torch.randn((n, E), generator=g, device="cuda")
    idx = torch.zeros((T, 2), dtype=torch.int32, device="cuda")
    idx[:, 1] = 7
    D = torch.randn((T, 2), generator=g, device="cuda")
    got = moe.moe_route_backward(l, idx, D)
    want = moe.moe_route_backward(l[-n:].contiguous(), idx[-n:].contiguous(), D[-n:].contiguous())
    assert torch.equal(got[-n:], want)


@pytest.mark.parametrize("R", [64, 5000])
def test_offsets_that_do_not_ascend_stay_inside(R):
    """Nothing outside the arrays is touched; which rows come out of overlapping groups is not defined."""
    N, K = 264, 72
    x = torch.ones((R, K), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, R, 0, R + 4999, -7, R, 2, R], dtype=torch.int32, device="cuda")
    w = torch.ones((7, 2 * N, K), dtype=torch.bfloat16, device="cuda")
    for gated in (True, False):
        cols = N if gated else 2 * N
        y = torch.full((R + 2, cols + 8), 3.0, dtype=torch.bfloat16, device="cuda")
        pre = torch.full((R + 2, 2 * N), 3.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_mm_act(x, w, off, gated=gated, keep_pre=True, out=y[1:-1, 4:-4], pre=pre[1:-1])
        for t in (y[0], y[-1], y[:, :4], y[:, -4:], pre[0], pre[-1]):
            assert bool((t == 3).all())
    o = moe.moe_grouped_mm_dact(x, w, off, torch.ones((R, 4 * N), dtype=torch.bfloat16, device="cuda"), w_kn=False)
    torch.cuda.synchronize()
    assert o["dpre"].shape == (R, 4 * N)
