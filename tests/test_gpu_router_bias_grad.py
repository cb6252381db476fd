"""The router's gradient and the bias gradients against 64-bit sums and automatic differentiation."""
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def loss64(l, idx, D, renorm, c, z):
    """The scalar whose gradient in l the call returns."""
    p = torch.softmax(l, 1)
    w = p.gather(1, idx)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    loss = (w * D).sum()
    if c is not None:
        loss = loss + (p * c).sum()
    return loss + z * torch.logsumexp(l, 1).square().sum()


def check_route(l, idx, D, got, renorm, c, z):
    """fp32 throughout: exp of an argument below 40 in size is off by 2^-18 of
    itself (its argument's rounding, 40 * 2^-24 / 2, and the function's), a sum of
    E terms by fewer roundings than 64, so 2^-16 of the terms' sizes covers them."""
    l64 = l.double().requires_grad_(True)
    ref, = torch.autograd.grad(loss64(l64, idx.long(), D, renorm, c, z), l64)
    p = torch.softmax(l.double(), 1)
    w = p.gather(1, idx.long())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    own = torch.zeros_like(p).scatter_add_(1, idx.long(), w * (D.abs() + (D.abs() * w).sum(1, keepdim=True)))
    mag = own + p * (D.abs() * w).sum(1, keepdim=True)
    if c is not None:
        mag = mag + p * (c.abs() + (p * c.abs()).sum(1, keepdim=True))
    mag = mag + 2 * abs(z) * p * (torch.logsumexp(l.double(), 1, keepdim=True).abs() + 8)
    bad = (got.double() - ref).abs() / (2 ** -16 * mag + 1e-30)
    print(f"  largest error / bound {float(bad.max()):.4f}", flush=True)
    assert bool((bad <= 1).all())


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 4, 2), (3, 64, 16), (5, 64, 17), (100, 66, 8), (33, 128, 32), (17, 250, 8),
                                   (9, 257, 5), (6, 512, 8), (7, 1000, 20), (4, 2048, 32), (2000, 8, 2)])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("aux", [False, True])
def test_route_backward(T, E, k, renorm, aux):
    banner(f"route backward T={T} E={E} k={k} renorm={renorm} aux={aux}")
    g = gen(T + E + k)
    l = torch.randn((T, E), generator=g, device="cuda") * 3
    flags = moe.MOE_ROUTE_RENORM if renorm else 0
    idx, _ = moe.moe_route(l, k, flags)
    D = torch.randn((T, k), generator=g, device="cuda")
    c = torch.randn(E, generator=g, device="cuda") if aux else None
    z = 0.25 if aux else 0.0
    got = moe.moe_route_backward(l, idx, D, prob_grad=c, z_coef=z, flags=flags)
    check_route(l, idx, D.double(), got, renorm, c.double() if aux else None, z)


def test_route_backward_from_grouped_rows():
    """dw in grouped rows, through the slots that moe_permute writes (the shared
    expert's last column is not read); other GPUs' experts have none."""
    g = gen(1)
    T, E, k, e0, n = 77, 32, 4, 8, 12
    l = torch.randn((T, E), generator=g, device="cuda")
    for shared in (False, True):
        idx, w = moe.moe_route(l, k)
        p = moe.moe_permute(idx, w, e0, n, shared)
        dw = torch.randn(p["row_src"].shape[0], generator=g, device="cuda")
        slot = p["slot_row"][:, :k].long()
        D = torch.where(slot >= 0, dw[slot.clamp_min(0)], 0.0).double()
        got = moe.moe_route_backward(l, idx, dw, slot_row=p["slot_row"])
        check_route(l, idx, D, got, False, None, 0.0)
        # slots past dw count as not here
        got = moe.moe_route_backward(l, idx, dw[:5], slot_row=p["slot_row"])
        check_route(l, idx, torch.where(slot < 5, D, 0.0), got, False, None, 0.0)
        # none of them: zeros
        assert not bool(moe.moe_route_backward(l, idx, dw[:0], slot_row=p["slot_row"]).any())


def test_route_backward_differences():
    """Against differences of moe_route's own weights: the second-order term of
    a step of 2^-6 is below 2^-6 of the slope's bound (|D|), fp32 adds 2^-23 / 2^-6."""
    g = gen(2)
    T, E, k, step = 8, 16, 3, 2.0 ** -6
    l = torch.randn((T, E), generator=g, device="cuda")
    l += torch.sort(torch.rand((T, E), generator=g, device="cuda"), 1)[0] * 8       # no choice changes by a step
    D = torch.randn((T, k), generator=g, device="cuda")
    for flags in (0, moe.MOE_ROUTE_RENORM):
        idx, _ = moe.moe_route(l, k, flags)
        got = moe.moe_route_backward(l, idx, D, flags=flags)
        for e in range(E):
            up, dn = l.clone(), l.clone()
            up[:, e] += step
            dn[:, e] -= step
            (iu, wu), (i_d, wd) = moe.moe_route(up, k, flags), moe.moe_route(dn, k, flags)
            same = (iu == idx).all(1) & (i_d == idx).all(1)
            diff = ((wu - wd) * D).sum(1) / (2 * step)
            tol = 2.0 ** -6 * D.abs().sum(1)
            assert bool(((diff - got[:, e]).abs() <= tol)[same].all())


def test_route_backward_masked_and_odd_values():
    g = gen(3)
    inf = float("inf")
    l = torch.randn((6, 10), generator=g, device="cuda")
    l[0, 3:] = -inf
    l[1] = -inf
    l[2, 4] = float("nan")
    l[3, 4] = inf
    idx = torch.tensor([[0, 1], [0, 1], [4, 0], [4, 0], [2, 2], [-1, 10]], dtype=torch.int32, device="cuda")
    D = torch.randn((6, 2), generator=g, device="cuda")
    c = torch.randn(10, generator=g, device="cuda")
    for flags in (0, moe.MOE_ROUTE_RENORM):
        got = moe.moe_route_backward(l, idx, D, prob_grad=c, z_coef=0.5, flags=flags)
        assert bool((got[0, 3:] == 0).all()) and bool(torch.isfinite(got[0]).all())
        check_route(l[:1, :3].contiguous(), idx[:1], D[:1].double(), got[:1, :3], bool(flags), c[:3].double(), 0.5)
        assert bool((got[1] == 0).all())
        assert bool(got[2].isnan().all()) and bool(got[3].isnan().all())
        # the same expert twice, and experts that do not exist
        check_route(l[4:5], idx[4:5], D[4:5].double(), got[4:5], bool(flags), c.double(), 0.5)
        none = moe.moe_route_backward(l[5:], idx[5:], D[5:], flags=flags)
        assert bool((none == 0).all())


def test_route_backward_unaligned_rows():
    """Logits and gradients whose rows are no multiples of 16 bytes from a 16-byte start."""
    g = gen(4)
    base = torch.randn(1 + 12 * 64, generator=g, device="cuda")
    l = base[1:].view(12, 64)
    idx, _ = moe.moe_route(l.clone(), 3)
    D = torch.randn((12, 3), generator=g, device="cuda")
    out = torch.full((1 + 12 * 64 + 1,), 9.0, device="cuda")
    got = moe.moe_route_backward(l, idx, D, out=out[1:-1].view(12, 64))
    assert torch.equal(got, moe.moe_route_backward(l.clone(), idx, D))
    assert float(out[0]) == 9.0 and float(out[-1]) == 9.0


# ----------------------------------------------------------------- bias gradients
def bias_ref(dy, off, src, w, N):
    o = off.tolist()
    rows = src.long() if src is not None else torch.arange(dy.shape[0], device="cuda")
    ok = (rows >= 0) & (rows < dy.shape[0])
    d = torch.where(ok[:, None], dy.double()[rows.clamp(0, max(dy.shape[0] - 1, 0))], 0.0)
    if w is not None:
        d = d * w.double()[:, None]
    sums = [(d[a:b].sum(0), d[a:b].abs().sum(0)) for a, b in zip(o, o[1:])]
    return torch.stack([s for s, _ in sums]), torch.stack([m for _, m in sums])


def check_bias(got, ref, mag, R):
    """A chain of fp32 additions: at most pass / 4 + 3 in a pass and a quarter of
    the passes and 3 over them, with passes of 32 rows or more (up to 150 rows here
    in one), and a rounding for the weight: below R / 32 + 40."""
    tol = (R / 32 + 40) * 2.0 ** -24 * mag + 1e-30
    bad = (got.double() - ref).abs() / tol
    print(f"  largest error / bound {float(bad.max()):.3f}", flush=True)
    assert bool((bad <= 1).all())


@pytest.mark.parametrize("R,N,G", [(0, 8, 3), (1, 8, 1), (5, 520, 2), (33, 512, 1), (150, 264, 2), (257, 1032, 70),
                                   (3000, 264, 5), (20000, 2816, 4), (4096, 4104, 1), (700, 40, 2049)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gather", [False, True])
def test_bias_grad(R, N, G, dtype, gather):
    banner(f"bias gradient R={R} N={N} G={G} {dtype} gather={gather}")
    g = gen(R + N + G)
    cuts = torch.sort(torch.randint(0, R + 1, (G - 1,), generator=g, device="cuda"))[0]
    off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), R)]).to(torch.int32)
    T = max(R // 2, 1) if gather else R
    dy = torch.randn((T, N), generator=g, device="cuda").to(dtype)
    src = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    w = torch.randn(R, generator=g, device="cuda") if gather else None
    got = moe.moe_grouped_bias_grad(dy, off, dy_src=src, row_w=w)
    ref, mag = bias_ref(dy, off, src, w, N)
    check_bias(got, ref, mag, R)
    assert torch.equal(moe.moe_grouped_bias_grad(dy, off, dy_src=src, row_w=w), got)
    more = moe.moe_grouped_bias_grad(dy, off, dy_src=src, row_w=w, out=got.clone(), accumulate=True)
    check_bias(more, 2 * ref, 2 * mag, R + 64)


def test_bias_grad_rows_of_no_group_strides_and_sources_outside():
    g = gen(7)
    wide = torch.randn((900, 300), generator=g, device="cuda").to(torch.bfloat16)
    dy = wide[:, :264]                                      # not a multiple of 16 bytes a row
    with pytest.raises(moe.MoeError):
        moe.moe_grouped_bias_grad(dy, torch.tensor([0, 900], dtype=torch.int32, device="cuda"))
    wide = torch.randn((900, 320), generator=g, device="cuda").to(torch.bfloat16)
    dy = wide[:, 16:280]
    off = torch.tensor([100, 100, 700, 850], dtype=torch.int32, device="cuda")
    wide[:100], wide[850:] = float("nan"), float("nan")     # rows of no group
    got = moe.moe_grouped_bias_grad(dy, off)
    ref, mag = bias_ref(dy, off, None, None, 264)
    check_bias(got, ref, mag, 900)
    src = torch.randint(-5, 1000, (850,), generator=g, device="cuda", dtype=torch.int32)
    wide[:100], wide[850:] = 1.0, 2.0
    got = moe.moe_grouped_bias_grad(dy, off, dy_src=src)
    ref, mag = bias_ref(dy, off, src, None, 264)
    check_bias(got, ref, mag, 900)


def test_bias_grad_keeps_infinities_and_nan():
    dy = torch.ones((200, 8), dtype=torch.float16, device="cuda")
    dy[150, 0], dy[10, 1] = float("inf"), float("nan")
    off = torch.tensor([0, 120, 200], dtype=torch.int32, device="cuda")
    got = moe.moe_grouped_bias_grad(dy, off)
    assert float(got[1, 0]) == float("inf") and bool(got[0, 1].isnan())
    assert bool((got[0, [0, 2, 3, 4, 5, 6, 7]] == 120).all()) and bool((got[1, 1:] == 80).all())


def test_bias_grad_offsets_that_do_not_ascend_stay_inside():
    """Nothing outside the arrays is touched; which sums come out is not defined."""
    dy = torch.ones((5000, 520), dtype=torch.bfloat16, device="cuda")
    out = torch.full((7, 520), 3.0, device="cuda")
    off = torch.tensor([0, 5000, 0, 9999, -7, 5000, 2, 5000], dtype=torch.int32, device="cuda")
    moe.moe_grouped_bias_grad(dy, off, out=out)
    torch.cuda.synchronize()


def test_captured_gradients():
    g = gen(12)
    l = torch.randn((50, 64), generator=g, device="cuda")
    idx, _ = moe.moe_route(l, 4)
    D = torch.randn((50, 4), generator=g, device="cuda")
    dy = torch.randn((3000, 264), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, 10, 3000], dtype=torch.int32, device="cuda")
    call = lambda: (moe.moe_route_backward(l, idx, D), moe.moe_grouped_bias_grad(dy, off))   # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for _ in range(3):
        l.copy_(torch.randn(l.shape, generator=g, device="cuda"))
        dy.copy_(torch.randn(dy.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, call()):
            assert torch.equal(a, b)
