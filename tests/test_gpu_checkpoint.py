"""Block-128 FP8 quantisation and the gated activation that keeps its input in
8 bits, against plain 64-bit implementations.

The codes and scales are exact by definition (division by a power of two, one
rounding), so they are compared for equality. Activations: h and dpre are one
fp32 expression of a few factors, each within 4 fp32 steps (the exponential's
and the reciprocal's error among them), rounded once to the output type:
eps / 2 + 32 * 2^-24 of the value; dw sums I such terms: (I + 32) * 2^-24 of
the sum of |terms|. exp(-z) is taken of the rounded product z * log2(e), which
adds |z| * 2^-24 relative: |z| <= 40 here, so 64 * 2^-24 covers the factor of
1 - s in the derivative as well."""
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")

T16 = [torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ref_blocks(v):
    """Codes (as bytes) and scales of the rows of v (64-bit), from the definition."""
    codes, scales = [], []
    for b in range(0, v.shape[1], 128):
        p = v[:, b:b + 128]
        fin = torch.where(p.isfinite(), p.abs(), 0.0)
        top = fin.amax(1)
        _, e = torch.frexp(top)                    # top in [2^(e-1), 2^e)
        e = e.double() - 9                         # 2^(e-9) * 448 = 0.875 * 2^e
        e = torch.where(top > 448 * torch.exp2(e), e + 1, e).clamp_min(-126)
        s = torch.where(top > 0, torch.exp2(e), 1.0)
        x = p / s[:, None]
        a = x.abs()
        _, ea = torch.frexp(a.clamp_min(2.0 ** -6))
        quantum = torch.exp2(ea.double() - 1 - 3)
        val = torch.round(a / quantum) * quantum   # ties to even
        byte = val.float().to(torch.float8_e4m3fn).view(torch.uint8).int()
        byte = torch.where(p.isfinite(), byte, 0x7F) | (torch.signbit(p).int() << 7)
        codes.append(byte.to(torch.uint8))
        scales.append(s)
    return torch.cat(codes, 1), torch.stack(scales, 1).float()


def hard_rows(g, R, K, dtype):
    """Rows of very different sizes, with exact ties, zeros, subnormals, NaN and infinities."""
    x = torch.randn((R, K), generator=g, device="cuda", dtype=torch.float32)
    if R:
        lim = 2.0 ** 14 if dtype == torch.float16 else 2.0 ** 126
        small = 2.0 ** -20 if dtype == torch.float16 else 2.0 ** -126
        x[0] *= 3.0 / 4
        x[R // 2, : K // 2] = 0.0
        x[R // 3] *= lim / 8
        x[R // 4] *= small
        x[(2 * R) // 3] = torch.arange(K, device="cuda") % 449 - 224.5      # many ties
        x[R - 1, 0] = 448.0
        if K > 16:
            x[R - 1, 3] = float("nan")
            x[R - 1, 9] = -float("inf")
            x[R - 1, 10] = float("inf")
    return x.to(dtype)


@pytest.mark.parametrize("dtype", T16 + [torch.float32])
@pytest.mark.parametrize("R,K", [(1, 8), (3, 128), (7, 136), (5, 1000), (70, 512), (33, 2048), (0, 64)])
def test_quantize_block(R, K, dtype):
    banner(f"quantize_block {R} x {K} {dtype}")
    x = hard_rows(gen(R + K), R, K, dtype)
    q, s = moe.moe_quantize_block(x)
    rq, rs = ref_blocks(x.double()) if R else (q, s)
    assert torch.equal(s, rs)
    assert torch.equal(q, rq)


def test_quantize_block_strides_and_row_count():
    g = gen(3)
    xb = torch.randn((40, 320), generator=g, device="cuda").to(torch.bfloat16)
    x = xb[:, 64:264]
    n = torch.tensor([17], dtype=torch.int32, device="cuda")
    q = torch.full((40, 200), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((40, 2), 5.0, device="cuda")
    moe.moe_quantize_block(x, n_rows=n, codes=q, scales=s)
    rq, rs = ref_blocks(x.double())
    assert torch.equal(q[:17], rq[:17]) and torch.equal(s[:17], rs[:17])
    assert torch.all(q[17:] == 9) and torch.all(s[17:] == 5)


@pytest.mark.parametrize("dtype", T16 + [torch.float32])
@pytest.mark.parametrize("G,N,K", [(1, 1, 8), (2, 128, 128), (3, 130, 264), (2, 300, 1000)])
def test_quantize_block_weights(G, N, K, dtype):
    banner(f"quantize_block_weights {G} x {N} x {K} {dtype}")
    w = hard_rows(gen(N + K), G * N, K, dtype).view(G, N, K)
    q, s = moe.moe_quantize_block_weights(w)
    for e in range(G):
        for nb in range(s.shape[1]):
            for kb in range(s.shape[2]):
                p = w[e, nb * 128:(nb + 1) * 128, kb * 128:(kb + 1) * 128].double()
                # one block: its rows side by side have the same largest value
                top = torch.where(p.isfinite(), p.abs(), 0.0).max()
                probe = torch.zeros((p.shape[0], 128), dtype=torch.float64, device="cuda")
                probe[:, : p.shape[1]] = p
                if p.shape[1] < 128:
                    probe[:, p.shape[1]] = top
                    rq, rs = ref_blocks(probe)
                else:
                    _, rs = ref_blocks(top.reshape(1, 1))
                    rs = rs.expand(p.shape[0], 1)
                    x = (p / rs[0, 0].double())
                    rq, _ = ref_blocks(torch.cat([x, torch.full_like(x[:, :1], 448.0)], 1)[:, -128:])
                    # a column of 448 stands for the block's largest value; the
                    # first column is then compared by itself
                    r0, _ = ref_blocks(torch.cat([x[:, :1], torch.full_like(x[:, :1], 448.0)], 1))
                    rq = torch.cat([r0[:, :1], rq[:, :127]], 1)
                if float(top) > 0:
                    got = q[e, nb * 128:(nb + 1) * 128, kb * 128:(kb + 1) * 128]
                    assert torch.equal(got, rq[:, : p.shape[1]]), (e, nb, kb)
                    assert float(s[e, nb, kb]) == float(rs[0, 0])
                else:
                    assert float(s[e, nb, kb]) == 1.0


# ------------------------------------------------------------ gated activation
def act64(z, act, beta):
    if act == moe.MOE_ACT_GEGLU:
        cdf = 0.5 * (1 + torch.erf(z / 2 ** 0.5))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    if act == moe.MOE_ACT_SRELU:
        r = z.clamp_min(0)
        return r * r, 2 * r
    s = torch.sigmoid(beta * z)
    return z * s, s + beta * z * s * (1 - s)


EPIS = [None, (moe.MOE_ACT_SWIGLU, 1.7, 2.0), (moe.MOE_ACT_GEGLU, 1.0, 0.0), (moe.MOE_ACT_SRELU, 1.0, 3.0)]


def epi_of(e):
    return (None, moe.MOE_ACT_SWIGLU, 1.0, 0.0) if e is None else (moe.Epilogue(e[0], e[1], e[2]), *e)


def close(got, ref, what, mag=None, n=64):
    eps = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps
    mag = ref.abs() if mag is None else mag
    one = eps * ref.abs() if got.dtype != torch.float32 else 0.0
    tol = one + n * 2.0 ** -24 * mag + tiny
    d = (got.double() - ref).abs()
    worst = float((d / tol).max()) if d.numel() else 0.0
    print(f"  {what}: largest |diff| / tolerance {worst:.3f}", flush=True)
    assert (d <= tol).all(), (what, worst)


@pytest.mark.parametrize("epi", EPIS)
@pytest.mark.parametrize("dtype", T16)
@pytest.mark.parametrize("R,I", [(1, 8), (3, 128), (5, 136), (9, 1000), (66, 1408), (2, 4096), (0, 64)])
def test_glu_checkpoint(R, I, dtype, epi):
    banner(f"glu {R} x {I} {dtype} {epi}")
    g = gen(R * 7 + I)
    e, act, beta, limit = epi_of(epi)
    pre = (torch.randn((R, 2 * I), generator=g, device="cuda") * 1.5).to(dtype)
    w = torch.rand(R, generator=g, device="cuda")
    h, q, s = moe.moe_glu_checkpoint(pre, row_w=w, epi=e)
    p = pre.double()
    cl = (lambda v: v.clamp(-limit, limit)) if limit else (lambda v: v)
    a, _ = act64(cl(p[:, :I]), act, beta)
    # the exact GELU's factor 1 + erf cancels for negative gates: the bound is
    # on |gate| * 1 there, not on the (smaller) product
    amag = p[:, :I].abs() if act == moe.MOE_ACT_GEGLU else a.abs()
    close(h, a * cl(p[:, I:]) * w.double()[:, None], "h", (amag * cl(p[:, I:])).abs() * w.double()[:, None])
    if R:
        rq, rs = ref_blocks(p.view(2 * R, I))
        assert torch.equal(q, rq.view(R, 2 * I)) and torch.equal(s, rs.view(R, 2, -1))
    h2, none_q, none_s = moe.moe_glu_checkpoint(pre, row_w=w, epi=e, keep=False)
    assert none_q is None and none_s is None and torch.equal(h2, h)

    # the backward pass from the kept bytes
    dh = (torch.randn((R, I), generator=g, device="cuda") * 0.1).to(dtype)
    o = moe.moe_glu_checkpoint_backward(q, s, dh, row_w=w, epi=e)
    kept = q.view(torch.float8_e4m3fn).double().view(2 * R, I) * s.double().view(2 * R, (I + 127) // 128).repeat_interleave(128, 1)[:, :I]
    kept = kept.view(R, 2 * I)
    G, U, D, W = kept[:, :I], kept[:, I:], dh.double(), w.double()[:, None]
    mg = (G.abs() <= limit).double() if limit else 1.0
    mu = (U.abs() <= limit).double() if limit else 1.0
    a, da = act64(cl(G), act, beta)
    gm = cl(G).abs()
    amag = gm if act == moe.MOE_ACT_GEGLU else a.abs()
    damag = 2 + gm if act != moe.MOE_ACT_SRELU else da.abs()     # a sum of terms up to |z|: bounded by them
    close(o["dpre"][:, :I], D * W * cl(U) * da * mg, "dg", (D * W * cl(U)).abs() * damag)
    close(o["dpre"][:, I:], D * W * a * mu, "du", (D * W).abs() * amag)
    close(o["h"], a * cl(U) * W, "h again", (cl(U) * W).abs() * amag)
    close(o["dw"], (D * a * cl(U)).sum(1), "dw", (D * cl(U)).abs().mul(amag).sum(1), n=I + 64)
    o2 = moe.moe_glu_checkpoint_backward(q, s, dh, row_w=w, epi=e, want_h=False, want_dw=False)
    assert o2["h"] is None and o2["dw"] is None and torch.equal(o2["dpre"], o["dpre"])


def test_glu_gradient_against_differences():
    """dg, du and dw against central differences of the forward formula."""
    g = gen(11)
    R, I = 4, 136
    for act, beta, limit in ((moe.MOE_ACT_SWIGLU, 1.3, 0.0), (moe.MOE_ACT_GEGLU, 1.0, 0.0), (moe.MOE_ACT_SRELU, 1.0, 0.0)):
        e = moe.Epilogue(act, beta, limit)
        pre = (torch.randn((R, 2 * I), generator=g, device="cuda")).to(torch.float16)
        w = torch.rand(R, generator=g, device="cuda") + 0.1
        _, q, s = moe.moe_glu_checkpoint(pre, row_w=w, epi=e)
        dh = torch.randn((R, I), generator=g, device="cuda").to(torch.float16)
        o = moe.moe_glu_checkpoint_backward(q, s, dh, row_w=w, epi=e)
        kept = (q.view(torch.float8_e4m3fn).double().view(2 * R, I)
                * s.double().view(2 * R, (I + 127) // 128).repeat_interleave(128, 1)[:, :I]).view(R, 2 * I)

        def loss(p, ww):
            a, _ = act64(p[:, :I], act, beta)
            return (dh.double() * a * p[:, I:] * ww.double()[:, None])

        step = 1e-5
        up, dn = kept.clone(), kept.clone()
        up[:, :I] += step
        dn[:, :I] -= step
        dg = (loss(up, w) - loss(dn, w)) / (2 * step)
        # differences: off by step^2 times the third derivative (below 10 |dh u w|),
        # and at the squared ReLU's kink by step; the result by fp16's rounding
        scale = (dh.double() * kept[:, I:] * w.double()[:, None]).abs()
        assert ((o["dpre"][:, :I].double() - dg).abs() <= 2.0 ** -11 * dg.abs() + 4e-5 * scale + 1e-7).all()
        up, dn = kept.clone(), kept.clone()
        up[:, I:] += step
        dn[:, I:] -= step
        du = (loss(up, w) - loss(dn, w)) / (2 * step)
        scale = (dh.double() * w.double()[:, None]).abs() * (1 + kept[:, :I].abs())
        assert ((o["dpre"][:, I:].double() - du).abs() <= 2.0 ** -11 * du.abs() + 4e-5 * scale + 1e-7).all()
        dw = (loss(kept, w + step) - loss(kept, w - step)).sum(1) / (2 * step)
        mag = loss(kept, torch.ones_like(w)).abs().sum(1)
        # w + step is rounded to fp32: 2^-24 / step of relative error
        assert ((o["dw"].double() - dw).abs() <= 2e-2 * mag).all()


def test_glu_row_count_strides_and_specials():
    g = gen(12)
    R, I, n = 23, 200, 14
    cnt = torch.tensor([3, n], dtype=torch.int32, device="cuda")[1:]        # a view: the last offset
    preb = torch.randn((R, 2 * I + 16), generator=g, device="cuda").to(torch.bfloat16)
    pre = preb[:, 8:8 + 2 * I]
    pre[2, 5] = float("nan")
    pre[3, I + 7] = float("inf")
    h = torch.full((R, I), 3.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((R, 2 * I), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((R, 2, 2), 5.0, device="cuda")
    moe.moe_glu_checkpoint(pre, n_rows=cnt, h=h, codes=q, scales=s)
    rq, rs = ref_blocks(pre.double().reshape(2 * R, I))
    assert torch.equal(q[:n], rq.view(R, -1)[:n]) and torch.equal(s[:n], rs.view(R, 2, -1)[:n])
    assert (h[n:] == 3).all() and (q[n:] == 9).all() and (s[n:] == 5).all()
    assert torch.isnan(h[2, 5]) and torch.isinf(h[3, 7]) and h[:n].isfinite().sum() == n * I - 2
    lim = moe.Epilogue(moe.MOE_ACT_SWIGLU, 1.0, 1.0)
    h3, _, _ = moe.moe_glu_checkpoint(pre, epi=lim)
    assert torch.isnan(h3[2, 5]) and h3[3, 7].isfinite()                    # a clamp keeps a NaN
    dh = torch.ones((R, 2 * I), dtype=torch.bfloat16, device="cuda")[:, I:]
    o = moe.moe_glu_checkpoint_backward(q, s, dh, n_rows=cnt)
    assert torch.isnan(o["dpre"][2, 5]) and torch.isnan(o["dw"][2])
    assert o["dw"][[0, 1, 4, 5]].isfinite().all()
