"""Grouped products with an epilogue and the activation's gradient in one, against
the same formulas in 64 bits, on every kernel that the sizes choose."""
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")

SWI, GELU, RELU2, NONE = moe.MOE_ACT_SWIGLU, moe.MOE_ACT_GEGLU, moe.MOE_ACT_SRELU, moe.MOE_ACT_NONE
INF = float("inf")

# (rows, groups, output columns, K)
SHAPES = [(1, 1, 8, 8), (5, 3, 40, 72), (16, 1, 512, 4096), (40, 1, 256, 2048), (300, 2, 264, 520), (700, 3, 136, 264),
          (2000, 4, 520, 264), (1500, 40, 264, 136), (3000, 1, 1032, 136), (3000, 40, 1288, 72), (6000, 2, 1032, 136),
          (9000, 4, 1032, 200)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def test_shapes_reach_every_kernel():
    """Tiles of 32 and 64 rows (weight-streaming), 128 and 256 (LDS-tiled), and a split along K."""
    for wide in (1, 2):
        plans = [moe.moe_grouped_mm_plan(R, G, wide * N, K) for R, G, N, K in SHAPES]
        assert {p[0] for p in plans} == {32, 64, 128, 256} and max(p[1] for p in plans) > 1


def a64(z, act, beta=1.0):
    if act == GELU:
        return z * 0.5 * torch.erfc(z * -0.5 ** 0.5)          # (ndtr loses the tail: 2% at -8)
    if act == RELU2:
        return torch.relu(z).square()
    return z if act == NONE else z * torch.sigmoid(beta * z)


def slope64(z, act, beta=1.0):
    z = z.detach().clone().requires_grad_(True)
    return torch.autograd.grad(a64(z, act, beta).sum(), z)[0]


class Plan:
    """Uneven groups (an empty one among them where there are several), and
    optional sources, weights and residual."""

    def __init__(self, R, G, seed, T=0, weighted=False, lo=0, hi=None):
        g = gen(seed)
        hi = R if hi is None else hi
        cuts = torch.sort(torch.randint(lo, hi + 1, (G - 1,), generator=g, device="cuda"))[0]
        if G > 2:
            cuts[1] = cuts[0]
        self.R, self.G = R, G
        self.off = torch.cat([cuts.new_full((1,), lo), cuts, cuts.new_full((1,), hi)]).to(torch.int32)
        self.src = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32) if T else None
        self.w = torch.rand(R, generator=g, device="cuda") * 2 - 0.5 if weighted else None

    def groups(self):
        o = self.off.tolist()
        return [(e, a, b) for e, (a, b) in enumerate(zip(o, o[1:])) if b > a]

    def rows(self, t):
        s = self.src.long() if self.src is not None else torch.arange(self.R, device="cuda")
        ok = (s >= 0) & (s < t.shape[0])
        return torch.where(ok[:, None], t.double()[s.clamp(0, t.shape[0] - 1)], 0.0)


def products(pl, t, w, kn):
    """(product, sum of |terms|) of every row in 64 bits; rows of no group 0."""
    x = pl.rows(t)
    n = w.shape[2 if kn else 1]
    z = torch.zeros((pl.R, n), dtype=torch.float64, device="cuda")
    m = torch.zeros_like(z)
    for e, a, b in pl.groups():
        we = w[e].double() if kn else w[e].double().t()
        z[a:b], m[a:b] = x[a:b] @ we, x[a:b].abs() @ we.abs()
    return z, m


def used(pl):
    u = torch.zeros(pl.R, dtype=torch.bool, device="cuda")
    for _, a, b in pl.groups():
        u[a:b] = True
    return u


def sum_err(K):
    """Of an fp32 sum of K products of 16-bit values, relative to the sum of
    |terms|: one rounding for each 32 of the chain, up to 16 parts and the
    matrix instruction's own 32-term sum."""
    return (K / 32 + 48) * 2.0 ** -24


def check(got, ref, tol, rows, what):
    """got within tol of ref in the groups' rows, untouched elsewhere (the caller filled it with 7)."""
    assert bool((got[~rows] == 7).all()), what
    bad = (got.double() - ref).abs()[rows] / tol[rows]
    worst = float(bad.max()) if bad.numel() else 0.0
    print(f"  {what}: largest error / bound {worst:.3f}", flush=True)
    assert bool((bad <= 1).all()), what


def forward(R, G, N, K, dtype, gated, act, kn=False, T=0, weighted=False, bias=True, residual=True, limit=0.0, beta=1.0,
            seed=0, lo=0, hi=None):
    g = gen(seed)
    pl = Plan(R, G, seed + 1, T, weighted, lo, hi)
    wide = 2 * N if gated else N
    x = torch.randn((T or R, K), generator=g, device="cuda").to(dtype)
    w = (torch.randn((G, K, wide) if kn else (G, wide, K), generator=g, device="cuda") * K ** -0.5).to(dtype)
    b = torch.randn((G, wide), generator=g, device="cuda") * 0.5 if bias else None
    res = torch.randn((R, N), generator=g, device="cuda").to(dtype) if residual else None
    out = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
    pre = torch.full((R, wide), 7.0, dtype=dtype, device="cuda")
    epi = moe.Epilogue(act=act, beta=beta, limit=limit, bias=b)
    call = lambda **kw: moe.moe_grouped_mm_act(x, w, pl.off, epi=epi, gated=gated, w_kn=kn, row_src=pl.src, row_w=pl.w,  # noqa: E731
                                               residual=res, **kw)
    y, p = call(keep_pre=True, out=out, pre=pre)
    assert y is out and p is pre
    rows = used(pl)
    z, m = products(pl, x, w, kn)
    if bias:
        for e, a, c in pl.groups():
            z[a:c] += b[e].double()
            m[a:c] += b[e].double().abs()
    u = torch.finfo(dtype).eps / 2
    small = torch.finfo(dtype).tiny * u                     # half a step of the subnormal range
    dz = sum_err(K) * m
    check(p, z, dz + u * z.abs() * (1 + 2 ** -7) + small, rows, "pre")
    cut = limit if limit > 0 else INF
    gz, dg = z[:, :N].clamp(-cut, cut), dz[:, :N]
    a, da = a64(gz, act, beta), slope64(gz, act, beta).abs()
    # second order: |a''| is at most 2 (squared ReLU; below beta + 1 for the others)
    d = (da + (2 + beta) * dg) * dg + 2 ** -18 * a.abs() * (1 + gz.abs() / 8)
    h = a
    if gated:
        uz, du = z[:, N:].clamp(-cut, cut), dz[:, N:]
        d = d * (uz.abs() + du) + a.abs() * du
        h = a * uz
    if weighted:
        h, d = h * pl.w.double()[:, None], d * pl.w.double().abs()[:, None]
    ref = h + res.double() if residual else h
    tol = d + 2 ** -22 * (h.abs() + (res.double().abs() if residual else 0.0))
    check(y, ref, tol + u * (ref.abs() + tol) + small, rows, "y")
    # without the kept pre-activation, and again: the same bits
    assert torch.equal(call()[rows], y[rows])
    assert torch.equal(call(keep_pre=True)[0][rows], y[rows])


@pytest.mark.parametrize("R,G,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["gated", "nk", "kn"])
def test_forward_on_every_kernel(R, G, N, K, dtype, kind):
    banner(f"act {kind} R={R} G={G} N={N} K={K} {dtype}")
    i = SHAPES.index((R, G, N, K))
    act = [SWI, GELU, RELU2, NONE][(i + (kind == "kn")) % 4]
    forward(R, G, N, K, dtype, kind == "gated", act, kn=kind == "kn", T=(R // 2 + 1) * (i % 2), weighted=i % 3 != 1,
            bias=i % 4 != 2, residual=i % 2 == 0, seed=i)


# One group whose last tiles are mostly empty: a few rows past 32 tiles, a few
# columns past 8, both, and up to the 64 that still go apart; hi < R: fewer rows
# in the group than the call allows for, so that its tail is another one
TAILS = [(8195, 2048, 8195), (8192, 2056, 8192), (8195, 2056, 8195), (8256, 2112, 8256), (8195, 2056, 7900), (8195, 2056, 2),
         (8191, 2040, 8191)]


@pytest.mark.parametrize("R,N,hi", TAILS)
@pytest.mark.parametrize("kind", ["gated", "nk", "kn"])
def test_one_group_with_mostly_empty_last_tiles(R, N, hi, kind):
    banner(f"act tails {kind} R={R} N={N} hi={hi}")
    gated = kind == "gated"
    forward(R, 1, N // 2 // 8 * 8 if gated else N, 136, torch.bfloat16, gated, SWI, kn=kind == "kn", weighted=True, seed=R + N, hi=hi)


@pytest.mark.parametrize("R,N,hi", TAILS)
@pytest.mark.parametrize("gated", [False, True])
def test_gradient_of_one_group_with_mostly_empty_last_tiles(R, N, hi, gated):
    banner(f"dact tails gated={gated} R={R} N={N} hi={hi}")
    gradient(R, 1, N, 136, torch.bfloat16, gated, GELU, kn=gated, weighted=True, T=500, seed=R + N, hi=hi)


# The same where the launches of the tails are split along K: 3 rows past 16
# tiles, 8 columns, both; fewer rows in the group (160 past the whole tiles, 2)
SPLIT_TAILS = [(4099, 4096, 4099), (4095, 4104, 4095), (4099, 4104, 4099), (4099, 4104, 4000), (4099, 4104, 2)]


@pytest.mark.parametrize("R,N,hi", SPLIT_TAILS)
@pytest.mark.parametrize("kind", ["gated", "nk", "kn"])
def test_split_tails(R, N, hi, kind):
    banner(f"act split tails {kind} R={R} N={N} hi={hi}")
    gated = kind == "gated"
    assert moe.lib.moe_grouped_mm_act_workspace_size(R, 1, N, 2040) > 0         # (only what is split has one)
    cols = (N // 2 + 7) // 8 * 8 if gated else N
    forward(R, 1, cols, 2040, torch.float16, gated, GELU, kn=kind == "kn", weighted=True, residual=True, seed=R + N, hi=hi)


@pytest.mark.parametrize("R,N,hi", SPLIT_TAILS)
@pytest.mark.parametrize("gated", [False, True])
def test_gradient_split_tails(R, N, hi, gated):
    banner(f"dact split tails gated={gated} R={R} N={N} hi={hi}")
    gradient(R, 1, N, 2040, torch.bfloat16, gated, SWI, kn=gated, weighted=True, T=500, seed=R + N, hi=hi)


@pytest.mark.parametrize("act,beta,limit", [(SWI, 1.0, 0.0), (SWI, 1.702, 0.75), (GELU, 1.0, 0.0), (GELU, 1.0, 1.5),
                                            (RELU2, 1.0, 1.0), (NONE, 1.0, 0.5)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R", [30, 6000])
def test_activations(act, beta, limit, gated, R):
    banner(f"act {act} beta {beta} limit {limit} gated {gated} R={R}")
    forward(R, 2, 264, 136, torch.float16, gated, act, beta=beta, limit=limit, weighted=True, seed=act)


@pytest.mark.parametrize("R", [33, 500, 7000])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_of_no_group_are_left(R, gated):
    forward(R, 3, 136, 264, torch.bfloat16, gated, SWI, weighted=True, seed=R, lo=R // 5, hi=R - R // 4)


@pytest.mark.parametrize("R", [20, 5000])
def test_strides_in_place_and_sources_outside(R):
    g = gen(R)
    N, K, T = 264, 136, 50
    wide = torch.randn((T, K + 24), generator=g, device="cuda").to(torch.bfloat16)
    x = wide[:, 8:8 + K]
    w = torch.randn((2, N, K), generator=g, device="cuda").to(torch.bfloat16) * 0.1
    pl = Plan(R, 2, R, T)
    pl.src = torch.randint(-3, T + 3, (R,), generator=g, device="cuda", dtype=torch.int32)
    buf = torch.randn((R, N + 20), generator=g, device="cuda").to(torch.bfloat16)
    keep = buf.clone()
    y = buf[:, 4:4 + N]                                      # rows at multiples of 8 bytes only
    res = y.clone()
    want = moe.moe_grouped_mm_act(x, w, pl.off, row_src=pl.src, residual=res)
    got = moe.moe_grouped_mm_act(x, w, pl.off, row_src=pl.src, residual=y, out=y)
    assert got.data_ptr() == y.data_ptr() and torch.equal(got, want)
    assert torch.equal(buf[:, :4], keep[:, :4]) and torch.equal(buf[:, 4 + N:], keep[:, 4 + N:])
    z, m = products(pl, x, w, False)
    u = 2.0 ** -8
    ref = z + res.double()
    assert bool(((got.double() - ref).abs() <= sum_err(K) * m + u * ref.abs() * (1 + u) + 2.0 ** -22 * m + 1e-30).all())


def test_default_epilogue_is_the_plain_product():
    g = gen(3)
    for R in (17, 600, 4000):
        x = torch.randn((R, 264), generator=g, device="cuda").to(torch.bfloat16)
        w = torch.randn((2, 520, 264), generator=g, device="cuda").to(torch.bfloat16)
        off = torch.tensor([0, R // 3, R], dtype=torch.int32, device="cuda")
        assert torch.equal(moe.moe_grouped_mm_act(x, w, off), moe.moe_grouped_mm(x, w, off))
        with pytest.raises(moe.MoeError):                    # halves of 260 rows: no multiple of 8
            moe.moe_grouped_mm_act(x, w, off, gated=True, keep_pre=True)
        w = w[:, :512].contiguous()
        both = moe.moe_grouped_mm_act(x, w, off, gated=True, keep_pre=True)
        assert torch.equal(both[1], moe.moe_grouped_mm(x, w, off))


@pytest.mark.parametrize("R", [20, 3000])
def test_nan_stays_in_its_row_and_column(R):
    g = gen(R)
    x = torch.randn((R, 136), generator=g, device="cuda").to(torch.float16)
    w = (torch.randn((1, 2 * 136, 136), generator=g, device="cuda") * 0.1).to(torch.float16)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    for act in (SWI, GELU, RELU2, NONE):
        for limit in (0.0, 1.0):
            epi = moe.Epilogue(act=act, limit=limit)
            want = moe.moe_grouped_mm_act(x, w, off, epi=epi, gated=True)
            xn, wn = x.clone(), w.clone()
            xn[R - 1, 5] = float("nan")
            wn[0, 7, 3], wn[0, 136 + 9, 3] = float("nan"), float("nan")        # a gate column and an up column
            got = moe.moe_grouped_mm_act(xn, wn, off, epi=epi, gated=True)
            hit = torch.zeros_like(got, dtype=torch.bool)
            hit[R - 1], hit[:, 7], hit[:, 9] = True, True, True
            # (a product of NaN and 0 is NaN too)
            assert bool(got[hit].isnan().all())
            assert torch.equal(got[~hit], want[~hit])


# ------------------------------------------------------------------- gradient
def gradient(R, G, N, K, dtype, gated, act, kn=True, T=0, weighted=False, limit=0.0, beta=1.0, seed=0, lo=0, hi=None):
    g = gen(seed)
    pl = Plan(R, G, seed + 1, T, weighted, lo, hi)
    wide = 2 * N if gated else N
    dy = torch.randn((T or R, K), generator=g, device="cuda").to(dtype)
    w = (torch.randn((G, K, N) if kn else (G, N, K), generator=g, device="cuda") * K ** -0.5).to(dtype)
    buf = (torch.randn((R, wide + 8), generator=g, device="cuda") * 1.5).to(dtype)
    pre = buf[:, 4:4 + wide]
    if limit > 0:
        pre[::3, ::2] = limit                                # on the border: still inside
    epi = moe.Epilogue(act=act, beta=beta, limit=limit)
    call = lambda **kw: moe.moe_grouped_mm_dact(dy, w, pl.off, pre, epi=epi, gated=gated, w_kn=kn, dy_src=pl.src,   # noqa: E731
                                                row_w=pl.w, **kw)
    o = call()
    rows = used(pl)
    for t in o.values():
        t[~rows] = 7.0                                       # (allocated inside: nothing to check there)
    dh, m = products(pl, dy, w, kn)
    ddh = sum_err(K) * m
    z = pre.double()
    cut = limit if limit > 0 else INF
    gz = z[:, :N].clamp(-cut, cut)
    a, s = a64(gz, act, beta), slope64(gz, act, beta)
    ea = 2 ** -18 * a.abs() * (1 + gz.abs() / 8)             # the activation's own error (exp of an argument below 16)
    es = 2 ** -18 * (1 + gz.abs()) * (1 + beta)
    gin = (z[:, :N].abs() <= cut).double()
    uz = z[:, N:].clamp(-cut, cut) if gated else torch.ones_like(gz)
    wr = pl.w.double()[:, None] if weighted else torch.ones((R, 1), dtype=torch.float64, device="cuda")
    u = torch.finfo(dtype).eps / 2
    small = torch.finfo(dtype).tiny * u
    dg = dh * wr * uz * s * gin
    tg = (wr * uz).abs() * gin * (ddh * s.abs() + (dh.abs() + ddh) * es)
    ref, tol = dg, tg
    if gated:
        uin = (z[:, N:].abs() <= cut).double()
        ref = torch.cat([dg, dh * wr * a * uin], 1)
        tol = torch.cat([tg, wr.abs() * uin * (ddh * a.abs() + (dh.abs() + ddh) * ea)], 1)
    tol = tol + 2 ** -21 * ref.abs()
    check(o["dpre"], ref, tol + u * (ref.abs() + tol) + small, rows, "dpre")
    h = a * uz * wr
    th = (uz * wr).abs() * ea + 2 ** -21 * h.abs()
    check(o["h"], h, th + u * (h.abs() + th) + small, rows, "h")
    terms = (dh * a * uz).abs()
    # N terms, added 4 to 64 at a time and then one after another: fewer than N / 16 + 40 roundings in a row
    tw = (ddh * (a * uz).abs() + dh.abs() * ea * uz.abs()).sum(1) + (N / 16 + 40) * 2 ** -24 * terms.sum(1)
    check(o["dw"], (dh * a * uz).sum(1), tw + 1e-30, rows, "dw")
    p = call(want_h=False, want_dw=False)
    assert p["h"] is None and p["dw"] is None and torch.equal(p["dpre"][rows], o["dpre"][rows])
    p = call(want_h=False)
    assert torch.equal(p["dw"][rows], o["dw"][rows])


@pytest.mark.parametrize("R,G,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kn", [False, True])
def test_gradient_on_every_kernel(R, G, N, K, dtype, gated, kn):
    banner(f"dact gated={gated} kn={kn} R={R} G={G} N={N} K={K} {dtype}")
    i = SHAPES.index((R, G, N, K))
    gradient(R, G, N, K, dtype, gated, [SWI, GELU, RELU2, NONE][(i + gated) % 4], kn=kn, T=(R // 2 + 1) * (i % 2),
             weighted=i % 3 != 1, seed=i)


@pytest.mark.parametrize("act,beta,limit", [(SWI, 1.0, 0.0), (SWI, 1.702, 0.75), (GELU, 1.0, 0.0), (GELU, 1.0, 1.5),
                                            (RELU2, 1.0, 1.0), (NONE, 1.0, 0.5)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R", [30, 6000])
def test_gradient_activations(act, beta, limit, gated, R):
    banner(f"dact {act} beta {beta} limit {limit} gated {gated} R={R}")
    gradient(R, 2, 264, 136, torch.float16, gated, act, beta=beta, limit=limit, weighted=True, seed=act)


@pytest.mark.parametrize("R", [33, 500, 7000])
def test_gradient_leaves_rows_of_no_group(R):
    gradient(R, 3, 136, 264, torch.bfloat16, True, SWI, weighted=True, seed=R, lo=R // 5, hi=R - R // 4)


def test_gradient_of_an_infinite_row_stays_there():
    """Tiles that end past N: the sums of the columns that are not there stay out."""
    for R in (20, 3000):
        g = gen(R)
        N, K = 136, 264
        dy = torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16)
        w = torch.rand((1, K, N), generator=g, device="cuda").to(torch.bfloat16) + 0.5
        pre = torch.rand((R, 2 * N), generator=g, device="cuda").to(torch.bfloat16) + 0.5
        off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
        want = moe.moe_grouped_mm_dact(dy, w, off, pre)
        dy[3] = dy[3].abs()
        dy[3, 7] = INF
        got = moe.moe_grouped_mm_dact(dy, w, off, pre)
        keep = torch.arange(R, device="cuda") != 3
        for n in ("dpre", "h", "dw"):
            assert torch.equal(got[n][keep], want[n][keep]), n
        assert float(got["dw"][3]) == INF and bool((got["dpre"][3] == INF).all())


def test_gradient_against_differences():
    """dpre as the slope of sum(dy . (w_r a(g) u) W2): differences of the
    activation's own 64-bit values with a step of 2^-10; their error is below
    2^-12 of the curvature's bound, the output's rounding 2^-8 of itself."""
    g = gen(4)
    R, N, K, step = 12, 16, 24, 2.0 ** -10
    dy = torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((1, K, N), generator=g, device="cuda").to(torch.bfloat16)
    pre = torch.randn((R, 2 * N), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    rw = torch.rand(R, generator=g, device="cuda")
    for act in (SWI, GELU):
        got = moe.moe_grouped_mm_dact(dy, w, off, pre, epi=moe.Epilogue(act=act), row_w=rw)["dpre"].double()
        dh = dy.double() @ w[0].double()

        def value(z):
            return (dh * rw.double()[:, None] * a64(z[:, :N], act) * z[:, N:]).sum(1)

        for c in range(0, 2 * N, 3):
            up, dn = pre.double(), pre.double()
            up[:, c] += step
            dn[:, c] -= step
            diff = (value(up) - value(dn)) / (2 * step)
            scale = (dh.abs() * (1 + pre.double()[:, :N].abs()) * (1 + pre.double()[:, N:].abs()))[:, c % N]
            assert bool(((got[:, c] - diff).abs() <= 2 ** -12 * scale + 2 ** -8 * diff.abs() * 1.01 + 1e-6).all())


# ------------------------------------------------------------ in a run together
def test_feed_forward_block_with_residual():
    """A dense block out = x + W2 a(W1 x + b1) + b2, forward and backward, against
    64-bit automatic differentiation: each tensor is rounded a few times on the way."""
    g = gen(5)
    R, H, I = 700, 264, 520
    dt = torch.bfloat16
    x = torch.randn((R, H), generator=g, device="cuda").to(dt)
    w1 = (torch.randn((1, I, H), generator=g, device="cuda") * 0.06).to(dt)
    w2 = (torch.randn((1, H, I), generator=g, device="cuda") * 0.04).to(dt)
    b1, b2 = (torch.randn((1, n), generator=g, device="cuda") * 0.2 for n in (I, H))
    dout = torch.randn((R, H), generator=g, device="cuda").to(dt)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    e1 = moe.Epilogue(act=GELU, bias=b1)
    h, pre = moe.moe_grouped_mm_act(x, w1, off, epi=e1, keep_pre=True)
    out = moe.moe_grouped_mm_act(h, w2, off, epi=moe.Epilogue(act=NONE, bias=b2), residual=x)
    o = moe.moe_grouped_mm_dact(dout, w2, off, pre, epi=e1, gated=False, want_dw=False)
    got = dict(out=out, db2=moe.moe_grouped_bias_grad(dout, off), dw2=moe.moe_grouped_wgrad(dout, o["h"], off),
               db1=moe.moe_grouped_bias_grad(o["dpre"], off), dw1=moe.moe_grouped_wgrad(o["dpre"], x, off),
               dx=moe.moe_grouped_mm_act(o["dpre"], w1, off, w_kn=True, residual=dout))
    leaves = [t.double().requires_grad_(True) for t in (x, w1, w2, b1, b2)]
    X, W1, W2, B1, B2 = leaves
    y = X + a64(X @ W1[0].t() + B1, GELU) @ W2[0].t() + B2
    dx, dw1, dw2, db1, db2 = torch.autograd.grad(y, leaves, dout.double())
    want = dict(out=y.detach(), dx=dx, dw1=dw1, dw2=dw2, db1=db1, db2=db2)
    for n, ref in want.items():
        rel = float((got[n].double().view_as(ref) - ref).norm() / ref.norm())
        print(f"  {n}: rel-L2 {rel:.2e}", flush=True)
        assert rel <= 4 * torch.finfo(dt).eps, n


@pytest.mark.parametrize("shape", [(96, 8, 2, 0, 8, 512, 256), (257, 16, 3, 4, 8, 256, 136), (1, 8, 2, 0, 8, 256, 128),
                                   (2500, 4, 2, 0, 4, 512, 264)])
@pytest.mark.parametrize("renorm", [False, True])
def test_routed_training_step(shape, renorm):
    """Route, permute, both products, and every gradient down to the logits,
    against 64-bit automatic differentiation of the same formulas (the
    rounding budget of the existing step's test: four halves of a step, twice)."""
    T, E, k, e0, E_loc, H, I = shape
    banner(f"routed step {shape} renorm={renorm}")
    g = gen(sum(shape))
    dt = torch.bfloat16
    logits = torch.randn((T, E), generator=g, device="cuda")
    x = torch.randn((T, H), generator=g, device="cuda").to(dt)
    w1 = (torch.randn((E_loc, 2 * I, H), generator=g, device="cuda") * 0.05).to(dt)
    w2 = (torch.randn((E_loc, H, I), generator=g, device="cuda") * 0.05).to(dt)
    b1 = torch.randn((E_loc, 2 * I), generator=g, device="cuda") * 0.2
    dout = torch.randn((T, H), generator=g, device="cuda").to(dt)
    flags = moe.MOE_ROUTE_RENORM if renorm else 0

    idx, tw = moe.moe_route(logits, k, flags)
    p = moe.moe_permute(idx, tw, e0, E_loc, False)
    off, src, rw, slots = p["offsets"], p["row_src"], p["row_w"], p["slot_row"]
    epi = moe.Epilogue(bias=b1)
    h, pre = moe.moe_grouped_mm_act(x, w1, off, epi=epi, gated=True, row_src=src, row_w=rw, keep_pre=True)
    out = moe.moe_combine(moe.moe_grouped_mm(h, w2, off), slots, H).view(dt)
    o = moe.moe_grouped_mm_dact(dout, w2, off, pre, epi=epi, dy_src=src, row_w=rw)
    got = dict(out=out, dw2=moe.moe_grouped_wgrad(dout, o["h"], off, dy_src=src),
               db1=moe.moe_grouped_bias_grad(o["dpre"], off), dw1=moe.moe_grouped_wgrad(o["dpre"], x, off, x_src=src),
               dx=moe.moe_combine(moe.moe_grouped_mm(o["dpre"], w1, off, w_kn=True), slots, H).view(dt),
               dlogits=moe.moe_route_backward(logits, idx, o["dw"], slot_row=slots, flags=flags))

    leaves = [t.double().requires_grad_(True) for t in (logits, x, w1, w2, b1)]
    L, X, W1, W2, B1 = leaves
    pr = torch.softmax(L, 1).gather(1, idx.long())
    if renorm:
        pr = pr / pr.sum(1, keepdim=True)
    y = torch.zeros_like(X)
    for e in range(E_loc):
        t, j = torch.nonzero(idx == e + e0, as_tuple=True)
        if t.numel():
            z = X[t] @ W1[e].t() + B1[e]
            y = y.index_add(0, t, pr[t, j][:, None] * (a64(z[:, :I], SWI) * z[:, I:]) @ W2[e].t())
    if not y.requires_grad:                                  # no token chose a local expert
        assert not bool(out.any())
        return
    dl, dx, dw1, dw2, db1 = torch.autograd.grad(y, leaves, dout.double())
    want = dict(out=y.detach(), dx=dx, dw1=dw1, dw2=dw2, db1=db1, dlogits=dl)
    for n, ref in want.items():
        d = float((got[n].double() - ref).norm())
        # the logits' gradient is a difference of dw, whose terms are one size with dout . y
        scale = float((dout.double() * y.detach()).norm()) if n == "dlogits" else float(ref.norm())
        print(f"  {n}: {d / scale:.2e}", flush=True)
        assert d <= 4 * torch.finfo(dt).eps * scale, n


def test_captured_and_on_two_streams():
    g = gen(6)
    cases = []
    for R, G, N, K in ((16, 1, 512, 4096), (300, 2, 264, 520), (6000, 2, 1032, 136)):
        x = torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16)
        w = (torch.randn((G, 2 * N, K), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
        w2 = (torch.randn((G, K, N), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
        off = torch.tensor([R * i // G for i in range(G + 1)], device="cuda", dtype=torch.int32)
        cases.append((x, w, w2, off))

    def all_of(c, stream=None):
        x, w, w2, off = c
        h, pre = moe.moe_grouped_mm_act(x, w, off, gated=True, keep_pre=True, stream=stream)
        o = moe.moe_grouped_mm_dact(x, w2, off, pre, stream=stream)
        return h, pre, o["dpre"], o["h"], o["dw"]

    want = [all_of(c) for c in cases]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [[all_of(c, st[i % 2]) for i, c in enumerate(cases)] for _ in range(5)]
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, want):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [all_of(c) for c in cases]
    for _ in range(3):
        for c in cases:
            c[0].copy_(torch.randn(c[0].shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            assert all(torch.equal(s, t) for s, t in zip(o, all_of(c)))


def test_no_rows():
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 32, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    y, pre = moe.moe_grouped_mm_act(x, w, off, gated=True, keep_pre=True)
    assert y.shape == (0, 16) and pre.shape == (0, 32)
    o = moe.moe_grouped_mm_dact(x[:, :32], w, off, torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda"))
    assert o["dpre"].shape == (0, 128) and o["h"].shape == (0, 64) and o["dw"].shape == (0,)
    # rows without a group: nothing is written
    y = torch.full((9, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_mm_act(torch.ones((9, 64), dtype=torch.bfloat16, device="cuda"), w, off, gated=True, out=y)
    assert bool((y == 7).all())
