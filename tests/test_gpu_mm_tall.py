"""The LDS-tiled grouped products (tiles of 128 and 256 rows), weight gradients
of several rounds of workgroups, and weight scales of more than 64 K-tiles,
against plain 64-bit products. Each shape states the plan that it is there for
and asserts it, so that a change of the cost model cannot take the kernel away
from its tests. (The shapes of test_gpu_grouped_mm.py, the outputs at multiples
of 8 bytes of test_gpu_mm_edges.py and the steps of test_gpu_training_step.py
are planned as tiles of 32 or 64 rows.) Tolerances as in test_gpu_grouped_mm.py."""
import pytest
import torch

from gpu_util import MFMA_REL, banner
from test_gpu_grouped_mm import check, decode, decode_w, gen, offsets_of, randn, ref_mm, ref_wgrad
from test_gpu_training_step import Step

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")

BF, FP16 = torch.bfloat16, torch.float16
LEAD, BEHIND = 3, 6                                  # rows of no group before and behind the groups'


def uneven(seed, G, R):
    """G group sizes that add up to R: empty ones, one row, a tile's rows and one more among them."""
    p = torch.rand(G, generator=torch.Generator().manual_seed(seed)) ** 3
    c = (p / p.sum() * R).long().tolist()
    for i, n in zip((1, G // 2, G - 2, G - 1), (0, 1, 128, 257)):
        if G > 4:
            c[i] = n
    c[c.index(max(c))] += R - sum(c)
    assert min(c) >= 0 and sum(c) == R
    return c


def items(counts, rows, N):
    return sum(-(-c // rows) for c in counts) * -(-N // 256)


def wild_sources(g, R, T):
    """Sources in [0, T) with duplicates, and some outside; which are outside."""
    src = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
    bad = torch.rand(R, generator=g, device="cuda") < 0.1
    out = torch.tensor([-1, T, 2**31 - 1, -2**31, T + 5], device="cuda", dtype=torch.int32)
    return torch.where(bad, out[torch.arange(R, device="cuda") % 5], src), bad


def take(t, src, bad):
    """Rows of t as the definition has them: sources outside read as zero."""
    return torch.where(bad[:, None], 0.0, t.double()[torch.where(bad, 0, src).long()])


def both_ways(call, x, counts, N, K, w, kn, dtype, n, what, extra=0.0, decoded=None):
    """call(x rows, offsets, sources, out) ungathered, with rows of no group (x: NaN) and
    an output at odd multiples of 8 bytes, and gathered from fewer rows with sources outside."""
    g, R = gen(sum(counts) + N), sum(counts)
    total = LEAD + R + BEHIND
    off = offsets_of(counts) + LEAD
    xd = x.double() if decoded is None else decoded
    ref, mag = ref_mm(xd, w, off, None, kn)
    yb = torch.full((total + 2, N + 12), -7.0, dtype=dtype, device="cuda")
    y = yb[1:1 + total, 4:4 + N]
    call(total, None, off, y)
    inside = slice(LEAD, LEAD + R)
    check(y[inside].contiguous(), ref[inside], mag[inside], n, what, extra=extra)
    again = torch.full((total, N), -7.0, dtype=dtype, device="cuda")
    call(total, None, off, again)
    assert torch.equal(again[inside], y[inside]), "a repeat gave other bits"
    y[inside] = -7.0
    assert (yb == -7).all(), "written outside its rows"
    T = R // 3
    src, bad = wild_sources(g, R, T)
    off = offsets_of(counts)
    ref, mag = ref_mm(take(xd[LEAD:LEAD + T], src, bad), w, off, None, kn)
    out = torch.empty((R, N), dtype=dtype, device="cuda")
    call(slice(LEAD, LEAD + T), src, off, out)
    check(out, ref, mag, n, what + " gathered", extra=extra)


# rows of a tile, group sizes, N, K
TALL = [
    (256, [3001, 0, 5000, 17, 3982], 2056, 328),     # several rounds, 6 K-tiles, tails everywhere
    (256, uneven(1, 5, 20000), 1032, 64),            # several rounds of one K-tile
    (256, [2999, 6001, 0], 1032, 264),
    (128, uneven(2, 40, 5000), 2056, 328),           # several rounds
    (128, uneven(3, 16, 6000), 2056, 72),            # of two K-tiles, fewer than stages
    (128, uneven(3, 16, 6000), 2056, 64),            # of one
    (128, [1029, 971], 2056, 520),
]


@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP16])
@pytest.mark.parametrize("case", TALL, ids=lambda c: f"{c[0]}x{sum(c[1])}x{c[2]}x{c[3]}")
def test_mm(case, dtype, kn):
    rows, counts, N, K = case
    R, G = sum(counts), len(counts)
    banner(f"tall mm {rows} rows, {R} x {N} x {K} in {G} groups, {dtype} kn={kn}, {items(counts, rows, N)} items")
    assert moe.moe_grouped_mm_plan(LEAD + R + BEHIND, G, N, K) == (rows, 1)
    assert moe.moe_grouped_mm_plan(R, G, N, K) == (rows, 1)
    g = gen(R + K)
    x = randn(g, (LEAD + R + BEHIND, K), dtype)
    x[:LEAD] = float("nan")
    x[LEAD + R:] = float("nan")
    w = randn(g, (G, K, N) if kn else (G, N, K), dtype, 0.1)

    def call(rows_of, src, off, out):
        moe.moe_grouped_mm(x[rows_of] if src is not None else x, w, off, w_kn=kn, row_src=src, out=out)

    both_ways(call, x, counts, N, K, w, kn, dtype, K, "mm")


TALL_FP8 = [
    (256, [3001, 0, 5000, 17, 3982], 2056, 336),
    (256, uneven(1, 5, 20000), 1032, 64),
    (256, [2999, 6001, 0], 1032, 272),
    (256, [1300, 1700], 8200, 8336),                 # 66 blocks along K: the scales of a second 64, in several rounds
    (128, uneven(2, 40, 5000), 2056, 336),
    (128, uneven(3, 16, 6000), 2056, 64),
    (128, [1029, 971], 2056, 528),
    (128, [1303, 1297], 2056, 8336),
    (32, [4, 3, 0, 5] * 8, 1024, 8336),              # unsplit, and more than 64 blocks along K
]


@pytest.mark.parametrize("dtype", [BF, FP16])
@pytest.mark.parametrize("case", TALL_FP8, ids=lambda c: f"{c[0]}x{sum(c[1])}x{c[2]}x{c[3]}")
def test_mm_fp8(case, dtype):
    rows, counts, N, K = case
    R, G = sum(counts), len(counts)
    banner(f"tall fp8 {rows} rows, {R} x {N} x {K} in {G} groups, {dtype}, {items(counts, rows, N)} items")
    assert moe.moe_grouped_mm_plan(LEAD + R + BEHIND, G, N, K, fp8=True) == (rows, 1)
    assert moe.moe_grouped_mm_plan(R, G, N, K, fp8=True) == (rows, 1)
    g = gen(R + K)
    xq, xs = moe.moe_quantize_block(randn(g, (LEAD + R + BEHIND, K), BF))
    wq, ws = moe.moe_quantize_block_weights(randn(g, (G, N, K), BF, 0.1))
    xs = xs * (0.6 + 0.8 * torch.rand(xs.shape, generator=g, device="cuda"))
    ws = ws * (0.6 + 0.8 * torch.rand(ws.shape, generator=g, device="cuda"))
    xd = decode(xq, xs)
    xq[:LEAD] = 0x7F                                 # NaN codes and scales in rows of no group
    xq[LEAD + R:] = 0x7F
    xs[:LEAD] = float("nan")
    xs[LEAD + R:] = float("nan")

    def call(rows_of, src, off, out):
        at = rows_of if src is not None else slice(None)
        moe.moe_grouped_mm_fp8(xq[at], xs[at], wq, ws, off, row_src=src, out=out)

    both_ways(call, xq, counts, N, K, decode_w(wq, ws), False, dtype, K // 128 + 4, "fp8", extra=MFMA_REL, decoded=xd)


# ---------------------------------------------------------- weight gradients
def dealing(counts, N, K):
    """The weight gradient's items and how they are dealt out, as its kernel adds
    it up: (dealt, items), dealt None where one round holds all."""
    grid, tiles = torch.cuda.get_device_properties(0).multi_processor_count, -(-N // 256) * -(-K // 256)
    part = moe.moe_grouped_wgrad_plan(sum(counts), len(counts), N, K) // 64
    groups = []
    for c in counts:
        nk = -(-c // 64)
        n = max(1, -(-nk // part)) if part else 1
        groups.append((-(-nk // n), n))
    groups.sort(key=lambda e: -e[0])
    length = [k for k, n in groups for _ in range(n * tiles)]
    n = len(length)
    if not grid < n <= 16 * grid:
        return None, n
    ends = []
    for dealt in (0, 1):
        total = [0] * grid
        for rnd in range(-(-n // grid)):
            back = rnd > 0 if dealt else (rnd & 1) and (rnd + 1) * grid <= n
            for slot in range(grid):
                i = rnd * grid + (grid - 1 - slot if back else slot)
                if i < n:
                    total[slot] += length[i] + 4
        ends.append(max(total))
    return int(ends[1] < ends[0]), n


# how the items are dealt out, whether a group is split, group sizes, N, K
WGRAD = [
    (0, True, [2000, 1200, 700, 400, 250, 130, 64, 3], 2816, 1032),
    (1, True, [1700, 900, 500, 300, 200, 150, 100, 64], 2056, 1032),
    (1, True, [2500, 700, 300, 64, 5], 2056, 1544),
    (0, False, [640] * 8, 2056, 1032),
    (0, False, [130, 0] * 12, 1416, 1544),           # short groups, empty ones between
]


@pytest.mark.parametrize("rows", ["16-bit bf16", "16-bit fp16", "8-bit"])
@pytest.mark.parametrize("case", WGRAD, ids=lambda c: f"dealt{c[0]}-{sum(c[2])}x{c[3]}x{c[4]}")
def test_wgrad(case, rows):
    dealt, split, counts, N, K = case
    R, G = sum(counts), len(counts)
    banner(f"wgrad of several rounds, {R} rows in {G} groups, {N} x {K}, {rows}")
    how, n_items = dealing(counts, N, K)
    part = moe.moe_grouped_wgrad_plan(R, G, N, K)
    assert how == dealt and n_items > 256 and (0 < part < max(counts)) == split
    g, dtype = gen(R + N), FP16 if rows.endswith("fp16") else BF
    off = offsets_of(counts)
    dy, x = randn(g, (R, N), dtype, 0.1), randn(g, (R, K), dtype)
    xr, kw, xd = x, {}, x.double()
    if rows == "8-bit":
        xr, xs = moe.moe_quantize_block(x)
        kw, xd = dict(x_scales=xs), decode(xr, xs)
    n = max(counts)
    ref, mag = ref_wgrad(dy, xd, off, N, K)
    dw = moe.moe_grouped_wgrad(dy, xr, off, **kw)
    check(dw, ref, mag, n, "fp32")
    assert torch.equal(moe.moe_grouped_wgrad(dy, xr, off, **kw), dw), "a repeat gave other bits"
    check(moe.moe_grouped_wgrad(dy, xr, off, out_dtype=dtype, **kw), ref, mag, n, "16 bits")
    for out_dtype in (torch.float32, dtype):
        base = randn(g, (G, N, K), out_dtype)
        acc = base.clone()
        moe.moe_grouped_wgrad(dy, xr, off, out=acc, out_dtype=out_dtype, accumulate=True, **kw)
        check(acc, ref + base.double(), mag + base.double().abs(), n + 1, f"added to {out_dtype}")
    T = R // 2
    xsrc, xbad = wild_sources(g, R, T)
    ysrc, ybad = wild_sources(g, R, T)
    if kw:
        kw["x_scales"] = kw["x_scales"][:T]
    ref, mag = ref_wgrad(dy, take(xd[:T], xsrc, xbad), off, N, K)
    check(moe.moe_grouped_wgrad(dy, xr[:T], off, x_src=xsrc, **kw), ref, mag, n, "x gathered")
    ref, mag = ref_wgrad(take(dy[:T], ysrc, ybad), take(xd[:T], xsrc, xbad), off, N, K)
    check(moe.moe_grouped_wgrad(dy[:T], xr[:T], off, x_src=xsrc, dy_src=ysrc, **kw), ref, mag, n, "both gathered")
    if kw:
        kw["x_scales"] = xs
    ref, mag = ref_wgrad(take(dy[:T], ysrc, ybad), xd, off, N, K)
    check(moe.moe_grouped_wgrad(dy[:T], xr, off, dy_src=ysrc, **kw), ref, mag, n, "dy gathered")


# -------------------------------------------------------- as they are used
@pytest.mark.parametrize("T,I,rows", [(4096, 512, 128), (8192, 768, 256)])
def test_training_step(T, I, rows):
    """The layer's step with its products on the LDS-tiled kernel; bounds as in
    test_gpu_training_step.py (roundings on the way, whatever the sizes)."""
    banner(f"training step of {T} tokens")
    E, k, H = 8, 2, 1024
    for N, K in ((2 * I, H), (H, I), (I, H), (H, 2 * I)):
        assert moe.moe_grouped_mm_plan(T * k, E, N, K)[0] == rows
    st = Step(T, E, k, 0, E, H, I, seed=T)
    for eight in (False, True):
        r = st.run(eight)
        ref = st.reference(r)
        for name in ("out", "dx", "dw1", "dw2", "drow_w"):
            tol = 4 * torch.finfo(BF).eps + (2.0 ** -4 if eight and name == "dw1" else 0.0)
            rel = float((r[name].double() - ref[name]).norm() / ref[name].norm())
            print(f"  {name}: rel-L2 {rel:.2e} (bound {tol:.2e})", flush=True)
            assert rel <= tol, (name, rel)


def test_captured_tall_calls_replay():
    """One shape per tile height and type, and a split weight gradient of several
    rounds, captured; new inputs and eager calls between the replays."""
    banner("captured tall calls")
    g = gen(31)
    cases = []
    for rows, counts, N, K in (TALL[0], TALL[3]):
        R, G = sum(counts), len(counts)
        K16 = K // 16 * 16
        assert moe.moe_grouped_mm_plan(R, G, N, K)[0] == rows and moe.moe_grouped_mm_plan(R, G, N, K16, True)[0] == rows
        wq, ws = moe.moe_quantize_block_weights(randn(g, (G, N, K16), BF))
        cases.append((randn(g, (R, K), BF), randn(g, (G, N, K), BF), randn(g, (R, N), BF), offsets_of(counts), wq, ws, K16))
    _, split, counts, N, K = WGRAD[1]
    R = sum(counts)
    grad = (randn(g, (R, N), BF), randn(g, (R, K), BF), offsets_of(counts))

    def all_of():
        out = [moe.moe_grouped_wgrad(*grad), moe.moe_grouped_wgrad(*grad, out_dtype=BF)]
        for x, w, dy, off, wq, ws, K16 in cases:
            xq, xs = moe.moe_quantize_block(x[:, :K16])
            out += [moe.moe_grouped_mm(x, w, off), moe.moe_grouped_mm(dy, w, off, w_kn=True),
                    moe.moe_grouped_mm_fp8(xq, xs, wq, ws, off)]
        return out

    all_of()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = all_of()
    for rep in range(3):
        for t in [grad[0], grad[1]] + [c[0] for c in cases] + [c[2] for c in cases]:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, all_of())):
            assert torch.equal(a, b), (rep, i)
        torch.cuda.synchronize()


def test_gathered_arrays_close_to_4_gib():
    """Sources near the end of arrays of almost 2^32 - 2^22 bytes, the largest that
    rows are gathered from: byte offsets that need all 32 bits."""
    banner("gathered arrays close to 4 GiB")
    g, counts, N, K, LD = gen(41), [2999, 6001, 0], 1032, 264, 8192
    R, T = sum(counts), ((1 << 32) - (1 << 22)) // (2 * LD) - 1
    off = offsets_of(counts)
    assert moe.moe_grouped_mm_plan(R, 3, N, K) == (256, 1)
    buf = torch.empty((T, LD), dtype=BF, device="cuda")
    x = buf[:, LD - K:]                              # the array's last bytes among them
    x[:400] = randn(g, (400, K), BF)
    x[T - 400:] = randn(g, (400, K), BF)
    src = torch.randint(0, 400, (R,), generator=g, device="cuda", dtype=torch.int32)
    src = torch.where(torch.rand(R, generator=g, device="cuda") < 0.8, T - 1 - src, src)
    near = x[src.long()].double()
    w = randn(g, (3, N, K), BF, 0.1)
    ref, mag = ref_mm(near, w, off, None, False)
    check(moe.moe_grouped_mm(x, w, off, row_src=src), ref, mag, K, "mm")
    dy = randn(g, (R, N), BF)
    ref, mag = ref_wgrad(dy, near, off, N, K)
    check(moe.moe_grouped_wgrad(dy, x, off, x_src=src), ref, mag, max(counts), "wgrad, x gathered")
    ref, mag = ref_wgrad(near, dy, off, K, N)
    check(moe.moe_grouped_wgrad(x, dy, off, dy_src=src), ref, mag, max(counts), "wgrad, dy gathered")
    few = offsets_of([3, 0, 9])
    ref, mag = ref_mm(near[:12], w, few, None, False)
    assert moe.moe_grouped_mm_plan(12, 3, N, K)[0] == 32
    check(moe.moe_grouped_mm(x, w, few, row_src=src[:12].contiguous()), ref, mag, K, "few rows")
    del buf, x
    torch.cuda.empty_cache()
