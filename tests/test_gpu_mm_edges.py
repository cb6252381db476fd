"""The grouped products and weight gradients where a caller leaves the usual
path: arrays longer than the groups, sources outside the array, offsets that do
not ascend, rows past 32-bit byte offsets, and what the bindings refuse."""
import pytest
import torch

from gpu_util import MFMA_REL, banner
from test_gpu_grouped_mm import check, decode, decode_w, gen, randn, ref_mm, ref_wgrad

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")

BF = torch.bfloat16


def i32(v):
    return torch.tensor(v, device="cuda", dtype=torch.int32)


# rows of the arrays, offsets, N, K: few rows split along K, tiles of 32 to 256 rows
RAGGED = [(64, [3, 3, 19], 136, 4096), (200, [0, 7, 7, 90], 264, 520), (700, [128, 140, 600], 520, 264),
          (3000, [1, 2, 2900], 264, 72), (9000, [0, 4000, 4000, 8999], 1032, 264)]


@pytest.mark.parametrize("R,off,N,K", RAGGED)
def test_rows_of_no_group(R, off, N, K):
    """Rows before the first and behind the last group: nothing reads them (they
    hold NaN) and nothing writes theirs."""
    banner(f"no group {R} {off} {N} {K}")
    g, o, G = gen(R + N), i32(off), len(off) - 1
    lo, hi = off[0], off[-1]
    x, dy = randn(g, (R, K), BF), randn(g, (R, N), BF)
    for t in (x, dy):
        t[:lo] = float("nan")
        t[hi:] = float("nan")
    w = randn(g, (G, N, K), BF, 0.1)
    inside = torch.zeros(R, dtype=torch.bool, device="cuda")
    inside[lo:hi] = True

    def rows(y, ref, mag, what, **kw):
        check(y[lo:hi], ref[lo:hi], mag[lo:hi], K, what, **kw)
        assert (y[~inside] == -7).all(), what

    ref, mag = ref_mm(x, w, o, None, False)
    rows(moe.moe_grouped_mm(x, w, o, out=torch.full((R, N), -7.0, dtype=BF, device="cuda")), ref, mag, "mm")
    wk = w.transpose(1, 2).contiguous()
    rows(moe.moe_grouped_mm(x, wk, o, w_kn=True, out=torch.full((R, N), -7.0, dtype=BF, device="cuda")), ref, mag, "kn")
    K16 = K // 16 * 16
    xq, xs = moe.moe_quantize_block(x[:, :K16])
    wq, ws = moe.moe_quantize_block_weights(w[:, :, :K16].contiguous())
    ref, mag = ref_mm(decode(xq, xs), decode_w(wq, ws), o, None, False)
    y = moe.moe_grouped_mm_fp8(xq, xs, wq, ws, o, out=torch.full((R, N), -7.0, dtype=BF, device="cuda"))
    rows(y, ref, mag, "fp8", extra=MFMA_REL)
    ref, mag = ref_wgrad(dy, x, o, N, K)
    check(moe.moe_grouped_wgrad(dy, x, o), ref, mag, R, "wgrad")
    xq, xs = moe.moe_quantize_block(x)
    ref, mag = ref_wgrad(dy, decode(xq, xs), o, N, K)
    check(moe.moe_grouped_wgrad(dy, xq, o, x_scales=xs), ref, mag, R, "wgrad 8-bit")


@pytest.mark.parametrize("counts,N,K", [([16, 3], 136, 4096), ([70], 264, 520), ([300, 1, 0, 511], 520, 264)])
def test_sources_outside_read_as_zero(counts, N, K):
    banner(f"sources {counts} {N} {K}")
    R, G, T = sum(counts), len(counts), 40
    g = gen(R + K)
    o = torch.cat([i32([0]), i32(counts).cumsum(0).to(torch.int32)])
    src = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
    bad = torch.rand(R, generator=g, device="cuda") < 0.3
    wild = torch.tensor([-1, T, 2**31 - 1, -2**31, T + 5], device="cuda", dtype=torch.int32)
    src = torch.where(bad, wild[torch.arange(R, device="cuda") % 5], src)
    x, dy, dx = randn(g, (T, K), BF), randn(g, (T, N), BF), randn(g, (R, N), BF)
    w = randn(g, (G, N, K), BF, 0.1)

    def take(t):                                    # the rows as the definition has them
        return torch.where(bad[:, None], 0.0, t.double()[src.clamp(0, T - 1).long()])

    ref, mag = ref_mm(take(x), w, o, None, False)
    check(moe.moe_grouped_mm(x, w, o, row_src=src), ref, mag, K, "mm")
    check(moe.moe_grouped_mm(x, w.transpose(1, 2).contiguous(), o, w_kn=True, row_src=src), ref, mag, K, "kn")
    K16 = K // 16 * 16
    xq, xs = moe.moe_quantize_block(x[:, :K16])
    wq, ws = moe.moe_quantize_block_weights(w[:, :, :K16].contiguous())
    ref, mag = ref_mm(take(decode(xq, xs)), decode_w(wq, ws), o, None, False)
    check(moe.moe_grouped_mm_fp8(xq, xs, wq, ws, o, row_src=src), ref, mag, K, "fp8", extra=MFMA_REL)
    xq, xs = moe.moe_quantize_block(x)
    for what, xr, kw in (("16-bit", x, {}), ("8-bit", xq, dict(x_scales=xs))):
        xd = take(decode(xq, xs) if kw else x)
        ref, mag = ref_wgrad(dx, xd, o, N, K)
        check(moe.moe_grouped_wgrad(dx, xr, o, x_src=src, **kw), ref, mag, R, what + ", x gathered")
        ref, mag = ref_wgrad(take(dy), xd, o, N, K)
        check(moe.moe_grouped_wgrad(dy, xr, o, dy_src=src, x_src=src, **kw), ref, mag, R, what + ", both gathered")
    ref, mag = ref_wgrad(take(dy), randn(gen(5), (R, K), BF), o, N, K)
    check(moe.moe_grouped_wgrad(dy, randn(gen(5), (R, K), BF), o, dy_src=src), ref, mag, R, "dy gathered")


@pytest.mark.parametrize("off", [[0, 30, 10, 60], [5, -4, 200, 64], [60, 0, 0, 0], [0, 64, 0, 64], [99, 99, 99, 99]])
@pytest.mark.parametrize("R", [64, 600])
def test_offsets_that_do_not_ascend_stay_inside(R, off):
    """Held inside the array: each group is rows [clamp(off[g]), max of that and
    clamp(off[g + 1])); memory around the outputs stays as it was."""
    banner(f"offsets {off} of {R}")
    g = gen(R)
    o = i32([v * R // 64 if abs(v) < 1000 else v for v in off])
    N, K, G = 136, 264, 3
    x, dy, w = randn(g, (R, K), BF), randn(g, (R, N), BF), randn(g, (G, N, K), BF)
    big = torch.full((R + 512, N), -7.0, dtype=BF, device="cuda")
    moe.moe_grouped_mm(x, w, o, out=big[256:256 + R])
    assert (big[:256] == -7).all() and (big[256 + R:] == -7).all()
    dw = torch.full((G + 2, N, K), -7.0, device="cuda")
    moe.moe_grouped_wgrad(dy, x, o, out=dw[1:1 + G])
    assert (dw[0] == -7).all() and (dw[-1] == -7).all()
    c = [min(max(v, 0), R) for v in o.tolist()]
    for i in range(G):
        lo, hi = c[i], max(c[i], c[i + 1])
        ref, mag = ref_wgrad(dy, x, i32([lo, hi]), N, K)
        check(dw[1 + i:2 + i], ref, mag, R, f"group {i}")
    xq, xs = moe.moe_quantize_block(x)
    assert moe.moe_grouped_wgrad(dy, xq, o, x_scales=xs).isfinite().all()


def test_rows_past_4_gib():
    """Rows whose byte offsets need more than 32 bits, read and written."""
    banner("rows past 4 GiB")
    g = gen(3)
    R, K, N, LD = 300000, 72, 136, 8192              # 4.9 GB an array
    o = i32([R - 400, R - 390, R - 3])
    xb = torch.empty((R, LD), dtype=BF, device="cuda")
    yb = torch.empty((R, LD), dtype=BF, device="cuda")
    x, y = xb[:, 40:40 + K], yb[:, 8:8 + N]
    x[R - 500:] = randn(g, (500, K), BF)
    y[R - 500:] = -7.0
    w = randn(g, (2, N, K), BF)
    moe.moe_grouped_mm(x, w, o, out=y)
    lo = R - 400
    xs = x[lo:].contiguous()
    ref, mag = ref_mm(xs, w, o - lo, None, False)
    check(y[lo:R - 3].contiguous(), ref[:-3], mag[:-3], K, "mm past 4 GiB")
    assert (y[R - 500:lo] == -7).all() and (y[R - 3:] == -7).all()
    dy = yb[:, 4096:4096 + N]
    dy[lo:] = randn(g, (400, N), BF)
    ref, mag = ref_wgrad(dy[lo:].contiguous(), xs, o - lo, N, K)
    check(moe.moe_grouped_wgrad(dy, x, o), ref, mag, 400, "wgrad past 4 GiB")


def test_largest_number_of_groups():
    """2049 groups (more than the weight gradient orders by length)."""
    banner("2049 groups")
    g, G, N, K = gen(6), 2049, 16, 24
    counts = torch.randint(0, 4, (G,), generator=g, device="cuda")
    o = torch.cat([i32([0]), counts.cumsum(0).to(torch.int32)])
    R = int(o[-1])
    x, dy, w = randn(g, (R, K), BF), randn(g, (R, N), BF), randn(g, (G, N, K), BF)
    group = torch.repeat_interleave(torch.arange(G, device="cuda"), counts)
    wr = w.double()[group]
    ref, mag = (wr * x.double()[:, None]).sum(-1), (wr * x.double()[:, None]).abs().sum(-1)
    check(moe.moe_grouped_mm(x, w, o), ref, mag, K, "mm")
    outer = dy.double()[:, :, None] * x.double()[:, None]
    ref = torch.zeros((G, N, K), dtype=torch.float64, device="cuda").index_add_(0, group, outer)
    mag = torch.zeros((G, N, K), dtype=torch.float64, device="cuda").index_add_(0, group, outer.abs())
    check(moe.moe_grouped_wgrad(dy, x, o), ref, mag, 4, "wgrad")


def test_bindings_refuse():
    """Refused on the host, before anything is launched."""
    x, w, o = torch.zeros((16, 64), dtype=BF, device="cuda"), torch.zeros((2, 32, 64), dtype=BF, device="cuda"), i32([0, 8, 16])
    dy = torch.zeros((16, 32), dtype=BF, device="cuda")
    q, s = torch.zeros((16, 64), dtype=torch.uint8, device="cuda"), torch.ones((16, 1), device="cuda")
    wq, ws = torch.zeros((2, 32, 64), dtype=torch.uint8, device="cuda"), torch.ones((2, 1, 1), device="cuda")
    pre = torch.zeros((16, 64), dtype=BF, device="cuda")
    bad = [
        lambda: moe.moe_grouped_mm(x.half(), w, o),                            # types differ
        lambda: moe.moe_grouped_mm(x.float(), w.float(), o),
        lambda: moe.moe_grouped_mm(x[:, ::2], w[:, :, :32].contiguous(), o),   # rows not dense
        lambda: moe.moe_grouped_mm(x[:1].expand(16, 64), w, o),                # rows overlap
        lambda: moe.moe_grouped_mm(x, w[:, :, :32], o),                        # w of another K
        lambda: moe.moe_grouped_mm(x, w.transpose(1, 2), o, w_kn=True),        # w not contiguous
        lambda: moe.moe_grouped_mm(x, w, o.long()),
        lambda: moe.moe_grouped_mm(x, w, o[:2]),                               # one group short
        lambda: moe.moe_grouped_mm(x, w, o.cpu()),
        lambda: moe.moe_grouped_mm(x, w, o, row_src=torch.zeros(16, dtype=torch.int64, device="cuda")),
        lambda: moe.moe_grouped_mm(x, w, o, out=torch.zeros((16, 40), dtype=BF, device="cuda")),
        lambda: moe.moe_grouped_mm(x, w, o, out=torch.zeros((16, 32), dtype=torch.float16, device="cuda")),
        lambda: moe.moe_grouped_mm(x[:, 1:57], w[:, :, :56].contiguous(), o),  # rows at odd addresses
        lambda: moe.moe_grouped_mm(x[:, :60].contiguous(), w[:, :, :60].contiguous(), o),   # K not a multiple of 8
        lambda: moe.moe_grouped_wgrad(dy[:8], x, o),                           # numbers of rows differ
        lambda: moe.moe_grouped_wgrad(dy.half(), x, o),
        lambda: moe.moe_grouped_wgrad(dy, x, o, accumulate=True),              # nothing to add to
        lambda: moe.moe_grouped_wgrad(dy, x, o, out_dtype=torch.float16),
        lambda: moe.moe_grouped_wgrad(dy, q, o),                               # codes without scales
        lambda: moe.moe_grouped_wgrad(dy, q, o, x_scales=s[:8]),
        lambda: moe.moe_grouped_wgrad(dy.half(), q, o, x_scales=s),            # 8-bit rows: bf16 only
        lambda: moe.moe_grouped_wgrad(dy, x, o, out=torch.zeros((2, 64, 32), device="cuda")),
        lambda: moe.moe_quantize_block(x.to(torch.float64)),
        lambda: moe.moe_quantize_block(x, n_rows=torch.ones(2, dtype=torch.int32, device="cuda")),
        lambda: moe.moe_quantize_block_weights(w.transpose(1, 2)),
        lambda: moe.moe_grouped_mm_fp8(q, s.half(), wq, ws, o),
        lambda: moe.moe_grouped_mm_fp8(q, s, wq, ws[:1], o),
        lambda: moe.moe_grouped_mm_fp8(q, s, wq, ws, o, out_dtype=torch.float32),
        lambda: moe.moe_grouped_mm_fp8(q[:, :56].contiguous(), s, wq[:, :, :56].contiguous(), ws, o),   # K % 16
        lambda: moe.moe_glu_checkpoint(pre[:, :63]),
        lambda: moe.moe_glu_checkpoint(pre, keep=False, codes=q),
        lambda: moe.moe_glu_checkpoint(pre, row_w=torch.ones(15, device="cuda")),
        lambda: moe.moe_glu_checkpoint(pre, h=pre[:, :32]),
        lambda: moe.moe_glu_checkpoint_backward(q, torch.ones((16, 2, 2), device="cuda"), dy),
        lambda: moe.moe_glu_checkpoint_backward(q[:8], torch.ones((16, 2, 1), device="cuda"), dy),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoeError):
            f()
            print(f"call {i} was accepted", flush=True)
    with pytest.raises(moe.MoeError):                # too many groups
        moe.moe_grouped_mm(x, torch.zeros((2050, 8, 64), dtype=BF, device="cuda"), torch.zeros(2051, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("R,counts", [(1200, [300, 900]), (500, [130, 0, 129, 100]), (20, [3, 17])])
def test_outputs_at_multiples_of_8_bytes(R, counts):
    """Rows of y that start at odd multiples of 8 bytes, columns beside them
    untouched, with every tile height."""
    banner(f"8-byte rows {R} {counts}")
    g, N, K = gen(R), 264, 144
    o = torch.cat([i32([0]), i32(counts).cumsum(0).to(torch.int32)])
    x, w = randn(g, (R, K), BF), randn(g, (len(counts), N, K), BF, 0.1)
    xq, xs = moe.moe_quantize_block(x)
    wq, ws = moe.moe_quantize_block_weights(w)
    used = sum(counts)
    for what in ("mm", "kn", "fp8"):
        yb = torch.full((R + 2, N + 12), -7.0, dtype=BF, device="cuda")
        y = yb[1:1 + R, 4:4 + N]
        if what == "fp8":
            moe.moe_grouped_mm_fp8(xq, xs, wq, ws, o, out=y)
            ref, mag = ref_mm(decode(xq, xs), decode_w(wq, ws), o, None, False)
        else:
            moe.moe_grouped_mm(x, w.transpose(1, 2).contiguous() if what == "kn" else w, o, w_kn=what == "kn", out=y)
            ref, mag = ref_mm(x, w, o, None, False)
        check(y[:used].contiguous(), ref[:used], mag[:used], K, what, extra=MFMA_REL if what == "fp8" else 0.0)
        y[:used] = -7.0
        assert (yb == -7).all(), what


def test_more_groups_than_three_stages_leave_tables_for():
    """2049 groups at a size that asks for tiles of 128 rows."""
    banner("2049 groups, 128 rows")
    g, G, N, K, per = gen(16), 2049, 256, 512, 100
    R = G * per
    x = randn(g, (R, K), BF)
    w = randn(g, (G, N, K), BF, 0.1)
    y = moe.moe_grouped_mm(x, w, torch.arange(0, R + 1, per, device="cuda", dtype=torch.int32))
    for e in (0, 1, 1023, 2047, 2048):
        a, b = x[e * per:(e + 1) * per].double(), w[e].double().t()
        check(y[e * per:(e + 1) * per], a @ b, a.abs() @ b.abs(), K, f"group {e}")
    assert y.isfinite().all()
