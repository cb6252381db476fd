"""The 16-bit and block-scaled FP8 grouped products against plain 64-bit
products of the same inputs, at the sizes where tiles, tails and groups end.

Tolerances. A sum of n products in fp32, in any order, is off by at most
n * 2^-24 of the sum of |products| when every addition rounds to nearest;
2^-23 allows for truncating additions inside a matrix instruction. The output
is then rounded once: eps / 2 of its value. FP8: the inner sums are bounded by
MFMA_REL of the sum of |products| (see gpu_util), the outer ones as above."""
import pytest
import torch

from gpu_util import MFMA_REL, banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")

T16 = [torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def offsets_of(counts):
    c = torch.tensor([0] + list(counts), device="cuda")
    return c.cumsum(0).to(torch.int32)


def check(got, ref, mag, n, what, rel=2.0 ** -23, extra=0.0):
    """|got - ref| <= half a step of the output type + n * rel of the sum of
    |products| (+ extra of it), and close to it in the 2-norm."""
    eps = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny * eps * 2
    d = (got.double() - ref).abs()
    tol = eps * ref.abs() + (n * rel + extra) * mag * (1 + eps) + tiny
    bad = ~(d <= tol)
    worst = float((d / tol).max()) if d.numel() else 0.0
    l2 = float(d.norm() / ref.norm()) if float(ref.norm()) else float(d.norm())
    print(f"  {what}: largest |diff| / tolerance {worst:.3f}, rel-L2 {l2:.2e}", flush=True)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond tolerance"
    assert l2 <= eps + n * 2.0 ** -23 + extra, (what, l2)


def ref_mm(x, w, off, src, kn):
    rows = x.double() if src is None else x.double()[src.long()]
    o = off.tolist()
    R, N = rows.shape[0], w.shape[2 if kn else 1]
    y = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    m = torch.zeros_like(y)
    for g in range(len(o) - 1):
        a = rows[o[g]:o[g + 1]]
        b = w[g].double() if kn else w[g].double().t()
        y[o[g]:o[g + 1]] = a @ b
        m[o[g]:o[g + 1]] = a.abs() @ b.abs()
    return y, m


def ref_wgrad(dy, x, off, N, K):
    o = off.tolist()
    out, mag = [], []
    for lo, hi in zip(o, o[1:]):
        a, b = dy[lo:hi].double().t(), x[lo:hi].double()
        out.append(a @ b)
        mag.append(a.abs() @ b.abs())
    return torch.stack(out), torch.stack(mag)


# rows of each group, N, K
MM = [
    ([1], 8, 8),
    ([0, 1, 0, 2, 0], 64, 72),
    ([3, 0, 5, 8], 136, 200),
    ([16, 1, 0, 15], 512, 512),
    ([17, 31, 33, 2], 264, 1000),
    ([64, 65, 40, 0], 256, 328),
    ([100, 128, 129, 60], 520, 264),
    ([257, 300, 0, 511, 256], 776, 456),
    ([1000, 24], 1416, 2040),
    ([0, 0, 0], 128, 128),
    ([5] * 70, 72, 96),
    ([1, 2, 700, 3], 264, 520),
    # few tiles: the reduction axis is split and joined
    ([16], 1024, 2048),
    ([5, 0, 9], 136, 4096),
    ([70], 256, 4104),
    ([300], 264, 1544),
    ([3000], 264, 520),
    ([2000, 10, 1000], 256, 264),
    ([0, 1300, 0, 0, 64, 1], 72, 136),
]


@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dtype", T16)
@pytest.mark.parametrize("counts,N,K", MM)
def test_mm(counts, N, K, dtype, kn):
    banner(f"mm {counts} N={N} K={K} {dtype} kn={kn}")
    G, R = len(counts), sum(counts)
    g = gen(R * 31 + N)
    off = offsets_of(counts)
    x = randn(g, (R, K), dtype)
    w = randn(g, (G, K, N) if kn else (G, N, K), dtype, 0.05)
    y = moe.moe_grouped_mm(x, w, off, w_kn=kn)
    ref, mag = ref_mm(x, w, off, None, kn)
    check(y, ref, mag, K, "mm")
    if R:
        T = max(1, R // 3)
        src = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
        y = moe.moe_grouped_mm(x[:T], w, off, w_kn=kn, row_src=src)
        ref, mag = ref_mm(x[:T], w, off, src, kn)
        check(y, ref, mag, K, "mm gathered")


def test_mm_strides_and_untouched_rows():
    """Row strides of x and y; rows behind the last group keep what they held,
    and so do the columns beside a strided output."""
    g = gen(5)
    counts, N, K = [33, 0, 70], 200, 136
    R, extra = sum(counts), 29
    off = offsets_of(counts)
    for kn in (False, True):
        xb = randn(g, (R + extra, 2 * K + 8), torch.bfloat16)
        xb[R:] = float("nan")                      # never read into a result
        x = xb[:, K:2 * K]
        w = randn(g, (3, K, N) if kn else (3, N, K), torch.bfloat16, 0.05)
        yb = torch.full((R + extra, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_mm(x, w, off, w_kn=kn, out=yb[:, 8:8 + N])
        ref, mag = ref_mm(x[:R], w, off, None, kn)
        check(yb[:R, 8:8 + N], ref, mag, K, "strided")
        assert torch.all(yb[R:] == 7) and torch.all(yb[:, :8] == 7) and torch.all(yb[:, 8 + N:] == 7)


def test_mm_neighbours_do_not_leak():
    """Infinities and NaN in one group's rows and weights stay in that group,
    and a NaN row stays in its own output row."""
    g = gen(6)
    for counts, K in (([20, 30, 40], 72), ([200, 130, 40], 264), ([3, 5, 2], 520)):
        off = offsets_of(counts)
        R, N = sum(counts), 136
        x, w = randn(g, (R, K), torch.bfloat16), randn(g, (3, N, K), torch.bfloat16)
        lo, hi = counts[0], counts[0] + counts[1]
        x[lo:hi] = float("inf")
        w[1] = float("nan")
        x[R - 1] = float("nan")
        y = moe.moe_grouped_mm(x, w, off)
        ref, mag = ref_mm(x, w, off, None, False)
        keep = torch.ones(R, dtype=torch.bool, device="cuda")
        keep[lo:hi] = False
        keep[R - 1] = False
        check(y[keep], ref[keep], mag[keep], K, "other groups")
        assert torch.isnan(y[lo:hi]).all() and torch.isnan(y[R - 1]).all()
        wk = w.transpose(1, 2).contiguous()
        assert torch.equal(moe.moe_grouped_mm(x, wk, off, w_kn=True)[keep].isfinite(), y[keep].isfinite())


@pytest.mark.parametrize("out", ["fp32", "same"])
@pytest.mark.parametrize("dtype", T16)
@pytest.mark.parametrize("counts,N,K", MM)
def test_wgrad(counts, N, K, dtype, out):
    banner(f"wgrad {counts} N={N} K={K} {dtype} {out}")
    G, R = len(counts), sum(counts)
    g = gen(R * 17 + K)
    off = offsets_of(counts)
    od = torch.float32 if out == "fp32" else dtype
    dy, x = randn(g, (R, N), dtype, 0.1), randn(g, (R, K), dtype)
    n = max(counts) if R else 1
    ref, mag = ref_wgrad(dy, x, off, N, K)
    dw = moe.moe_grouped_wgrad(dy, x, off, out_dtype=od)
    check(dw, ref, mag, n, "wgrad")
    base = randn(g, (G, N, K), od)
    acc = base.clone()
    moe.moe_grouped_wgrad(dy, x, off, out=acc, accumulate=True, out_dtype=od)
    check(acc, ref + base.double(), mag + base.double().abs(), n + 1, "accumulated")
    if R:
        T = max(1, R // 2)
        xs = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
        ds = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
        ref, mag = ref_wgrad(dy[ds.long()], x[xs.long()], off, N, K)
        dw = moe.moe_grouped_wgrad(dy[:T], x[:T], off, dy_src=ds, x_src=xs, out_dtype=od)
        check(dw, ref, mag, n, "wgrad gathered")


def test_wgrad_rows_of_other_groups_do_not_leak():
    g = gen(8)
    for counts in ([37, 64, 90], [3, 1, 2], [200, 300, 10]):
        off = offsets_of(counts)
        R = sum(counts)
        dy, x = randn(g, (R + 9, 72), torch.bfloat16), randn(g, (R + 9, 104), torch.bfloat16)
        lo, hi = counts[0], counts[0] + counts[1]
        x[lo:hi] = float("nan")
        dy[lo:hi] = float("inf")
        x[R:] = float("nan")
        dy[R:] = float("nan")
        dw = moe.moe_grouped_wgrad(dy, x, off)
        ref, mag = ref_wgrad(dy, x, off, 72, 104)
        check(dw[[0, 2]], ref[[0, 2]], mag[[0, 2]], max(counts), "other groups")
        assert torch.isnan(dw[1]).all()


# ------------------------------------------------------------------ FP8
def decode(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double()
    return v * scales.double().repeat_interleave(128, -1)[:, : codes.shape[-1]]


def decode_w(codes, scales):
    G, N, K = codes.shape
    s = scales.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return codes.view(torch.float8_e4m3fn).double() * s


FP8 = [([1], 8, 16), ([0, 1, 0, 2, 0], 64, 80), ([3, 0, 5, 8], 136, 208), ([16, 1, 0, 15], 512, 512),
       ([17, 31, 33, 2], 264, 1008), ([64, 65, 40, 0], 256, 336), ([100, 128, 129, 60], 520, 272),
       ([257, 300, 0, 511, 256], 776, 464), ([1000, 24], 1416, 2048), ([0, 0], 128, 128),
       ([16], 1024, 4096), ([5, 0, 9], 136, 8208), ([300], 264, 3088), ([600, 3], 520, 10256)]


@pytest.mark.parametrize("dtype", T16)
@pytest.mark.parametrize("counts,N,K", FP8)
def test_mm_fp8(counts, N, K, dtype):
    banner(f"fp8 {counts} N={N} K={K} {dtype}")
    G, R = len(counts), sum(counts)
    g = gen(R * 13 + N)
    off = offsets_of(counts)
    xq, xs = moe.moe_quantize_block(randn(g, (R, K), torch.bfloat16))
    wq, ws = moe.moe_quantize_block_weights(randn(g, (G, N, K), torch.bfloat16, 0.05))
    ws = ws * (0.6 + 0.8 * torch.rand(ws.shape, generator=g, device="cuda"))       # any fp32 scale
    xs = xs * (0.6 + 0.8 * torch.rand(xs.shape, generator=g, device="cuda"))
    xd, wd = decode(xq, xs), decode_w(wq, ws)
    y = moe.moe_grouped_mm_fp8(xq, xs, wq, ws, off, out_dtype=dtype)
    ref, mag = ref_mm(xd, wd, off, None, False)
    check(y, ref, mag, K // 128 + 4, "fp8", extra=MFMA_REL)
    if R:
        T = max(1, R // 3)
        src = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
        y = moe.moe_grouped_mm_fp8(xq[:T], xs[:T], wq, ws, off, row_src=src, out_dtype=dtype)
        ref, mag = ref_mm(xd[:T], wd, off, src, False)
        check(y, ref, mag, K // 128 + 4, "fp8 gathered", extra=MFMA_REL)


# ------------------------------------------- weight gradient from 8-bit rows
@pytest.mark.parametrize("counts,N,K", MM)
def test_wgrad_8bit_rows(counts, N, K):
    banner(f"wgrad 8-bit {counts} N={N} K={K}")
    G, R = len(counts), sum(counts)
    g = gen(R * 19 + K)
    off = offsets_of(counts)
    dy, x = randn(g, (R, N), torch.bfloat16, 0.1), randn(g, (R, K), torch.bfloat16)
    xq, xs = moe.moe_quantize_block(x)
    xd = decode(xq, xs)
    n = max(counts) if R else 1
    ref, mag = ref_wgrad(dy, xd, off, N, K)
    dw = moe.moe_grouped_wgrad(dy, xq, off, x_scales=xs)
    check(dw, ref, mag, n, "wgrad 8-bit")
    if R:
        # exactly the product of the decoded rows (power-of-two scales decode exactly to bf16)
        assert torch.equal(dw, moe.moe_grouped_wgrad(dy, xd.to(torch.bfloat16), off))
        T = max(1, R // 2)
        src = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
        ds = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
        ref, mag = ref_wgrad(dy[ds.long()], xd[src.long()], off, N, K)
        acc = torch.ones((G, N, K), device="cuda")
        moe.moe_grouped_wgrad(dy[:T], xq[:T], off, dy_src=ds, x_src=src, x_scales=xs[:T], out=acc, accumulate=True)
        check(acc, ref + 1, mag + 1, n + 1, "wgrad 8-bit gathered, accumulated")
        # rows at a stride that is no multiple of 16, starting at 8
        xw = torch.full((R, K + 24), 0x7F, dtype=torch.uint8, device="cuda")
        xw[:, 8:8 + K] = xq
        assert torch.equal(moe.moe_grouped_wgrad(dy, xw[:, 8:8 + K], off, x_scales=xs), dw)
