"""A training step of the layer in 16 bits, made of the operators as a program
would call them, against 64-bit autograd of the same formulas; the FP8 forward
chain; and the operators under graph capture, on another stream and twice."""
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Step:
    """One expert-parallel share of a layer: T tokens, E experts of which
    E_loc from e0 on are local, top-k, H -> 2I -> H."""

    def __init__(self, T, E, k, e0, E_loc, H, I, seed, dtype=torch.bfloat16):
        g = gen(seed)
        self.k, self.e0, self.E_loc, self.I = k, e0, E_loc, I
        self.logits = torch.randn((T, E), generator=g, device="cuda")
        self.x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
        self.w1 = (torch.randn((E_loc, 2 * I, H), generator=g, device="cuda") * 0.05).to(dtype)
        self.w2 = (torch.randn((E_loc, H, I), generator=g, device="cuda") * 0.05).to(dtype)
        self.dout = torch.randn((T, H), generator=g, device="cuda").to(dtype)

    def run(self, eight=False):
        """Forward and backward; with `eight`, x is kept in 8 bits as well."""
        r = {}
        idx, tw = moe.moe_route(self.logits, self.k)
        p = moe.moe_permute(idx, tw, self.e0, self.E_loc, False)
        off, src, w, slots = p["offsets"], p["row_src"], p["row_w"], p["slot_row"]
        used = off[-1:]
        H = self.x.shape[1]
        # forward: the token rows are read through row_src, nothing is gathered
        pre = moe.moe_grouped_mm(self.x, self.w1, off, row_src=src)
        h, codes, scales = moe.moe_glu_checkpoint(pre, row_w=w, n_rows=used)
        y = moe.moe_grouped_mm(h, self.w2, off)
        r["out"] = moe.moe_combine(y, slots, H).view(self.x.dtype)
        x8 = moe.moe_quantize_block(self.x) if eight else None
        # backward, from the 8-bit pre-activation
        dh = moe.moe_grouped_mm(self.dout, self.w2, off, w_kn=True, row_src=src)
        b = moe.moe_glu_checkpoint_backward(codes, scales, dh, row_w=w, n_rows=used)
        r["dw2"] = moe.moe_grouped_wgrad(self.dout, b["h"], off, dy_src=src)
        if eight:
            r["dw1"] = moe.moe_grouped_wgrad(b["dpre"], x8[0], off, x_src=src, x_scales=x8[1])
        else:
            r["dw1"] = moe.moe_grouped_wgrad(b["dpre"], self.x, off, x_src=src)
        dxr = moe.moe_grouped_mm(b["dpre"], self.w1, off, w_kn=True)
        r["dx"] = moe.moe_combine(dxr, slots, H).view(self.x.dtype)
        R = int(off[-1])
        r["drow_w"], r["rows"] = b["dw"][:R], R
        r["plan"] = (off, src, w)
        r["kept"] = (codes, scales)
        return r

    def reference(self, r):
        """The same step in 64 bits: exact forward, backward through the kept
        pre-activation (as the step's definition says)."""
        off, src, w = r["plan"]
        R, I = r["rows"], self.I
        o = off.tolist()
        src, w = src[:R].long(), w[:R].double()
        q = r["kept"][0][:R].view(torch.float8_e4m3fn).double().view(2 * R, I)
        s = r["kept"][1][:R].double().view(2 * R, -1)
        kept = (q * s.repeat_interleave(128, 1)[:, :I]).view(R, 2 * I)
        x, w1, w2, dout = self.x.double(), self.w1.double(), self.w2.double(), self.dout.double()
        out = torch.zeros_like(x)
        dx = torch.zeros_like(x)
        dw1, dw2 = torch.zeros_like(w1), torch.zeros_like(w2)
        drow = torch.zeros(R, dtype=torch.float64, device="cuda")
        for e in range(self.E_loc):
            a, b = o[e], o[e + 1]
            if a == b:
                continue
            rows = src[a:b]
            pre = x[rows] @ w1[e].t()
            h = torch.nn.functional.silu(pre[:, :I]) * pre[:, I:] * w[a:b, None]
            out.index_add_(0, rows, h @ w2[e].t())
            kp = kept[a:b].clone().requires_grad_(True)
            ww = w[a:b].clone().requires_grad_(True)
            hk = torch.nn.functional.silu(kp[:, :I]) * kp[:, I:] * ww[:, None]
            dh = dout[rows] @ w2[e]
            dpre, dww = torch.autograd.grad(hk, (kp, ww), dh)
            drow[a:b] = dww
            dw2[e] = dout[rows].t() @ hk.detach()
            dw1[e] = dpre.t() @ x[rows]
            dx.index_add_(0, rows, dpre @ w1[e])
        return dict(out=out, dx=dx, dw1=dw1, dw2=dw2, drow_w=drow)


# Bounds in the 2-norm: every 16-bit rounding on the way is a relative error of
# at most eps/2 of its tensor, products carry it on with a factor of at most
# one in the 2-norm for random operands: at most four roundings (pre, h, y, out
# forward; dh, dpre, dxr, dx backward; three before a weight gradient), so
# 4 * eps / 2, twice that for correlation between them. With x in 8 bits the
# weight gradient's operand adds E4M3's half step of 2^-4.
@pytest.mark.parametrize("shape", [(96, 8, 2, 0, 8, 512, 256), (257, 16, 3, 4, 8, 256, 136), (1, 8, 2, 0, 8, 256, 128),
                                   (700, 4, 1, 1, 2, 512, 264)])
@pytest.mark.parametrize("eight", [False, True])
def test_step_against_autograd(shape, eight):
    banner(f"training step {shape} eight={eight}")
    st = Step(*shape, seed=sum(shape))
    r = st.run(eight)
    ref = st.reference(r)
    eps = torch.finfo(torch.bfloat16).eps
    for name in ("out", "dx", "dw1", "dw2", "drow_w"):
        got, want = r[name].double(), ref[name]
        tol = 4 * eps + (2.0 ** -4 if eight and name == "dw1" else 0.0)
        n = float(want.norm())
        rel = float((got - want).norm()) / n if n else float(got.norm())
        print(f"  {name}: rel-L2 {rel:.2e} (bound {tol:.2e})", flush=True)
        assert rel <= tol, (name, rel)


def test_kept_preactivation_is_close_to_the_exact_one():
    """The gradients through the 8-bit pre-activation differ from those through
    the exact one by the rounding's share: E4M3's half step is 2^-4 of a value,
    and dg depends on both halves through factors of at most 2."""
    st = Step(300, 8, 2, 0, 8, 256, 128, seed=5)
    r = st.run()
    off, src, w = r["plan"]
    R, I = r["rows"], st.I
    q = r["kept"][0][:R].view(torch.float8_e4m3fn).double().view(2 * R, I)
    kept = (q * r["kept"][1][:R].double().view(2 * R, -1).repeat_interleave(128, 1)[:, :I]).view(R, 2 * I)
    o = off.tolist()
    pre = torch.cat([st.x[src[a:b].long()].double() @ st.w1[e].double().t() for e, (a, b) in enumerate(zip(o, o[1:]))])
    rel = float((kept - pre).norm() / pre.norm())
    print(f"  kept against exact pre-activation: rel-L2 {rel:.3e}", flush=True)
    assert rel <= 2.0 ** -4


def test_fp8_forward_chain():
    """Block-scaled FP8 forward (rows quantised between the products) against
    the same chain in 64 bits on the decoded weights."""
    g = gen(9)
    T, E, k, H, I = 200, 8, 2, 512, 256
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w1 = (torch.randn((E, 2 * I, H), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    w2 = (torch.randn((E, H, I), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    q1, s1 = moe.moe_quantize_block_weights(w1)
    q2, s2 = moe.moe_quantize_block_weights(w2)
    idx, tw = moe.moe_route(torch.randn((T, E), generator=g, device="cuda"), k)
    p = moe.moe_permute(idx, tw, 0, E, False)
    off, src = p["offsets"], p["row_src"]
    pre = moe.moe_grouped_mm_fp8(*moe.moe_quantize_block(x), q1, s1, off, row_src=src)
    h, _, _ = moe.moe_glu_checkpoint(pre, row_w=p["row_w"], keep=False)
    y = moe.moe_grouped_mm_fp8(*moe.moe_quantize_block(h), q2, s2, off)
    out = moe.moe_combine(y, p["slot_row"], H).view(torch.bfloat16)

    def dec(q, s):
        G, N, K = q.shape
        return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]

    d1, d2, o = dec(q1, s1), dec(q2, s2), off.tolist()
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = src[o[e]:o[e + 1]].long()
        a = x[rows].double() @ d1[e].t()
        hh = torch.nn.functional.silu(a[:, :I]) * a[:, I:] * p["row_w"][o[e]:o[e + 1], None].double()
        ref.index_add_(0, rows, hh @ d2[e].t())
    rel = float((out.double() - ref).norm() / ref.norm())
    print(f"  fp8 chain: rel-L2 {rel:.3e}", flush=True)
    # x and h each rounded once to E4M3 (half a step 2^-4 at most), the first
    # through a product of two nearly linear factors
    assert rel <= 3 * 2.0 ** -4


def test_step_repeats_bit_for_bit():
    st = Step(300, 8, 2, 0, 8, 512, 256, seed=3)
    a, b = st.run(True), st.run(True)
    for name in ("out", "dx", "dw1", "dw2", "drow_w"):
        assert torch.equal(a[name], b[name]), name


def test_captured_step_replays():
    """The operators captured into a graph (with their joining launches), with
    eager work and new inputs between the replays."""
    g = gen(21)
    cases = []
    # one shape per kernel: few rows split along K, tall tiles, weight gradients split and not, FP8
    for R, G, N, K in ((16, 1, 512, 4096), (300, 2, 264, 520), (2000, 1, 264, 264)):
        x = torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16)
        w = torch.randn((G, N, K), generator=g, device="cuda").to(torch.bfloat16)
        dy = torch.randn((R, N), generator=g, device="cuda").to(torch.bfloat16)
        off = torch.tensor([0] + [R * (i + 1) // G for i in range(G)], device="cuda", dtype=torch.int32)
        K16 = K // 16 * 16
        wq, ws = moe.moe_quantize_block_weights(w[:, :, :K16].contiguous())
        cases.append((x, w, dy, off, wq, ws, K16))

    def all_of(c):
        x, w, dy, off, wq, ws, K16 = c
        xq, xs = moe.moe_quantize_block(x[:, :K16])
        return (moe.moe_grouped_mm(x, w, off), moe.moe_grouped_mm(dy, w, off, w_kn=True),
                moe.moe_grouped_wgrad(dy, x, off), moe.moe_grouped_mm_fp8(xq, xs, wq, ws, off))

    for c in cases:
        all_of(c)                                   # first calls outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [all_of(c) for c in cases]
    for rep in range(3):
        for c in cases:
            c[0].copy_(torch.randn(c[0].shape, generator=g, device="cuda"))
            c[2].copy_(torch.randn(c[2].shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for c, got in zip(cases, outs):
            for a, b in zip(got, all_of(c)):
                assert torch.equal(a, b), rep
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Calls in flight together on two streams, each with its own workspace."""
    g = gen(22)
    R, N, K = 16, 512, 4096
    off = torch.tensor([0, R], device="cuda", dtype=torch.int32)
    xs = [torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    w = torch.randn((1, N, K), generator=g, device="cuda").to(torch.bfloat16)
    big = torch.randn((3000, K), generator=g, device="cuda").to(torch.bfloat16)
    boff = torch.tensor([0, 3000], device="cuda", dtype=torch.int32)
    want = [moe.moe_grouped_mm(x, w, off) for x in xs]
    wantg = moe.moe_grouped_wgrad(big[:, :N], big, boff)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(moe.moe_grouped_mm(xs[i], w, off, stream=st[i]))
        gw = moe.moe_grouped_wgrad(big[:, :N], big, boff, stream=st[0])
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])
    assert torch.equal(gw, wantg)
