"""The layer for a few tokens against the same formulas in 64 bits."""
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def decoded(q, s):
    G, N, K = q.shape
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]


class Case:
    def __init__(self, T, E, k, e0, E_loc, H, I, dtype="bf16", eight=False, shared=False, bias=False, residual=False,
                 act=moe.MOE_ACT_SWIGLU, limit=0.0, beta=1.0, renorm=False, seed=0):
        g = gen(seed)
        dt = TYPES[dtype]

        def n(*shape, std=1.0, t=dt):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(t)

        def weights(c):
            w1, w2 = n(c, 2 * I, H, std=H ** -0.5), n(c, H, I, std=I ** -0.5)
            if not eight:
                return w1, None, w2, None
            q1, s1 = moe.moe_quantize_block_weights(w1)
            q2, s2 = moe.moe_quantize_block_weights(w2)
            # scales that are no powers of two
            return q1, s1 * (torch.rand(s1.shape, generator=g, device="cuda") + 0.5), q2, s2 * 1.25

        self.T, self.E, self.k, self.e0, self.H, self.I, self.dt = T, E, k, e0, H, I, dt
        self.logits = n(T, E, t=torch.float32)
        self.x = n(T, H)
        self.w1, self.s1, self.w2, self.s2 = weights(E_loc)
        self.shared = weights(1) if shared else None
        G = E_loc + int(shared)
        self.b1 = n(G, 2 * I, std=0.3, t=torch.float32) if bias else None
        self.b2 = n(G, H, std=0.3, t=torch.float32) if bias else None
        self.res = n(T, H) if residual else None
        self.act, self.limit, self.beta = act, limit, beta
        self.flags = moe.MOE_ROUTE_RENORM if renorm else 0

    def run(self, **kw):
        epi = moe.Epilogue(act=self.act, beta=self.beta, limit=self.limit, bias=self.b1)
        a = dict(e0=self.e0, w1_scales=self.s1, w2_scales=self.s2, shared=self.shared, epi=epi, bias2=self.b2,
                 residual=self.res, flags=self.flags)
        a.update(kw)
        return moe.moe_layer_few(self.logits, a.pop("x", self.x), self.w1, self.w2, self.k, **a)

    def act64(self, z):
        if self.act == moe.MOE_ACT_GEGLU:
            return z * 0.5 * torch.erfc(z * -0.5 ** 0.5)          # (ndtr loses the tail: 2% at -8)
        if self.act == moe.MOE_ACT_SRELU:
            return torch.relu(z) ** 2
        return z if self.act == moe.MOE_ACT_NONE else z * torch.sigmoid(self.beta * z)

    def reference(self):
        """(out, bound): the layer in 64 bits and a bound on the kernel's error.
        u is half a step of the type. h is rounded once (u |h|), the sums of the
        first product are off by at most 2^-18 of their |terms| (fewer than 64
        roundings of 2^-24 follow one another), which the activation carries on
        with a slope of at most 1.2 (beta 1; squared ReLU 2 |z|) and the other
        factor; the second product adds 2^-18 of its own, the output one u."""
        u = torch.finfo(self.dt).eps / 2
        order = torch.sort(self.logits, dim=1, descending=True, stable=True)[1][:, :self.k]
        p = torch.softmax(self.logits.double(), 1).gather(1, order)
        if self.flags:
            p = p / p.sum(1, keepdim=True)
        w1 = decoded(self.w1, self.s1) if self.s1 is not None else self.w1.double()
        w2 = decoded(self.w2, self.s2) if self.s2 is not None else self.w2.double()
        if self.shared is not None:
            a, sa, b, sb = self.shared
            w1 = torch.cat([w1, decoded(a, sa) if sa is not None else a.double()])
            w2 = torch.cat([w2, decoded(b, sb) if sb is not None else b.double()])
        n_loc = self.w1.shape[0]
        x = self.x.double()
        out = self.res.double().clone() if self.res is not None else torch.zeros_like(x)
        tol = out.abs() * 2 ** -22
        cut = self.limit if self.limit > 0 else float("inf")
        for t in range(self.T):
            picks = [(int(order[t, j]) - self.e0, float(p[t, j])) for j in range(self.k)]
            picks = [(g, w) for g, w in picks if 0 <= g < n_loc] + ([(n_loc, 1.0)] if self.shared is not None else [])
            for g, w in picks:
                z, zm = w1[g] @ x[t], w1[g].abs() @ x[t].abs()
                if self.b1 is not None:
                    z, zm = z + self.b1[g].double(), zm + self.b1[g].double().abs()
                gz, uz = z[:self.I].clamp(-cut, cut), z[self.I:].clamp(-cut, cut)
                dg, du = 2 ** -18 * zm[:self.I], 2 ** -18 * zm[self.I:]
                a = self.act64(gz)
                h = a * uz * w
                slope = 2 * (gz.abs() + dg) if self.act == moe.MOE_ACT_SRELU else 1.2 * max(self.beta, 1.0)
                dh = w * (slope * dg * (uz.abs() + du) + a.abs() * du) + h.abs() * (u + 2 ** -19)
                y, ym = w2[g] @ h, w2[g].abs() @ h.abs()
                if self.b2 is not None:
                    y, ym = y + w * self.b2[g].double(), ym + w * self.b2[g].double().abs()
                out[t] += y
                tol[t] += w2[g].abs() @ dh + 2 ** -18 * ym
        return out, tol + u * (out.abs() + tol) + torch.finfo(self.dt).tiny * u

    def check(self, got):
        ref, tol = self.reference()
        bad = (got.double() - ref).abs() / tol
        print(f"  largest error / bound {float(bad.max()) if bad.numel() else 0:.3f}", flush=True)
        assert bool((bad <= 1).all())


SHAPES = [
    dict(T=1, E=8, k=2, e0=0, E_loc=8, H=256, I=128),
    dict(T=1, E=64, k=6, e0=0, E_loc=64, H=520, I=264, renorm=True),
    dict(T=2, E=5, k=1, e0=4, E_loc=1, H=8, I=8),                       # the smallest sizes, most tokens without an expert
    dict(T=7, E=250, k=8, e0=13, E_loc=40, H=1048, I=120, residual=True),
    dict(T=16, E=8, k=2, e0=0, E_loc=8, H=512, I=256, shared=True, bias=True, residual=True),
    dict(T=17, E=16, k=4, e0=8, E_loc=8, H=264, I=72, bias=True, limit=0.7),
    dict(T=32, E=4, k=4, e0=0, E_loc=4, H=136, I=1032, shared=True, renorm=True),
    dict(T=32, E=300, k=8, e0=0, E_loc=300, H=72, I=40, residual=True),
    dict(T=31, E=1000, k=20, e0=500, E_loc=500, H=64, I=16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(s[n]) for n in ("T", "E", "k", "E_loc", "H", "I")))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", [moe.MOE_ACT_SWIGLU, moe.MOE_ACT_GEGLU])
def test_16bit_weights(shape, dtype, act):
    banner(f"few layer {shape} {dtype} act {act}")
    c = Case(dtype=dtype, act=act, seed=shape["T"] * 7 + act, **shape)
    c.check(c.run())


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(s[n]) for n in ("T", "E", "k", "E_loc", "H", "I")))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_8bit_weights(shape, dtype):
    shape = dict(shape, H=-(-shape["H"] // 16) * 16, I=-(-shape["I"] // 16) * 16)
    banner(f"few layer, E4M3 weights {shape} {dtype}")
    c = Case(dtype=dtype, eight=True, seed=shape["T"] * 5, **shape)
    c.check(c.run())


@pytest.mark.parametrize("act,beta,limit", [(moe.MOE_ACT_SRELU, 1.0, 0.0), (moe.MOE_ACT_NONE, 1.0, 0.5),
                                            (moe.MOE_ACT_SWIGLU, 1.7, 1.0)])
def test_activations(act, beta, limit):
    c = Case(T=5, E=8, k=3, e0=0, E_loc=8, H=256, I=136, act=act, beta=beta, limit=limit, bias=True, seed=act)
    c.check(c.run())


def test_every_expert_local_with_most_groups():
    """2048 experts and the shared one, 31 choices each: the tables at their largest."""
    c = Case(T=32, E=2048, k=31, e0=0, E_loc=2048, H=16, I=8, shared=True, seed=3)
    c.check(c.run())


def test_long_reduction():
    """Rows of 7168 and 2560: many units to a wave, several batches."""
    c = Case(T=3, E=4, k=2, e0=0, E_loc=2, H=7168, I=2560, shared=True, seed=4)
    c.check(c.run())
    c = Case(T=20, E=4, k=2, e0=0, E_loc=2, H=7168, I=2560, eight=True, dtype="fp16", seed=5)
    c.check(c.run())


def test_no_local_expert_and_no_token():
    c = Case(T=4, E=8, k=1, e0=7, E_loc=1, H=64, I=32, residual=True, seed=1)
    c.logits[:, 7] = -50.0
    assert torch.equal(c.run(), c.res)
    out = torch.full((4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(residual=None, out=out)
    assert bool((out == 0).all())
    assert moe.moe_layer_few(c.logits[:0], c.x[:0], c.w1, c.w2, 1).shape == (0, 64)


def test_ties_go_to_the_lower_expert():
    c = Case(T=6, E=8, k=2, e0=0, E_loc=8, H=64, I=32, seed=2)
    c.logits.zero_()
    c.check(c.run())


def test_other_tokens_experts_stay_out():
    """Infinities and NaN in an expert's weights, or in a token's row, reach
    the tokens that chose it and no other."""
    for eight in (False, True):
        c = Case(T=18, E=4, k=1, e0=0, E_loc=4, H=128, I=64, eight=eight, seed=6)
        pick = torch.arange(18, device="cuda") % 4
        c.logits.zero_()
        c.logits[torch.arange(18), pick] = 5.0
        want = c.run()
        c.x[4] = float("nan")                               # an expert-0 token
        if eight:
            c.w2[2, :, 3] = 0x7F
        else:
            c.w2[2, :, 3] = float("inf")
            c.w1[2, 0, :] = float("nan")
        got = c.run()
        hit = (pick == 2) | (torch.arange(18, device="cuda") == 4)
        assert torch.equal(got[~hit], want[~hit])
        assert not bool(torch.isfinite(got[hit]).all(1).any())


@pytest.mark.parametrize("T,k", [(16, 8), (32, 8), (12, 4)])
@pytest.mark.parametrize("bits", [-1, 0x7FC00000, 0xFFC00000 - (1 << 32)])
def test_nan_logits_stay_in_their_token(T, k, bits):
    """Every kind of NaN in a token's logits, all of them or one: its row is NaN, the others are as without."""
    c = Case(T=T, E=8, k=k, e0=0, E_loc=8, H=128, I=64, seed=T + k)
    ref, tol = c.reference()
    c.logits.view(torch.int32)[3] = bits
    c.logits.view(torch.int32)[5, 2] = bits
    got = c.run()
    assert bool(got[[3, 5]].isnan().all())
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[[3, 5]] = False
    assert bool(((got.double() - ref).abs() <= tol)[rest].all())


def test_masked_logits():
    """Experts masked by -inf: chosen last, with weight 0; fewer than k left to a token."""
    c = Case(T=20, E=12, k=3, e0=2, E_loc=8, H=128, I=64, residual=True, renorm=True, seed=9)
    c.logits[:, 1::2] = -float("inf")
    c.logits[4, 1:] = -float("inf")
    c.check(c.run())


def test_every_e4m3_code_is_exact():
    """Weights of every code, x and h powers of two: sums of exact products."""
    codes = torch.arange(256, device="cuda", dtype=torch.uint8)
    ok = codes.view(torch.float8_e4m3fn).double().isfinite()
    for dt in (torch.bfloat16, torch.float16):
        H = 256
        w1 = torch.zeros((1, 2 * 16, H), dtype=torch.uint8, device="cuda")
        w1[0, 0] = 0x38                                     # gate row 0: ones
        w1[0, 16] = 0x38
        w2 = torch.zeros((1, H, 16), dtype=torch.uint8, device="cuda")
        w2[0, :, 0] = torch.where(ok, codes, torch.zeros_like(codes))
        one = lambda a: torch.ones((1, -(-a.shape[1] // 128), -(-a.shape[2] // 128)), device="cuda")  # noqa: E731
        x = torch.zeros((1, H), dtype=dt, device="cuda")
        x[0, 0] = 2.0
        out = moe.moe_layer_few(torch.zeros((1, 1), device="cuda"), x, w1, w2, 1, w1_scales=one(w1), w2_scales=one(w2),
                                epi=moe.Epilogue(act=moe.MOE_ACT_NONE))
        want = 4.0 * w2[0, :, 0].view(torch.float8_e4m3fn).double()
        assert torch.equal(out[0].double(), want)
        # and through the first product: h_i = (x . code row)^2 with one column set
        w1[0, :16] = 0
        w1[0, 16:] = 0
        w2.zero_()
        w2[0, 0, 0] = 0x38
        for lo in range(0, 256, 64):
            for c in range(lo, lo + 64, 13):
                if not bool(ok[c]):
                    continue
                w1[0, 0, 0], w1[0, 16, 0] = c, 0x38
                out = moe.moe_layer_few(torch.zeros((1, 1), device="cuda"), x, w1, w2, 1, w1_scales=one(w1),
                                        w2_scales=one(w2), epi=moe.Epilogue(act=moe.MOE_ACT_NONE))
                assert float(out[0, 0]) == 4.0 * float(codes[c].view(torch.float8_e4m3fn).double()), c


def test_strides_in_place_and_repeats():
    c = Case(T=9, E=8, k=2, e0=0, E_loc=8, H=256, I=64, residual=True, seed=8)
    want = c.run()
    wide = torch.full((9, 512), 3.0, dtype=c.dt, device="cuda")
    wide[:, :256] = c.x
    outw = torch.full((9, 300), 5.0, dtype=c.dt, device="cuda")
    outw[:, 4:260] = c.res
    got = c.run(x=wide[:, :256], residual=outw[:, 4:260], out=outw[:, 4:260])      # the residual's own place
    assert torch.equal(got, want)
    assert bool((outw[:, :4] == 5.0).all()) and bool((outw[:, 260:] == 5.0).all())
    for _ in range(5):
        assert torch.equal(c.run(), want)


def test_captured_and_on_two_streams():
    a = Case(T=4, E=16, k=2, e0=0, E_loc=16, H=512, I=128, seed=9)
    b = Case(T=24, E=16, k=4, e0=0, E_loc=16, H=256, I=64, eight=True, seed=10)
    a.run(), b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = a.run(), b.run()
    g = gen(11)
    for _ in range(3):
        for c in (a, b):
            c.x.copy_(torch.randn(c.x.shape, generator=g, device="cuda"))
            c.logits.copy_(torch.randn(c.logits.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for c, got in zip((a, b), outs):
            assert torch.equal(got, c.run())
    want = a.run(), b.run()
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [[c.run(stream=s) for c, s in zip((a, b), st)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(32, 64, 2, 7168, 64), (12, 64, 2, 16384, 48), (20, 40, 1, 5120, 40), (3, 8, 2, 40000, 16)])
def test_groups_that_fit_lds_beside_groups_that_do_not(eight, T, E, k, H, I):
    """Long rows and a shared expert of all tokens: some groups' rows are staged, others read from memory."""
    H, I = (H // 16 * 16, -(-I // 16) * 16) if eight else (H, I)
    c = Case(T=T, E=E, k=k, e0=0, E_loc=E, H=H, I=I, eight=eight, shared=True, bias=True, residual=True, seed=T + eight)
    c.check(c.run())


@pytest.mark.parametrize("H", [64, 520, 1032, 2048, 2064, 4104])
@pytest.mark.parametrize("eight", [False, True])
def test_rows_split_among_waves(H, eight):
    """Every number of waves that share a row, with units past the row's end."""
    H = -(-H // 16) * 16 if eight else H
    c = Case(T=6, E=24, k=3, e0=3, E_loc=17, H=H, I=304, eight=eight, renorm=True, residual=True, seed=H)
    c.check(c.run())
