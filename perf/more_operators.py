"""Measured cases of the products with an epilogue, their backward pass, the
layer for a few tokens and the router's gradient.

Each case is one call of a user's program on tensors that the program already
holds: token rows, expert weights, biases, the group offsets on the device, the
router's logits. `own` selects the side: the library's calls, or the plain form
in elementary torch operations.

  act    y = residual + w_r a(x[src] . W_g^T + b_g), a gated or not, with the pre-activation kept on request
  dact   its backward pass up to the pre-activation: the product dy[src] . W_g, the activation's gradient,
         the activation again and the gradient of the row's weight
  bgrad  gradient of a bias, db_g = sum over the group's rows of w_r dy[src]
  few    the whole routed layer for up to 32 tokens on 16-bit weights or E4M3 weights with a scale per 128 x 128
  route  gradient of the router's logits, load-balancing and z terms included
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
SILU, GELU, RELU2, NONE = 0, 1, 2, 3                            # the library's MOE_ACT_* numbers


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token on two experts of a small model: latency
        dict(name="act-one-token", op="act", type="bf16", rows=2, tokens=1, G=8, cols=256, K=512, kn=False, gated=True,
             act=SILU, limit=0.0, bias=True, weighted=True, residual=False, keep=False, skew=0.0),
        # training forward over one GPU's experts: gate and up products, activation, routing weight, and what the
        # backward pass needs; skewed popularity, rows gathered from token order
        dict(name="act-forward", op="act", type="bf16", rows=24576, tokens=16384, G=16, cols=1408, K=2048, kn=False,
             gated=True, act=SILU, limit=0.0, bias=True, weighted=True, residual=False, keep=True, skew=1.1),
        # an always-on expert's second product: bias and the residual stream, an odd number of rows
        dict(name="act-residual", op="act", type="fp16", rows=8191, tokens=0, G=1, cols=4104, K=4096, kn=True, gated=False,
             act=NONE, limit=0.0, bias=True, weighted=False, residual=True, keep=False, skew=0.0),
        # backward pass of act-forward: dy in token order, W2 as the forward pass holds it
        dict(name="dact-grouped", op="dact", type="bf16", rows=24576, tokens=16384, G=16, cols=1408, K=2048, kn=True,
             gated=True, act=SILU, limit=0.0, weighted=True, skew=1.1),
        # the same of one dense feed-forward network without a gate; odd sizes
        dict(name="dact-dense", op="dact", type="fp16", rows=4099, tokens=0, G=1, cols=4096, K=2040, kn=True,
             gated=False, act=RELU2, limit=0.0, weighted=False, skew=0.0),
        # bias gradient of the gate and up products: many uneven groups
        dict(name="bgrad-grouped", op="bgrad", type="bf16", rows=24576, tokens=0, G=16, cols=2816, weighted=False,
             skew=1.1),
        # bias gradient behind the routing weight, from token order, one long group
        dict(name="bgrad-weighted", op="bgrad", type="fp16", rows=8191, tokens=8192, G=1, cols=4104, weighted=True,
             skew=0.0),
        # one token of a model whose experts are all local: the weights of 6 of 64 experts
        dict(name="few-one-token", op="few", type="bf16", eight=False, T=1, E=64, e0=0, E_loc=64, k=6, H=2048, I=1408,
             act=SILU, limit=0.0, bias=False, shared=False, residual=False, renorm=False),
        # a decode batch on one GPU's share of an expert-parallel layer, 8-bit weights
        dict(name="few-decode-8bit", op="few", type="bf16", eight=True, T=16, E=256, e0=0, E_loc=32, k=8, H=7168,
             I=2048, act=SILU, limit=0.0, bias=False, shared=False, residual=False, renorm=True),
        # a small layer with everything: biases, clamp, shared expert, residual; latency
        dict(name="few-small", op="few", type="fp16", eight=False, T=8, E=8, e0=0, E_loc=8, k=2, H=512, I=264,
             act=GELU, limit=7.0, bias=True, shared=True, residual=True, renorm=True),
        # a training batch's router: balance and z terms, every expert local
        dict(name="route-training", op="route", T=16384, E=64, k=6, E_loc=64, e0=0, renorm=False, aux=True),
        # many experts, some of which live on other GPUs; normalised weights
        dict(name="route-share", op="route", T=4099, E=250, k=8, E_loc=32, e0=16, renorm=True, aux=False),
    ]


def _log(rng, lo, hi, step):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v / step + 0.5) * step)


def draw(rng):
    while True:
        op = rng.choice(["act", "dact", "bgrad", "few", "route"])
        c = dict(op=op)
        if op == "route":
            E = _log(rng, 4, 512, 1)
            k = rng.randint(1, min(8, E))
            part = rng.random() < 0.5
            E_loc = rng.randint(1, E) if part else E
            return dict(c, T=_log(rng, 1, 16384, 1), E=E, k=k, E_loc=E_loc, e0=rng.randint(0, E - E_loc),
                        renorm=rng.random() < 0.5, aux=rng.random() < 0.5)
        c["type"] = rng.choice(["bf16", "fp16"])
        if op == "few":
            eight = rng.random() < 0.5
            step = 16 if eight else 8
            E = _log(rng, 4, 256, 1)
            E_loc = E if rng.random() < 0.4 else rng.randint(1, min(E, 64))
            c.update(eight=eight, T=_log(rng, 1, 32, 1), E=E, E_loc=E_loc, e0=rng.randint(0, E - E_loc),
                     k=rng.randint(1, min(8, E)), H=_log(rng, 256, 7168, step), I=_log(rng, 128, 2560, step),
                     act=rng.choice([SILU, SILU, GELU, RELU2]), limit=rng.choice([0.0, 0.0, 4.0]),
                     bias=rng.random() < 0.3, shared=rng.random() < 0.3, residual=rng.random() < 0.5,
                     renorm=rng.random() < 0.5)
            weights = (E_loc + c["shared"]) * 3 * c["H"] * c["I"]
            if weights <= 1.5e9 and work(c)["bytes"] <= 6.5e8:
                return c
            continue
        c.update(rows=_log(rng, 1, 24576, 1), tokens=rng.choice([0, _log(rng, 1, 16384, 1)]), G=_log(rng, 1, 64, 1),
                 cols=_log(rng, 128, 4104, 8), weighted=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.1]))
        if op != "bgrad":
            gated = rng.random() < 0.5
            c.update(K=_log(rng, 256, 7168, 8), gated=gated, limit=rng.choice([0.0, 0.0, 3.0]),
                     act=rng.choice([SILU, GELU, RELU2] if gated else [SILU, GELU, RELU2, NONE]))
            if op == "act":
                c.update(kn=not gated and rng.random() < 0.5, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                         keep=rng.random() < 0.5)
            else:
                c["kn"] = rng.random() < 0.7
        w = work(c)
        weights = c["G"] * _wide(c) * c.get("K", 0)
        if w["flops"] <= 2.9e11 and w["bytes"] <= 6.5e8 and weights <= 2.4e8:
            return c


def _wide(c):
    """Columns of an act case's product (gate and up), or of the others' rows."""
    return 2 * c["cols"] if c["op"] == "act" and c["gated"] else c["cols"]


def work(c):
    op = c["op"]
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 8 * T * E + 8 * T * k, "flops": 8 * T * E}
    if op == "few":
        T, H, I, s = c["T"], c["H"], c["I"], int(c["shared"])
        hit = 1 - (1 - c["k"] / c["E"]) ** T                    # chance that an expert has a token
        active = max(1.0, c["E_loc"] * hit) + s
        per = 3 * H * I * (1 if c["eight"] else 2) + (2 * (2 * I + H) * 2 if c["bias"] else 0)
        rows = T * c["k"] * c["E_loc"] / c["E"] + s * T
        return {"bytes": int(active * per + 4 * T * H + 4 * T * c["E"] + 2 * T * H * c["residual"]),
                "flops": int(6 * rows * H * I)}
    R, N, src = c["rows"], c["cols"], min(c["tokens"] or c["rows"], c["rows"])
    wr = 4 * R if c["weighted"] else 0
    if op == "bgrad":
        return {"bytes": 2 * src * N + wr + 4 * c["G"] * N, "flops": 2 * R * N}
    K, busy, wide = c["K"], min(c["G"], R), _wide(c)
    if op == "act":
        b = 2 * src * K + 2 * busy * wide * K + 2 * R * N + wr
        b += (4 * busy * wide if c["bias"] else 0) + (2 * R * N if c["residual"] else 0) + (2 * R * wide if c["keep"] else 0)
        return {"bytes": b, "flops": 2 * R * wide * K}
    pre = 2 * N if c["gated"] else N
    return {"bytes": 2 * src * K + 2 * busy * N * K + 4 * R * pre + 2 * R * N + 4 * R + wr, "flops": 2 * R * N * K}


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case

    def normal(shape, std, dtype):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        flat = out.view(-1)
        step = 1 << 26
        for i in range(0, flat.numel(), step):                  # in pieces: no 32-bit copy of the whole
            n = min(step, flat.numel() - i)
            flat[i:i + n] = torch.randn(n, generator=g, device="cuda") * std
        return out

    def eight(G, N, K):
        """Weights that were quantised once: E4M3 codes, any 32-bit scale per 128 x 128 block."""
        q = torch.empty((G, N, K), dtype=torch.uint8, device="cuda")
        for e in range(G):
            v = torch.randn((N, K), generator=g, device="cuda") * (E4M3_MAX / 4)
            q[e] = v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        sc = torch.rand((G, -(-N // BLOCK), -(-K // BLOCK)), generator=g, device="cuda") * 0.8 + 0.6
        return q, sc * (0.08 / E4M3_MAX)

    s = dict(case=c)
    if c["op"] == "route":
        T, k = c["T"], c["k"]
        s["logits"] = normal((T, c["E"]), 1.0, torch.float32)
        # the chosen experts, and the grouped rows that their weights' gradients come in (-1: another GPU's expert)
        s["idx"] = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
        local = (s["idx"] >= c["e0"]) & (s["idx"] < c["e0"] + c["E_loc"])
        order = torch.randperm(T * k, generator=g, device="cuda").view(T, k)
        s["slots"] = torch.where(local, order, -1).to(torch.int32)
        s["dw"] = normal((T * k,), 0.5, torch.float32)
        s["prob_grad"] = normal((c["E"],), 0.1, torch.float32) / T if c["aux"] else None
        s["z_coef"] = 1e-3 / T if c["aux"] else 0.0
        return s

    dt = TYPES[c["type"]]
    if c["op"] == "few":
        T, H, I, G = c["T"], c["H"], c["I"], c["E_loc"]
        s["logits"] = normal((T, c["E"]), 1.0, torch.float32)
        s["x"] = normal((T, H), 1.0, dt)
        s["residual"] = normal((T, H), 1.0, dt) if c["residual"] else None

        def pair(n):
            if c["eight"]:
                return eight(n, 2 * I, H) + eight(n, H, I)
            return normal((n, 2 * I, H), 0.02, dt), None, normal((n, H, I), 0.02, dt), None

        s["w1"], s["s1"], s["w2"], s["s2"] = pair(G)
        s["shared"] = pair(1) if c["shared"] else None
        n = G + int(c["shared"])
        s["b1"] = normal((n, 2 * I), 0.2, torch.float32) if c["bias"] else None
        s["b2"] = normal((n, H), 0.2, torch.float32) if c["bias"] else None
        return s

    R, G, T, N = c["rows"], c["G"], c["tokens"], c["cols"]
    p = torch.arange(1, G + 1, device="cuda", dtype=torch.float32) ** -c["skew"]
    p = p[torch.randperm(G, generator=g, device="cuda")]
    counts = torch.bincount(torch.multinomial(p, R, replacement=True, generator=g), minlength=G)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["bounds"] = s["offsets"].tolist()                         # for the plain form
    s["src"] = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32) if T else None
    s["row_w"] = torch.rand(R, generator=g, device="cuda") * 0.9 + 0.05 if c["weighted"] else None
    rows = T or R
    if c["op"] == "bgrad":
        s["dy"] = normal((rows, N), 0.1, dt)
        return s
    K, wide = c["K"], _wide(c)
    s["w"] = normal((G, K, wide) if c["kn"] else (G, wide, K), 0.02, dt)
    if c["op"] == "act":
        s["x"] = normal((rows, K), 1.0, dt)
        s["bias"] = normal((G, wide), 0.2, torch.float32) if c["bias"] else None
        s["residual"] = normal((R, N), 1.0, dt) if c["residual"] else None
    else:
        s["dy"] = normal((rows, K), 0.1, dt)
        s["pre"] = normal((R, 2 * N if c["gated"] else N), 1.5, dt)
    return s


# ------------------------------------------------------------------- one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import routed_grouped_gemm_amd as moe

    c = s["case"]
    if c["op"] == "route":
        return moe.moe_route_backward(s["logits"], s["idx"], s["dw"], slot_row=s["slots"], prob_grad=s["prob_grad"],
                                      z_coef=s["z_coef"], flags=moe.MOE_ROUTE_RENORM if c["renorm"] else 0)
    if c["op"] == "bgrad":
        return moe.moe_grouped_bias_grad(s["dy"], s["offsets"], dy_src=s["src"], row_w=s["row_w"])
    if c["op"] == "few":
        epi = moe.Epilogue(act=c["act"], limit=c["limit"], bias=s["b1"])
        return moe.moe_layer_few(s["logits"], s["x"], s["w1"], s["w2"], c["k"], e0=c["e0"], w1_scales=s["s1"],
                                 w2_scales=s["s2"], shared=s["shared"], epi=epi, bias2=s["b2"], residual=s["residual"],
                                 flags=moe.MOE_ROUTE_RENORM if c["renorm"] else 0)
    if c["op"] == "act":
        epi = moe.Epilogue(act=c["act"], limit=c["limit"], bias=s["bias"])
        return moe.moe_grouped_mm_act(s["x"], s["w"], s["offsets"], epi=epi, gated=c["gated"], w_kn=c["kn"],
                                      row_src=s["src"], row_w=s["row_w"], residual=s["residual"], keep_pre=c["keep"])
    epi = moe.Epilogue(act=c["act"], limit=c["limit"])
    o = moe.moe_grouped_mm_dact(s["dy"], s["w"], s["offsets"], s["pre"], epi=epi, gated=c["gated"], w_kn=c["kn"],
                                dy_src=s["src"], row_w=s["row_w"])
    return o["dpre"], o["h"], o["dw"]


def _act(z, act):
    if act == SILU:
        return z / (1 + torch.exp(-z))
    if act == GELU:
        return 0.5 * z * torch.erfc(z * -0.5 ** 0.5)
    if act == RELU2:
        return z.clamp_min(0) ** 2
    return z


def _act_grad(z, act):
    if act == SILU:
        sig = 1 / (1 + torch.exp(-z))
        return sig + z * sig * (1 - sig)
    if act == GELU:
        return 0.5 * torch.erfc(z * -0.5 ** 0.5) + z * torch.exp(-0.5 * z * z) / (2 * math.pi) ** 0.5
    if act == RELU2:
        return 2 * z.clamp_min(0)
    return torch.ones_like(z)


def _clamp(v, limit):
    return v.clamp(-limit, limit) if limit > 0 else v


def _inside(v, limit):
    return (v.abs() <= limit).to(v.dtype) if limit > 0 else torch.ones_like(v)


def _activated(z, act, limit, gated):
    if not gated:
        return _act(_clamp(z, limit), act)
    n = z.shape[-1] // 2
    return _act(_clamp(z[..., :n], limit), act) * _clamp(z[..., n:], limit)


def _plain(s):
    c = s["case"]
    if c["op"] == "route":
        return _plain_route(s)
    if c["op"] == "few":
        return _plain_few(s)
    b = s["bounds"]
    groups = [(e, lo, hi) for e, (lo, hi) in enumerate(zip(b, b[1:])) if hi > lo]

    def rows(t, lo, hi):
        return (t[s["src"][lo:hi].long()] if s["src"] is not None else t[lo:hi]).float()

    w_of = s["row_w"]
    if c["op"] == "bgrad":
        out = torch.zeros((c["G"], c["cols"]), dtype=torch.float32, device="cuda")
        for e, lo, hi in groups:
            d = rows(s["dy"], lo, hi).double()                  # long sums
            out[e] = (d * w_of[lo:hi, None] if w_of is not None else d).sum(0)
        return out
    dt, act, lim = TYPES[c["type"]], c["act"], c["limit"]
    if c["op"] == "act":
        y = torch.empty((c["rows"], c["cols"]), dtype=dt, device="cuda")
        kept = torch.empty((c["rows"], _wide(c)), dtype=dt, device="cuda") if c["keep"] else None
        for e, lo, hi in groups:
            w = s["w"][e].float()
            z = rows(s["x"], lo, hi) @ (w if c["kn"] else w.t())
            if s["bias"] is not None:
                z = z + s["bias"][e]
            if kept is not None:
                kept[lo:hi] = z
            h = _activated(z, act, lim, c["gated"])
            if w_of is not None:
                h = h * w_of[lo:hi, None]
            if s["residual"] is not None:
                h = h + s["residual"][lo:hi].float()
            y[lo:hi] = h
        return (y, kept) if kept is not None else y
    N = c["cols"]
    dpre, h, dw = torch.empty_like(s["pre"]), torch.empty((c["rows"], N), dtype=dt, device="cuda"), \
        torch.empty(c["rows"], dtype=torch.float32, device="cuda")
    for e, lo, hi in groups:
        w = s["w"][e].float()
        dh = rows(s["dy"], lo, hi) @ (w if c["kn"] else w.t())
        z = s["pre"][lo:hi].float()
        g, u = (z[:, :N], z[:, N:]) if c["gated"] else (z, torch.ones_like(z))
        gc, uc = _clamp(g, lim), _clamp(u, lim) if c["gated"] else u
        a = _act(gc, act)
        wr = w_of[lo:hi, None] if w_of is not None else 1.0
        dg = dh * wr * uc * _act_grad(gc, act) * _inside(g, lim)
        dpre[lo:hi] = torch.cat([dg, dh * wr * a * _inside(u, lim)], 1) if c["gated"] else dg
        h[lo:hi] = a * uc * wr
        dw[lo:hi] = (dh * a * uc).sum(1)
    return dpre, h, dw


def _plain_route(s):
    c = s["case"]
    l = s["logits"]
    top = l.amax(1, keepdim=True)
    ex = torch.exp(l - top)
    total = ex.sum(1, keepdim=True)
    p = ex / total
    idx = s["idx"].long()
    slots = s["slots"].long()
    dw = torch.where(slots >= 0, s["dw"][slots.clamp_min(0)], 0.0)
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
        d = torch.zeros_like(l).scatter_(1, idx, w * (dw - (dw * w).sum(1, keepdim=True)))
    else:
        d = torch.zeros_like(l).scatter_(1, idx, dw)
        d = p * (d - (dw * w).sum(1, keepdim=True))
    if s["prob_grad"] is not None:
        d = d + p * (s["prob_grad"] - (p * s["prob_grad"]).sum(1, keepdim=True))
    if s["z_coef"]:
        d = d + 2 * s["z_coef"] * (top + torch.log(total)) * p
    return d


def _decoded(q, sc, dtype):
    N, K = q.shape
    wide = sc.to(dtype).repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return q.view(torch.float8_e4m3fn).to(dtype) * wide


def _plain_few(s):
    c = s["case"]
    T, E, G = c["T"], c["E"], c["E_loc"]
    value, order = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    ex = torch.exp(value - value[:, :1])
    w = ex[:, :c["k"]] / (ex[:, :c["k"]] if c["renorm"] else ex).sum(1, keepdim=True)
    coef = torch.zeros((T, E), dtype=torch.float32, device="cuda").scatter_(1, order[:, :c["k"]], w)
    x = s["x"].float()
    out = torch.zeros_like(x)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    for g in range(G + int(c["shared"])):
        w1, s1, w2, s2 = (s["w1"], s["s1"], s["w2"], s["s2"]) if g < G else s["shared"]
        i = g if g < G else 0
        a = _decoded(w1[i], s1[i], torch.float32) if c["eight"] else w1[i].float()
        b = _decoded(w2[i], s2[i], torch.float32) if c["eight"] else w2[i].float()
        z = x @ a.t()
        if s["b1"] is not None:
            z = z + s["b1"][g]
        y = _activated(z, c["act"], c["limit"], True) @ b.t()
        if s["b2"] is not None:
            y = y + s["b2"][g]
        out = out + (y * coef[:, c["e0"] + g, None] if g < G else y)
    return out.to(s["x"].dtype)


# -------------------------------------------------- the definition in 64 bits
def _act64(z, act):
    if act == NONE:
        return z
    if act == RELU2:
        return torch.relu(z).square()
    if act == GELU:
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(z)


def _slope64(z, act):
    """The derivative by automatic differentiation of the definition."""
    z = z.detach().requires_grad_(True)
    with torch.enable_grad():
        return torch.autograd.grad(_act64(z, act).sum(), z)[0]


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "route":
        l = s["logits"].double()
        p = torch.softmax(l, 1)
        hit = torch.zeros_like(p)
        up = torch.zeros_like(p)
        rows = torch.arange(c["T"], device="cuda")
        for j in range(c["k"]):
            e, r = s["idx"][:, j].long(), s["slots"][:, j].long()
            hit[rows, e] = 1.0
            up[rows, e] = torch.where(r >= 0, s["dw"].double()[r.clamp_min(0)], 0.0)
        q = p * hit / (p * hit).sum(1, keepdim=True) if c["renorm"] else p
        d = q * (up - (up * q).sum(1, keepdim=True))
        if s["prob_grad"] is not None:
            pg = s["prob_grad"].double()
            d += p * (pg - (p @ pg)[:, None])
        return d + 2 * s["z_coef"] * torch.logsumexp(l, 1, keepdim=True) * p
    if c["op"] == "few":
        return _exact_few(s)
    b, R, N = s["bounds"], c["rows"], c["cols"]
    src = s["src"].long() if s["src"] is not None else torch.arange(R, device="cuda")
    wr = s["row_w"].double() if s["row_w"] is not None else torch.ones(R, dtype=torch.float64, device="cuda")
    if c["op"] == "bgrad":
        return torch.stack([wr[lo:hi] @ s["dy"][src[lo:hi]].double() for lo, hi in zip(b, b[1:])])
    act, lim = c["act"], c["limit"]
    lin, lout = s["x"] if c["op"] == "act" else s["dy"], []
    for e, (lo, hi) in enumerate(zip(b, b[1:])):
        w = s["w"][e].double()
        lout.append(lin[src[lo:hi]].double() @ (w if c["kn"] else w.t()))
        if c["op"] == "act" and s["bias"] is not None:
            lout[-1] += s["bias"][e].double()
    z = torch.cat(lout)
    cut = lim if lim > 0 else math.inf
    if c["op"] == "act":
        h = _act64(z[:, :N].clamp(-cut, cut), act)
        if c["gated"]:
            h = h * z[:, N:].clamp(-cut, cut)
        y = h * wr[:, None] + (s["residual"].double() if s["residual"] is not None else 0.0)
        return (y, z) if c["keep"] else y
    pre = s["pre"].double()
    g = pre[:, :N]
    a, slope = _act64(g.clamp(-cut, cut), act), _slope64(g.clamp(-cut, cut), act) * (g.abs() <= cut)
    if not c["gated"]:
        return z * wr[:, None] * slope, a * wr[:, None], (z * a).sum(1)
    u = pre[:, N:]
    uc = u.clamp(-cut, cut)
    d = torch.cat([z * uc * slope, z * a * (u.abs() <= cut)], 1) * wr[:, None]
    return d, a * uc * wr[:, None], (z * a * uc).sum(1)


def _exact_few(s):
    c = s["case"]
    T, k, I, G = c["T"], c["k"], c["I"], c["E_loc"]
    l = s["logits"].double()
    rank = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, :k].cpu().tolist()
    p = torch.softmax(l, 1)
    cut = c["limit"] if c["limit"] > 0 else math.inf
    out = s["residual"].double() if s["residual"] is not None else torch.zeros((T, c["H"]), dtype=torch.float64, device="cuda")
    users = {}
    for t in range(T):
        for e in rank[t]:
            if c["e0"] <= e < c["e0"] + G:
                w = p[t, e] / p[t, rank[t]].sum() if c["renorm"] else p[t, e]
                users.setdefault(e - c["e0"], []).append((t, w))
    if c["shared"]:
        users[G] = [(t, torch.ones((), dtype=torch.float64, device="cuda")) for t in range(T)]
    for g, who in users.items():
        w1, s1, w2, s2 = (s["w1"], s["s1"], s["w2"], s["s2"]) if g < G else s["shared"]
        i = g if g < G else 0
        a = _decoded(w1[i], s1[i], torch.float64) if c["eight"] else w1[i].double()
        b = _decoded(w2[i], s2[i], torch.float64) if c["eight"] else w2[i].double()
        t = torch.tensor([t for t, _ in who], device="cuda")
        z = s["x"][t].double() @ a.t()
        if s["b1"] is not None:
            z = z + s["b1"][g].double()
        y = (_act64(z[:, :I].clamp(-cut, cut), c["act"]) * z[:, I:].clamp(-cut, cut)) @ b.t()
        if s["b2"] is not None:
            y = y + s["b2"][g].double()
        out = out.index_add(0, t, y * torch.stack([w for _, w in who])[:, None])
    return out
