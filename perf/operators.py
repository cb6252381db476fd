"""Measured cases of the 16-bit and block-scaled FP8 operators of the routed layer.

Each case is one call of a user's program on tensors that the program already
holds: token rows, expert weights, the group offsets on the device, and (for
the plain forms) the largest group's row count. `own` selects the side: the
library's calls, or the plain form in elementary torch operations.

  mm     grouped product, y[r] = x[src[r]] . W_g^T (W [G, N, K]) or x . W_g (W [G, K, N])
  wgrad  weight gradient of a grouped product, dW_g = sum over the group's rows dy^T x
  fp8    block-128 FP8 product: the rows are quantised in the call, the weights were before
  glu    the gated activation that keeps its input in 8 bits, and its backward pass
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token on two experts of a small model: latency
        dict(name="mm-one-token", op="mm", type="bf16", rows=2, tokens=1, G=8, N=512, K=512, kn=False, skew=0.0),
        # a decode batch on one GPU's experts: weights read once, some experts idle
        dict(name="mm-decode", op="mm", type="bf16", rows=16, tokens=16, G=8, N=4096, K=7168, kn=False, skew=0.0),
        # training forward over one GPU's experts: skewed popularity, rows gathered from token order
        dict(name="mm-forward", op="mm", type="bf16", rows=24576, tokens=16384, G=16, N=2816, K=2048, kn=False,
             skew=1.1),
        # gradient of the rows: the same weights, read along their other axis
        dict(name="mm-backward", op="mm", type="fp16", rows=8192, tokens=0, G=8, N=7168, K=4096, kn=True, skew=0.5),
        # weight gradient in 32 bits, rows gathered from token order
        dict(name="wgrad-forward-rows", op="wgrad", type="bf16", rows=16384, tokens=16384, G=8, N=2816, K=2048,
             eight=False, out="fp32", skew=1.1),
        # weight gradient from rows that were kept in 8 bits; odd sizes
        dict(name="wgrad-8bit-rows", op="wgrad", type="bf16", rows=5001, tokens=4099, G=12, N=1416, K=2040,
             eight=True, out="fp32", skew=0.5),
        # block-scaled FP8 decode batch
        dict(name="fp8-decode", op="fp8", type="bf16", rows=16, tokens=16, G=8, N=4096, K=7168, skew=0.0),
        # block-scaled FP8 prefill over one GPU's experts
        dict(name="fp8-prefill", op="fp8", type="bf16", rows=16384, tokens=8192, G=16, N=2816, K=2048, skew=1.1),
        # an always-on (shared) expert: one dense product, no gather
        dict(name="fp8-shared", op="fp8", type="bf16", rows=8192, tokens=0, G=1, N=4096, K=7168, skew=0.0),
        # the activation of a decode batch
        dict(name="glu-decode", op="glu", type="bf16", rows=24, I=2048, back=False),
        # the activation of a training batch, its input kept in 8 bits
        dict(name="glu-forward", op="glu", type="bf16", rows=49152, I=1408, back=False),
        # its backward pass from those 8 bits
        dict(name="glu-backward", op="glu", type="fp16", rows=24576, I=2048, back=True),
    ]


def _log(rng, lo, hi, step):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v / step + 0.5) * step)


def draw(rng):
    while True:
        op = rng.choice(["mm", "wgrad", "fp8", "glu"])
        t = rng.choice(["bf16", "fp16"])
        rows = _log(rng, 1, 49152 if op == "glu" else 24576, 1)
        if op == "glu":
            c = dict(op=op, type=t, rows=rows, I=_log(rng, 128, 4096, 8), back=rng.random() < 0.5)
        else:
            c = dict(op=op, type=t, rows=rows, tokens=rng.choice([0, _log(rng, 1, 16384, 1)]), G=_log(rng, 1, 64, 1),
                     N=_log(rng, 256, 7168, 8), K=_log(rng, 256, 7168, 16 if op == "fp8" else 8),
                     skew=rng.choice([0.0, 0.5, 1.1]))
            if op == "mm":
                c["kn"] = rng.random() < 0.5
            elif op == "wgrad":
                c["eight"] = rng.random() < 0.4
                c["out"] = rng.choice(["fp32", "same"])
                if c["eight"]:
                    c["type"] = "bf16"
        w = work(c)
        weights = c.get("G", 0) * c.get("N", 0) * c.get("K", 0)
        if w["flops"] <= 4.8e11 and w["bytes"] <= 6.5e8 and weights <= 2.4e8:
            return c


def work(case):
    R = case["rows"]
    if case["op"] == "glu":
        I, nb = case["I"], -(-case["I"] // BLOCK)
        kept = 2 * R * (I + 4 * nb)                             # codes and scales
        if case["back"]:                                        # dh in, dpre and h out, row weights and their gradient
            return {"bytes": kept + R * I * (2 + 4 + 2) + 8 * R, "flops": 16 * R * I}
        return {"bytes": kept + R * I * (4 + 2) + 4 * R, "flops": 8 * R * I}
    G, N, K = case["G"], case["N"], case["K"]
    busy = min(G, R)                                            # groups whose weights a pass can need
    src = min(case["tokens"] or R, R)
    fl = 2 * R * N * K
    if case["op"] == "mm":
        return {"bytes": 2 * src * K + 2 * busy * N * K + 2 * R * N, "flops": fl}
    if case["op"] == "wgrad":
        x = src * (K + 4 * -(-K // BLOCK)) if case["eight"] else 2 * src * K
        return {"bytes": x + 2 * R * N + G * N * K * (4 if case["out"] == "fp32" else 2), "flops": fl}
    blocks = -(-N // BLOCK) * -(-K // BLOCK)
    return {"bytes": 2 * src * K + busy * (N * K + 4 * blocks) + 2 * R * N, "flops": fl}


# -------------------------------------------------------------------- inputs
def _pow2_blocks(v):
    """FP8 codes (as values) and power-of-two scales of the rows of v, per block of 128 along the last axis."""
    n, k = v.shape
    nb = -(-k // BLOCK)
    f = torch.zeros((n, nb * BLOCK), dtype=torch.float32, device=v.device)
    f[:, :k] = v
    f = f.view(n, nb, BLOCK)
    top = f.abs().amax(-1)
    m, e = torch.frexp(top)                                     # top = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 127)
    s = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.ones_like(top))
    q = (f / s[..., None]).to(torch.float8_e4m3fn)
    return q.view(n, nb * BLOCK)[:, :k].contiguous(), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["type"]]
    R = case["rows"]

    def normal(shape, std, dtype=dt):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        flat = out.view(-1)
        step = 1 << 26
        for i in range(0, flat.numel(), step):                  # in pieces: no 32-bit copy of the whole
            n = min(step, flat.numel() - i)
            flat[i:i + n] = torch.randn(n, generator=g, device="cuda") * std
        return out

    s = dict(case=case)
    if case["op"] == "glu":
        I = case["I"]
        pre = normal((R, 2 * I), 1.5)
        s["row_w"] = torch.rand(R, generator=g, device="cuda") * 0.9 + 0.05
        if case["back"]:
            q, sc = _pow2_blocks(pre.view(2 * R, I))
            s["codes"] = q.view(R, 2 * I).view(torch.uint8)
            s["scales"] = sc.view(R, 2, -1)
            s["dh"] = normal((R, I), 0.1)
        else:
            s["pre"] = pre
        return s

    G, N, K, T = case["G"], case["N"], case["K"], case["tokens"]
    p = torch.arange(1, G + 1, device="cuda", dtype=torch.float32) ** -case["skew"]
    p = p[torch.randperm(G, generator=g, device="cuda")]
    counts = torch.bincount(torch.multinomial(p, R, replacement=True, generator=g), minlength=G)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["most"] = int(counts.max())                               # for the plain form: rows of the largest group
    s["src"] = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32) if T else None
    rows = T or R
    if case["op"] == "wgrad":
        s["dy"] = normal((R, N), 0.1)
        x = normal((rows, K), 1.0)
        if case["eight"]:
            q, s["xs"] = _pow2_blocks(x)
            s["x"] = q.view(torch.uint8)
        else:
            s["x"], s["xs"] = x, None
        return s
    s["x"] = normal((rows, K), 1.0)
    if case["op"] == "mm":
        s["w"] = normal((G, K, N) if case["kn"] else (G, N, K), 0.02)
        return s
    # weights quantised once, per 128 x 128 block, with any 32-bit scale
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    s["ws"] = (torch.rand((G, nb, kb), generator=g, device="cuda") * 0.8 + 0.6) * (0.08 / E4M3_MAX)
    s["wq"] = torch.empty((G, N, K), dtype=torch.uint8, device="cuda")
    for e in range(G):
        q = torch.randn((N, K), generator=g, device="cuda") * (E4M3_MAX / 4)
        s["wq"][e] = q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return s


# ------------------------------------------------------------------- one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import routed_grouped_gemm_amd as moe

    c = s["case"]
    if c["op"] == "mm":
        return moe.moe_grouped_mm(s["x"], s["w"], s["offsets"], w_kn=c["kn"], row_src=s["src"])
    if c["op"] == "wgrad":
        return moe.moe_grouped_wgrad(s["dy"], s["x"], s["offsets"], x_src=s["src"], x_scales=s["xs"],
                                     out_dtype=torch.float32 if c["out"] == "fp32" else TYPES[c["type"]])
    if c["op"] == "fp8":
        xq, xs = moe.moe_quantize_block(s["x"])
        return moe.moe_grouped_mm_fp8(xq, xs, s["wq"], s["ws"], s["offsets"], row_src=s["src"],
                                      out_dtype=TYPES[c["type"]])
    if c["back"]:
        o = moe.moe_glu_checkpoint_backward(s["codes"], s["scales"], s["dh"], row_w=s["row_w"])
        return o["dpre"], o["h"], o["dw"]
    h, codes, scales = moe.moe_glu_checkpoint(s["pre"], row_w=s["row_w"])
    return h, codes.view(torch.float8_e4m3fn), scales


def _groups(offsets, most, n_rows):
    """Padded places: the row of place (g, i), whether it is one, and each row's own place."""
    at = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    real = at < offsets[1:, None]
    r = torch.arange(n_rows, device=offsets.device)
    grp = torch.searchsorted(offsets[1:].long(), r, right=True)
    return torch.where(real, at, 0), real, grp, r - offsets[:-1].long()[grp]


def _decoded(codes, scales):
    n, k = codes.shape
    v = codes.view(torch.float8_e4m3fn).float()
    return v * scales.repeat_interleave(BLOCK, -1)[:, :k]


def _plain(s):
    c = s["case"]
    if c["op"] == "glu":
        return _plain_glu_back(s) if c["back"] else _plain_glu(s)
    at, real, grp, place = _groups(s["offsets"], s["most"], c["rows"])
    from_row = s["src"].long()[at] if s["src"] is not None else at
    if c["op"] == "wgrad":
        dy = s["dy"].float()[at] * real[..., None]
        x = (s["x"].float() if s["xs"] is None else _decoded(s["x"], s["xs"]))[from_row] * real[..., None]
        dw = torch.bmm(dy.transpose(1, 2).contiguous(), x)
        return dw if c["out"] == "fp32" else dw.to(TYPES[c["type"]])
    if c["op"] == "mm":
        x, w = s["x"].float(), s["w"].float()
        w = w if c["kn"] else w.transpose(1, 2).contiguous()
    else:
        q, sc = _pow2_blocks(s["x"].float())
        x = _decoded(q.view(torch.uint8), sc)
        G, N, K = s["wq"].shape
        sw = s["ws"].repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
        w = (s["wq"].view(torch.float8_e4m3fn).float() * sw).transpose(1, 2).contiguous()
    y = torch.bmm(x[from_row] * real[..., None], w)
    return y[grp, place].to(TYPES[c["type"]])


def _plain_glu(s):
    pre = s["pre"]
    R, I = pre.shape[0], pre.shape[1] // 2
    g, u = pre[:, :I].float(), pre[:, I:].float()
    h = g / (1 + torch.exp(-g)) * u * s["row_w"][:, None]
    q, sc = _pow2_blocks(pre.float().view(2 * R, I))
    return h.to(pre.dtype), q.view(R, 2 * I), sc.view(R, 2, -1)


def _plain_glu_back(s):
    R, I = s["dh"].shape
    pre = _decoded(s["codes"].view(2 * R, I), s["scales"].view(2 * R, -1)).view(R, 2 * I)
    g, u = pre[:, :I], pre[:, I:]
    dh, w = s["dh"].float(), s["row_w"][:, None]
    sig = 1 / (1 + torch.exp(-g))
    a = g * sig
    dg = dh * w * u * (sig + a * (1 - sig))
    du = dh * w * a
    dt = s["dh"].dtype
    return torch.cat([dg, du], 1).to(dt), (a * u * w).to(dt), (dh * a * u).sum(1)


# -------------------------------------------------- the definition in 64 bits
def _e4m3_64(v):
    """Nearest E4M3 value (ties to even) of 64-bit numbers within +-448."""
    a = v.abs()
    quantum = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / quantum) * quantum


def _blocks_64(v):
    """Block values on the E4M3 grid and scales: the smallest power of two that brings a block within +-448."""
    n, k = v.shape
    codes, scales = [], []
    for b in range(0, k, BLOCK):
        piece = v[:, b:b + BLOCK]
        top = piece.abs().amax(1)
        e = torch.ceil(torch.log2((top / E4M3_MAX).clamp_min(2.0 ** -126)))
        sc = torch.where(top > 0, torch.exp2(e), torch.ones_like(top))
        codes.append(_e4m3_64(piece / sc[:, None]))
        scales.append(sc)
    return torch.cat(codes, 1), torch.stack(scales, 1)


def _from_blocks_64(codes, scales):
    out = codes.double()
    for b in range(scales.shape[1]):
        out[:, b * BLOCK:(b + 1) * BLOCK] *= scales[:, b:b + 1].double()
    return out


def _silu_64(z):
    return z * torch.sigmoid(z)


def exact(case, seed):
    s = prepare(case, seed)
    R = case["rows"]
    if case["op"] == "glu":
        I = case["I"]
        w = s["row_w"].double()[:, None]
        if not case["back"]:
            pre = s["pre"].double()
            q, sc = _blocks_64(pre.view(2 * R, I))
            return _silu_64(pre[:, :I]) * pre[:, I:] * w, q.view(R, 2 * I), sc.view(R, 2, -1)
        c8 = s["codes"].view(torch.float8_e4m3fn).view(2 * R, I)
        pre = _from_blocks_64(c8, s["scales"].view(2 * R, -1)).view(R, 2 * I)
        g, u, dh = pre[:, :I], pre[:, I:], s["dh"].double()
        sg = torch.sigmoid(g)
        a = _silu_64(g)
        dg = dh * w * u * sg * (1 + g * (1 - sg))
        return torch.cat([dg, dh * w * a], 1), a * u * w, (dh * a * u).sum(1)

    off = s["offsets"].tolist()
    src = s["src"].long() if s["src"] is not None else torch.arange(R, device="cuda")
    outs = []
    if case["op"] == "wgrad":
        x = s["x"].double() if s["xs"] is None else _from_blocks_64(s["x"].view(torch.float8_e4m3fn), s["xs"])
        for lo, hi in zip(off, off[1:]):
            outs.append(s["dy"][lo:hi].double().t() @ x[src[lo:hi]])
        return torch.stack(outs)
    x = s["x"].double()
    if case["op"] == "fp8":
        x = _from_blocks_64(*_blocks_64(x))
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if case["op"] == "fp8":
            we = s["wq"][e].view(torch.float8_e4m3fn).double()
            for n in range(s["ws"].shape[1]):
                we[n * BLOCK:(n + 1) * BLOCK] = _from_blocks_64(
                    we[n * BLOCK:(n + 1) * BLOCK], s["ws"][e, n:n + 1].expand(we[n * BLOCK:(n + 1) * BLOCK].shape[0], -1))
            we = we.t()
        else:
            we = s["w"][e].double() if case["kn"] else s["w"][e].double().t()
        outs.append(x[src[lo:hi]] @ we)
    return torch.cat(outs)
