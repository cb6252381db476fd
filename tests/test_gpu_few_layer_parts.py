"""The layer for a few tokens rounds its outputs only: between its two products h is held
in two parts of the operands' type. Every way that the second product can take:
groups of up to 8, 16 and 32 rows, h in LDS whole, in half or not at all."""
import pytest
import torch

from gpu_util import banner
from test_gpu_few_layer import Case, decoded

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")


def reference(c):
    """(out, bound) in 64 bits. u: half a step of the type. h is off by u^2 of itself (two
    parts; in FP16 at least 2^-36, half a step of the scaled second part below its
    smallest normal number), otherwise as in the bound of Case.reference: 2^-18 of the
    |terms| of each product (fewer than 64 roundings of 2^-24 follow one another;
    adding the parts is one of them for each unit), an activation whose slope is
    below 1.2, and one rounding at the end."""
    u = torch.finfo(c.dt).eps / 2
    order = torch.sort(c.logits, dim=1, descending=True, stable=True)[1][:, :c.k]
    p = torch.softmax(c.logits.double(), 1).gather(1, order)
    if c.flags:
        p = p / p.sum(1, keepdim=True)
    x = c.x.double()
    out = c.res.double().clone() if c.res is not None else torch.zeros_like(x)
    tol = out.abs() * 2 ** -22
    n = c.w1.shape[0]
    for g in range(n + (c.shared is not None)):
        w1, s1, w2, s2 = (c.w1[g:g + 1], c.s1, c.w2[g:g + 1], c.s2) if g < n else c.shared
        if s1 is not None:
            a, b = decoded(w1, s1[g:g + 1] if g < n else s1)[0], decoded(w2, s2[g:g + 1] if g < n else s2)[0]
        else:
            a, b = w1[0].double(), w2[0].double()
        if g < n:
            t, j = (order == g + c.e0).nonzero(as_tuple=True)
            w = p[t, j][:, None]
        else:
            t, w = torch.arange(c.T, device="cuda"), 1.0
        if t.numel() == 0:
            continue
        z, dz = x[t] @ a.t(), 2 ** -18 * (x[t].abs() @ a.abs().t())
        if c.b1 is not None:
            z = z + c.b1[g].double()
            dz = dz + 2 ** -18 * c.b1[g].double().abs()
        gz, uz, dg, du = z[:, :c.I], z[:, c.I:], dz[:, :c.I], dz[:, c.I:]
        act = c.act64(gz)
        h = act * uz * w
        dh = w * (1.2 * dg * (uz.abs() + du) + act.abs() * du) + h.abs() * (u * u + 2 ** -19)
        if c.dt == torch.float16:
            dh = dh + 2 ** -36
        y, dy = h @ b.t(), dh @ b.abs().t() + 2 ** -18 * (h.abs() @ b.abs().t())
        if c.b2 is not None:
            y = y + w * c.b2[g].double()
            dy = dy + 2 ** -18 * w * c.b2[g].double().abs()
        out.index_add_(0, t, y)
        tol.index_add_(0, t, dy)
    return out, tol + u * (out.abs() + tol) + torch.finfo(c.dt).tiny * u


def check(c):
    ref, tol = reference(c)
    got = c.run()
    bad = (got.double() - ref).abs() / tol
    print(f"  largest error / bound {float(bad.max()):.3f}", flush=True)
    assert bool((bad <= 1).all())


# tokens, experts, choices, inner size: up to 8 rows a group with tokens as columns, then
# with rows as columns; more than 8 with tokens, then rows as columns (more than
# 16 too); each with h small, and larger than half or all of a compute unit's LDS
FORMS = [(8, 8, 4, 64), (8, 8, 4, 2560), (3, 8, 2, 2064), (16, 64, 4, 64), (16, 64, 4, 1296), (9, 16, 2, 96),
         (16, 2, 2, 64), (16, 2, 2, 1040), (16, 2, 2, 2560), (20, 128, 2, 64), (20, 128, 2, 528), (32, 96, 3, 272),
         (32, 2, 1, 64), (32, 2, 1, 1040), (32, 2, 1, 2560), (25, 3, 3, 144), (17, 1, 1, 32)]


@pytest.mark.parametrize("T,E,k,I", FORMS)
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_outputs_are_rounded_once(T, E, k, I, eight, dtype):
    banner(f"few layer, h in two parts {T} {E} {k} {I} {eight} {dtype}")
    check(Case(T=T, E=E, k=k, e0=0, E_loc=E, H=272, I=I, dtype=dtype, eight=eight, seed=T + I + k))


@pytest.mark.parametrize("T,E,k,I", [(8, 8, 3, 40), (14, 40, 3, 72), (32, 64, 2, 40), (16, 4, 3, 1032), (32, 8, 6, 136)])
@pytest.mark.parametrize("eight", [False, True])
def test_with_everything(T, E, k, I, eight):
    """Biases, residual, a shared expert (every token's, so more than 8 or 16 rows), part of the experts."""
    I = -(-I // 16) * 16
    banner(f"few layer with everything {T} {E} {k} {I} {eight}")
    check(Case(T=T, E=E, k=k, e0=1, E_loc=E - 2, H=144, I=I, eight=eight, shared=True, bias=True, residual=True,
               renorm=True, seed=T * k))


@pytest.mark.parametrize("T", [5, 14, 30])
def test_infinite_weights_and_values_past_fp16(T):
    """An infinite weight of W2 gives an infinity where h is exact in one part too, and h past
    FP16's range an infinity, no NaN."""
    one = torch.zeros((T, 1), device="cuda")
    w1 = torch.zeros((1, 2 * 8, 16), dtype=torch.float16, device="cuda")
    w1[0, 0, 0] = w1[0, 8, 0] = 1.0
    w2 = torch.zeros((1, 8, 8), dtype=torch.float16, device="cuda")
    w2 = torch.cat([w2, w2], 1)
    w2[0, 1, 0], w2[0, 2, 0], w2[0, 3, 0] = 1.0, float("inf"), -float("inf")
    x = torch.zeros((T, 16), dtype=torch.float16, device="cuda")
    x[:, 0] = 2.0                                            # h = 4
    x[1, 0] = 300.0                                          # h = 90000
    x[2, 0] = 1.0009765625                                   # h = 1.001953... of two parts
    got = moe.moe_layer_few(one, x, w1, w2, 1, epi=moe.Epilogue(act=moe.MOE_ACT_NONE))
    inf = float("inf")
    assert bool((got[:, 2] == inf).all()) and bool((got[:, 3] == -inf).all())
    assert bool(got[:, 0].isnan()[1]) and float(got[1, 1]) == inf        # (an infinity times the weights 0 is none)
    rest = [t for t in range(T) if t != 1]
    assert bool((got[rest, 0] == 0).all()) and float(got[0, 1]) == 4.0
    assert float(got[2, 1]) == float((x[2, 0].double() ** 2).to(torch.float16))
