"""The layer for a few tokens where a token's mask leaves no expert at all."""
import pytest
import torch

from gpu_util import banner
from test_gpu_few_layer import Case
from test_gpu_few_layer_parts import reference

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")
INF = float("inf")


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (6, 64, 6), (16, 40, 3), (32, 200, 7), (9, 300, 4), (32, 1000, 20)])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_token_without_an_expert(T, E, k, renorm, shared):
    """Logits of -inf only: the residual and the shared expert, whatever the other tokens choose."""
    banner(f"few layer, masked tokens {T} {E} {k} {renorm} {shared}")
    c = Case(T=T, E=E, k=k, e0=1, E_loc=min(E - 1, 30), H=64, I=32, residual=True, bias=True, shared=shared, renorm=renorm,
             seed=T + E)
    masked = [t for t in (0, 5, T - 1) if t < T]
    c.logits[masked] = -1e30                                 # the same by weights of 0: expert 0 is not here
    c.logits[masked, 0] = 0.0
    ref, tol = reference(c)
    c.logits[masked] = -INF
    got = c.run()
    assert bool(((got.double() - ref).abs() <= tol).all())
    if not shared:
        assert torch.equal(got[masked], c.res[masked])
    out = torch.full_like(c.x, 7.0)
    c.run(residual=None, out=out)
    assert shared or bool((out[masked] == 0).all())


@pytest.mark.parametrize("E", [8, 300])
def test_no_token_has_an_expert(E):
    c = Case(T=5, E=E, k=2, e0=0, E_loc=8, H=64, I=32, residual=True, seed=E)
    c.logits.fill_(-INF)
    assert torch.equal(c.run(), c.res)


@pytest.mark.parametrize("bits", [0x7FC00000, 0xFFC00000 - (1 << 32), -1, 0x7F800000])
@pytest.mark.parametrize("E", [8, 300])
def test_one_nan_or_infinity_among_masked_logits(bits, E):
    """A NaN or +inf beside -inf everywhere else: still NaN, in that token only."""
    c = Case(T=4, E=E, k=2, e0=0, E_loc=8, H=64, I=32, seed=E)
    c.logits[:, 8:] = -INF
    c.logits[2] = -INF
    c.logits.view(torch.int32)[2, 3] = bits
    got = c.run()
    assert bool(got[2].isnan().all()) and bool(got[[0, 1, 3]].isfinite().all())
