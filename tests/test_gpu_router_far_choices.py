"""The router's gradient where the choices are far below the row's largest logit:
renormalised weights are relative to the choices alone."""
import pytest
import torch

from gpu_util import banner
from test_gpu_router_bias_grad import check_route, gen

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")


@pytest.mark.parametrize("T,E,k", [(9, 8, 2), (40, 64, 6), (5, 100, 17), (12, 250, 8), (6, 1000, 32)])
@pytest.mark.parametrize("top", [20.0, 88.0, 100.0, 110.0, 600.0])
def test_largest_logit_not_chosen(T, E, k, top):
    banner(f"route backward, choices far below {T} {E} {k} {top}")
    g = gen(int(top) + E)
    l = torch.randn((T, E), generator=g, device="cuda") * 3
    idx = torch.rand((T, E - 1), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    l[:, E - 1] = top
    D = torch.randn((T, k), generator=g, device="cuda")
    for aux in (False, True):
        c = torch.randn(E, generator=g, device="cuda") if aux else None
        got = moe.moe_route_backward(l, idx, D, prob_grad=c, z_coef=0.25 if aux else 0.0, flags=moe.MOE_ROUTE_RENORM)
        check_route(l, idx, D.double(), got, True, c.double() if aux else None, 0.25 if aux else 0.0)


def test_two_choices_of_three():
    l = torch.tensor([[110.0, 0.0, 1.0]], device="cuda")
    idx = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda")
    D = torch.tensor([[1.0, 0.0]], device="cuda")
    got = moe.moe_route_backward(l, idx, D, flags=moe.MOE_ROUTE_RENORM)[0].double()
    w = torch.softmax(torch.tensor([0.0, 1.0], dtype=torch.float64), 0)
    want = torch.tensor([0.0, float(w[0] * w[1]), -float(w[0] * w[1])], dtype=torch.float64, device="cuda")
    assert bool(((got - want).abs() <= 2 ** -20).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_and_infinity_beside_the_choices(value):
    """A NaN or +inf that is not chosen makes the chosen experts' gradients NaN all the same."""
    l = torch.zeros((2, 8), device="cuda")
    l[0, 7] = value
    idx = torch.tensor([[1, 2], [1, 2]], dtype=torch.int32, device="cuda")
    got = moe.moe_route_backward(l, idx, torch.ones((2, 2), device="cuda"), flags=moe.MOE_ROUTE_RENORM)
    assert bool(got[0, 1:3].isnan().all()) and bool(got[1].isfinite().all())
