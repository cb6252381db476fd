"""The products with an epilogue by their own plans: every tile height for several
groups, and for one group the launches of its last rows and columns in both heights,
split or not, beside main launches of 128 and 256 rows."""
import pytest
import torch

from gpu_util import banner
from test_gpu_mm_act import GELU, SWI, forward, gradient

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")

# rows, outputs, K, gated, plan: rows and parts of the main launch, of the last rows', of the last columns'
ONE = [(3597, 2056, 2040, False, [128, 1, 32, 4, 0, 0]), (3597, 1032, 2040, True, [128, 1, 32, 4, 0, 0]),
       (6681, 1032, 2040, False, [128, 1, 0, 0, 32, 2]), (6681, 520, 2040, True, [128, 1, 0, 0, 32, 2]),
       (20000, 4160, 136, False, [256, 1, 0, 0, 64, 1]), (14648, 1088, 136, True, [256, 1, 0, 0, 64, 1]),
       (770, 8200, 136, True, [256, 1, 64, 1, 0, 0]), (1027, 8200, 2040, True, [256, 1, 64, 1, 32, 4]),
       (16447, 1088, 2040, True, [256, 1, 32, 4, 64, 1]), (9251, 8256, 136, True, [256, 1, 64, 1, 64, 1])]
GROUPS = [(200, 40, 264, 136, [32, 1]), (400, 3, 264, 2040, [32, 4]), (2000, 3, 520, 136, [64, 1]), (6000, 3, 1032, 264, [128, 1]),
          (3000, 40, 1288, 72, [256, 1]), (20000, 6, 520, 136, [256, 1])]


@pytest.mark.parametrize("R,N,K,gated,plan", ONE)
def test_forward_of_one_group(R, N, K, gated, plan):
    banner(f"act plan {plan} R={R} N={N} K={K} gated={gated}")
    assert moe.moe_grouped_mm_act_plan(R, 1, 2 * N if gated else N, K, gated) == plan
    forward(R, 1, N, K, torch.bfloat16, gated, SWI, weighted=True, seed=R)
    forward(R, 1, N, K, torch.float16, gated, GELU, kn=not gated, T=300, seed=R + 1, hi=R - 130)


@pytest.mark.parametrize("R,N,K,plan", [(c[0], c[1], c[2], c[4]) for c in ONE if not c[3]] +
                         [(770, 16400, 136, [256, 1, 64, 1, 0, 0]), (1027, 16400, 2040, [256, 1, 64, 1, 32, 4])])
@pytest.mark.parametrize("gated", [False, True])
def test_gradient_of_one_group(R, N, K, plan, gated):
    banner(f"dact plan {plan} R={R} N={N} K={K} gated={gated}")
    assert moe.moe_grouped_mm_act_plan(R, 1, N, K) == plan
    gradient(R, 1, N, K, torch.bfloat16, gated, SWI, kn=gated, weighted=True, T=300, seed=R, hi=R - 130 if gated else None)


@pytest.mark.parametrize("R,G,N,K,plan", GROUPS)
@pytest.mark.parametrize("gated", [False, True])
def test_several_groups(R, G, N, K, plan, gated):
    banner(f"act and dact plan {plan} R={R} G={G} N={N} K={K} gated={gated}")
    assert moe.moe_grouped_mm_act_plan(R, G, N, K) == plan + [0, 0, 0, 0]
    if not gated:
        forward(R, G, N, K, torch.bfloat16, False, SWI, weighted=True, seed=R)
    gradient(R, G, N, K, torch.float16, gated, GELU, kn=not gated, weighted=True, T=100, seed=R + G)
