"""E4M3 weights whose scales are infinite or NaN: they reach what they scale, as the formula has it."""
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")
INF = float("inf")


@pytest.mark.parametrize("T", [1, 12, 30])
@pytest.mark.parametrize("H", [144, 272, 3088, 7184])
@pytest.mark.parametrize("block", [0, -1])
@pytest.mark.parametrize("product", [1, 2])
def test_infinite_scale(T, H, block, product):
    """Positive values throughout, so an infinite scale makes its sums +infinity: also the last
    block's, behind which a row has units that are not there."""
    banner(f"few layer, infinite scale {T} {H} {block} {product}")
    I = 144
    one = lambda n, k: torch.full((1, n, k), 0x38, dtype=torch.uint8, device="cuda")  # noqa: E731 (ones)
    sc = lambda n, k: torch.full((1, -(-n // 128), -(-k // 128)), 2.0 ** -6, device="cuda")  # noqa: E731
    w1, w2, s1, s2 = one(2 * I, H), one(H, I), sc(2 * I, H), sc(H, I)
    x = torch.full((T, H), 0.125, dtype=torch.bfloat16, device="cuda")
    run = lambda: moe.moe_layer_few(torch.zeros((T, 1), device="cuda"), x, w1, w2, 1, w1_scales=s1, w2_scales=s2,  # noqa: E731
                                    epi=moe.Epilogue(act=moe.MOE_ACT_NONE))
    assert bool(run().isfinite().all())
    if product == 1:
        s1[0, 0, block] = INF                                # gate rows 0 .. 127
        assert bool((run() == INF).all())
    else:
        s2[0, 0, block] = INF                                # outputs 0 .. 127
        got = run()
        assert bool((got[:, :128] == INF).all()) and bool(got[:, 128:].isfinite().all())
