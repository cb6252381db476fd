"""The grouped products at the far ends of what their header allows."""
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")

BF = torch.bfloat16


def test_overlapping_groups_with_more_passes_than_32_bits_hold():
    """Offsets that do not ascend: 1025 of 2049 groups are all of 2^28 rows, 2^32
    passes and more of 64 rows. Memory around the output stays as it was."""
    banner("overlapping groups of 2^28 rows")
    R, G, N, K, edge = 1 << 28, 2049, 64, 16, 256
    o = torch.zeros(G + 1, device="cuda", dtype=torch.int32)
    o[1::2] = R
    big = torch.full((R + 2 * edge, N), -7.0, dtype=BF, device="cuda")
    y = big[edge:edge + R]
    x = torch.zeros((R, K), dtype=BF, device="cuda")
    w = torch.zeros((G, N, K), dtype=BF, device="cuda")
    for kn in (False, True):
        moe.moe_grouped_mm(x, w.view(G, K, N) if kn else w, o, w_kn=kn, out=y)
        torch.cuda.synchronize()
    xq, wq = torch.zeros((R, K), dtype=torch.uint8, device="cuda"), torch.zeros((G, N, K), dtype=torch.uint8, device="cuda")
    moe.moe_grouped_mm_fp8(xq, torch.ones((R, 1), device="cuda"), wq, torch.ones((G, 1, 1), device="cuda"), o, out=y)
    torch.cuda.synchronize()
    assert (big[:edge] == -7).all() and (big[edge + R:] == -7).all()
    del big, y, x, xq
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,x,w", [(torch.float16, 2.0**-20, 1.0), (torch.float16, 2.0**-24, 2.0**10),
                                       (torch.float16, 2.0**-12, 2.0**-14), (torch.bfloat16, 2.0**-130, 2.0**40),
                                       (torch.bfloat16, 2.0**-70, 2.0**-60)])
@pytest.mark.parametrize("R,N", [(16, 64), (9000, 1032)])
def test_values_below_the_normal_range_count(R, N, dtype, x, w):
    """Operands, products and results below the types' normal range: powers of
    two, so that every sum is exact."""
    banner(f"below the normal range: {dtype} {x} * {w}, {R} rows")
    K = 64
    o = torch.tensor([0, R], device="cuda", dtype=torch.int32)
    a = torch.full((R, K), x, dtype=dtype, device="cuda")
    b = torch.full((1, N, K), w, dtype=dtype, device="cuda")
    want = torch.full((R, N), x * w * K, dtype=torch.float64, device="cuda").to(dtype)
    assert float(want[0, 0]) > 0
    assert torch.equal(moe.moe_grouped_mm(a, b, o), want)
    assert torch.equal(moe.moe_grouped_mm(a, b.transpose(1, 2).contiguous(), o, w_kn=True), want)
    g = torch.full((R, N), w, dtype=dtype, device="cuda")
    dw = moe.moe_grouped_wgrad(g, a, o)
    assert torch.equal(dw.double(), torch.full_like(dw, x * w * R, dtype=torch.float64).float().double())
