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
