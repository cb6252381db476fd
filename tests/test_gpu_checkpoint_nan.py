"""NaN in the checkpointed activation: every activation passes it on, forward and
through the kept codes, and only to the elements that depend on it."""
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("routed_grouped_gemm_amd")


@pytest.mark.parametrize("limit", [0.0, 2.0])
@pytest.mark.parametrize("act", [moe.MOE_ACT_SWIGLU, moe.MOE_ACT_GEGLU, moe.MOE_ACT_SRELU])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nan_gate_and_up(act, limit, dtype):
    """h = a(g) u: NaN where g or u is. dg = dh w u a'(g), du = dh w a(g): dg NaN
    where g or u is, du where g is (with a limit a NaN is outside it, |NaN| <=
    limit being false: its own gradient's factor is 0, and NaN * 0 is NaN in dg,
    where a'(NaN) stands beside the factor; du's factor of a NaN u is 0)."""
    banner(f"NaN through activation {act}, limit {limit}, {dtype}")
    R, I = 4, 264
    g = torch.Generator(device="cuda").manual_seed(1)
    pre = torch.rand((R, 2 * I), generator=g, device="cuda").add(0.25).to(dtype)     # positive: no factor is 0
    pre[1, 5] = float("nan")                         # a gate
    pre[2, I + 7] = float("nan")                     # an up value
    e = moe.Epilogue(act, 1.0, limit)
    h, q, s = moe.moe_glu_checkpoint(pre, epi=e)
    want = torch.zeros((R, I), dtype=torch.bool, device="cuda")
    want[1, 5] = want[2, 7] = True
    assert torch.equal(h.isnan(), want)
    o = moe.moe_glu_checkpoint_backward(q, s, torch.ones((R, I), dtype=dtype, device="cuda"), epi=e)
    assert torch.equal(o["h"].isnan(), want)
    assert torch.equal(o["dpre"][:, :I].isnan(), want)
    du = torch.zeros_like(want)
    du[1, 5] = True
    assert torch.equal(o["dpre"][:, I:].isnan(), du)
    assert o["dw"].isnan().tolist() == [False, True, True, False]
