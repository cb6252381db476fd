"""What the Python bindings refuse before any kernel is launched (host tensors
stand in for device tensors: every refusal here comes before they are read)."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("routed_grouped_gemm_amd")


@pytest.mark.parametrize("y", [torch.zeros((8, 256), dtype=torch.float16), torch.zeros((8, 256)),
                               torch.zeros((8, 512), dtype=torch.bfloat16)[:, :256],
                               torch.zeros((8, 264), dtype=torch.bfloat16)],
                         ids=["fp16", "fp32", "strided", "other width"])
def test_combine_reads_dense_bf16_rows(y):
    """The combine reads BF16 bits at row * H: FP16 rows (an FP16 grouped product's)
    or rows of another stride or width would be summed as something else."""
    with pytest.raises(moe.MoeError, match="y must be"):
        moe.moe_combine(y, torch.zeros((4, 2), dtype=torch.int32), 256)
