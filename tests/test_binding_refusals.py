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


def test_sources_and_offsets_of_no_dimension():
    """Refused as MoeError like every other argument, whatever their dimensions."""
    class Device(torch.Tensor):                     # a host tensor that claims a device, for the checks alone
        device = torch.device("cuda", 0)

    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype).as_subclass(Device)

    i32 = torch.int32
    x, dy, w, off = t(16, 64), t(16, 32), t(2, 32, 64), t(3, dtype=i32)
    q, s = t(16, 64, dtype=torch.uint8), t(16, 1, dtype=torch.float32)
    wq, ws = t(2, 32, 64, dtype=torch.uint8), t(2, 1, 1, dtype=torch.float32)
    none, empty = t(dtype=i32), t(0, dtype=i32)
    for f in (lambda: moe.moe_grouped_mm(x, w, off, row_src=none),
              lambda: moe.moe_grouped_mm_fp8(q, s, wq, ws, off, row_src=none),
              lambda: moe.moe_grouped_wgrad(dy, x, off, x_src=none),
              lambda: moe.moe_grouped_wgrad(dy, x, off, dy_src=none),
              lambda: moe.moe_grouped_mm(x, w, none), lambda: moe.moe_grouped_mm(x, w, empty),
              lambda: moe.moe_grouped_wgrad(dy, x, none), lambda: moe.moe_grouped_wgrad(dy, x, empty),
              lambda: moe.moe_grouped_wgrad(dy, x, t(1, dtype=i32))):
        with pytest.raises(moe.MoeError):
            f()
