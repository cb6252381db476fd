"""The largest h of the layer for a few tokens: refused from 2^26 values on (no GPU needed)."""
import ctypes as C

from routed_grouped_gemm_amd import _lib

lib = _lib.load()


def test_values_of_h():
    size = lib.moe_layer_few_workspace_size
    assert size(32, 31, 2048, 8, 65536, 1) == 0              # 2^26 values
    for T, k, s, I in ((32, 31, 1, 65520), (31, 31, 1, 65536), (32, 31, 0, 65536), (1, 1, 0, 8)):
        assert size(T, k, 2048, 8, I, s) >= 4 * T * (k + s) * I
    F = 4096
    a = _lib.moe_few_args(logits=F, T=32, E_tot=64, k=31, e0=0, E_loc=64, dtype=_lib.MOE_T_BF16, x=F, ldx=8, H=8, I=65536, w1=F, w2=F,
                          shared_w1=F, shared_w2=F, out=F, ld_out=8)
    assert lib.moe_layer_few(C.byref(a), F, 1 << 40, None) == 2      # MOE_ERR_SHAPE
