"""routed_grouped_gemm_amd: one GPU's share of a routed MoE layer on MI355X.

A thin PyTorch binding over libmoe (include/moe.h). Every function here only
marshals arguments (device pointers, sizes, the current HIP stream) and calls
the C ABI of the same name; all computation runs in the library's HIP kernels.
PyTorch provides device memory and streams. No call records a gradient: the
gradients of the products and of the activation are calls of their own
(moe_grouped_mm with w_kn, moe_grouped_wgrad, moe_glu_checkpoint_backward), and
outputs do not require one whatever the inputs do. Importing the package fails
if the library has not been built (python routed_grouped_gemm_amd/build.py).
"""
from __future__ import annotations

import contextlib
import ctypes as C

import torch

from . import _lib
from ._lib import (MOE_ACT_GEGLU, MOE_ACT_SRELU, MOE_ACT_SWIGLU, MOE_FMT_MXFP4,  # noqa: F401
                   MOE_FMT_MXFP8, MOE_GEMM_PASS, MOE_GEMM_STREAMED, MOE_GEMM_TILED,
                   MOE_LAYER_SEPARATE_KERNELS,
                   MOE_LAYER_TOKEN_RING, MOE_MM_W_KN, MOE_ROUTE_RENORM,
                   MOE_SCALE_RULE_CEIL, MOE_T_BF16, MOE_T_F16, MOE_T_F32, MOE_W1_WRITE_TRANSPOSE,
                   MOE_WEIGHT_AT_COMBINE, MOE_WGRAD_ACCUMULATE, MOE_WGRAD_F32,
                   moe_epilogue, moe_layer_args, moe_weights)

lib = _lib.load()


class MoeError(RuntimeError):
    pass


def _check(status: int, name: str) -> None:
    if status != 0:
        raise MoeError(f"{name} failed: {lib.moe_status_string(status).decode()} (status {status})")


def _p(t):
    return None if t is None else t.data_ptr()


def _on(stream):
    """Context in which a wrapper allocates and launches: `stream` made the
    current stream (so the caching allocator ties every temporary and output
    to the stream whose kernels use it), or the current stream left as it is."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _stream():
    """Handle of the current stream (inside `_on`, the caller's stream)."""
    return torch.cuda.current_stream().cuda_stream


def _dev(t: torch.Tensor, dtype, name: str) -> torch.Tensor:
    if t.device.type != "cuda":
        raise MoeError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise MoeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise MoeError(f"{name} must be contiguous")
    return t


def version() -> str:
    return lib.moe_version().decode()


# ------------------------------------------------------------------ weights
def moe_prepacked_size(G: int, N: int, K: int, fmt: int) -> int:
    return int(lib.moe_prepacked_size(G, N, K, fmt))


def moe_quantize_mx(src: torch.Tensor, fmt: int, flags: int = 0, q=None, s=None, stream=None):
    """fp32 [rows, K] -> (codes, E8M0 scales); codes are [rows, K] E4M3 or
    [rows, K/2] packed E2M1."""
    _dev(src, torch.float32, "src")
    rows, K = src.shape
    with _on(stream):
        if q is None:
            q = torch.empty((rows, K if fmt == MOE_FMT_MXFP8 else K // 2), dtype=torch.uint8,
                            device=src.device)
        if s is None:
            s = torch.empty((rows, K // 32), dtype=torch.uint8, device=src.device)
        _check(lib.moe_quantize_mx(_p(src), rows, K, fmt, flags, _p(q), _p(s), _stream()),
               "moe_quantize_mx")
    return q, s


MOE_HBM_PROBE_SINK_WORDS = 8192


def moe_hbm_read_probe(src: torch.Tensor, sink=None, stream=None):
    """One streaming read of the bytes of `src` (a measurement utility).
    Returns sink (uint32 words, int32 dtype); their XOR is the XOR of the
    buffer's 4-byte words."""
    if not src.is_cuda or not src.is_contiguous():
        raise MoeError("src must be a contiguous device tensor")
    nbytes = src.numel() * src.element_size()
    with _on(stream):
        if sink is None:
            sink = torch.empty(MOE_HBM_PROBE_SINK_WORDS, dtype=torch.int32, device=src.device)
        _check(lib.moe_hbm_read_probe(_p(src), nbytes, _p(sink), _stream()), "moe_hbm_read_probe")
    return sink


class PackedWeights:
    """Prepacked expert weights (device buffer + its moe_weights descriptor)."""

    def __init__(self, q: torch.Tensor, s: torch.Tensor, fmt: int, is_w1: bool, stream=None):
        _dev(q, torch.uint8, "q")
        _dev(s, torch.uint8, "s")
        G, N = q.shape[0], q.shape[1]
        K = s.shape[2] * 32
        nbytes = moe_prepacked_size(G, N, K, fmt)
        if nbytes == 0:
            raise MoeError(f"bad weight shape G={G} N={N} K={K}")
        with _on(stream):
            self.buf = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
            _check(lib.moe_prepack_weights(_p(q), _p(s), G, N, K, fmt, int(is_w1), _p(self.buf),
                                           nbytes, _stream()), "moe_prepack_weights")
        self.desc = moe_weights(fmt, G, N, K, int(is_w1), 0, _p(self.buf), nbytes)
        self.G, self.N, self.K, self.fmt, self.is_w1 = G, N, K, fmt, bool(is_w1)

    @classmethod
    def empty(cls, G: int, N: int, K: int, fmt: int, is_w1: bool, device="cuda"):
        """An unfilled buffer of the right size (filled later, e.g. one group at a time)."""
        self = cls.__new__(cls)
        nbytes = moe_prepacked_size(G, N, K, fmt)
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.desc = moe_weights(fmt, G, N, K, int(is_w1), 0, _p(self.buf), nbytes)
        self.G, self.N, self.K, self.fmt, self.is_w1 = G, N, K, fmt, bool(is_w1)
        return self

    @property
    def group_stride(self) -> int:
        return moe_prepacked_size(1, self.N, self.K, self.fmt)

    def fill_group(self, g: int, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
        """Prepack one expert's logical codes q [N, K or K/2] and scales s [N, K/32]
        into group slot g."""
        _dev(q, torch.uint8, "q")
        _dev(s, torch.uint8, "s")
        st = self.group_stride
        dst = self.buf[g * st:(g + 1) * st]
        with _on(stream):
            _check(lib.moe_prepack_weights(_p(q), _p(s), 1, self.N, self.K, self.fmt, int(self.is_w1),
                                           _p(dst), st, _stream()), "moe_prepack_weights")

    def ref(self):
        return C.byref(self.desc)


def _wref(w):
    return None if w is None else w.ref()


class Epilogue:
    """The W1 epilogue variant (moe_epilogue): activation (MOE_ACT_*), Swish
    slope beta, clamp limit (0: none), optional per-group bias f32 [G, 2I] and
    optional BF16 pre-activation output [R_max, 2I] (both device tensors,
    referenced here so they outlive the call)."""

    def __init__(self, act: int = MOE_ACT_SWIGLU, beta: float = 1.0, limit: float = 0.0, bias=None,
                 save_pre=None):
        if bias is not None:
            _dev(bias, torch.float32, "bias")
        if save_pre is not None:
            _dev(save_pre, torch.uint16, "save_pre")
        self.bias, self.save_pre = bias, save_pre
        self.desc = moe_epilogue(act, beta, limit, 0, _p(bias), _p(save_pre))

    def ref(self):
        return C.byref(self.desc)


def _eref(e):
    return None if e is None else e.ref()


# ------------------------------------------------------------------- route
def moe_route(logits: torch.Tensor, k: int, flags: int = 0, topk_idx=None, topk_w=None, stream=None):
    _dev(logits, torch.float32, "logits")
    T, E = logits.shape
    with _on(stream):
        if topk_idx is None:
            topk_idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
        if topk_w is None:
            topk_w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
        _check(lib.moe_route(_p(logits), T, E, k, flags, _p(topk_idx), _p(topk_w), _stream()),
               "moe_route")
    return topk_idx, topk_w


# ----------------------------------------------------------------- permute
def moe_permute(topk_idx, topk_w, e0: int, n_local: int, shared: bool, xq=None, xs=None,
                stream=None):
    """Returns a dict: counts, offsets, offsets32, row_src, row_w, slot_row,
    xq_perm, xs_perm (the last two only when xq/xs are given)."""
    _dev(topk_idx, torch.int32, "topk_idx")
    _dev(topk_w, torch.float32, "topk_w")
    T, k = topk_idx.shape
    s = int(bool(shared))
    G = n_local + s
    R_max = T * k + s * T
    dev = topk_idx.device
    H = xq.shape[1] if xq is not None else 256
    with _on(stream):
        out = dict(
            counts=torch.empty(G, dtype=torch.int32, device=dev),
            offsets=torch.empty(G + 1, dtype=torch.int32, device=dev),
            offsets32=torch.empty(G + 1, dtype=torch.int32, device=dev),
            row_src=torch.empty(max(R_max, 1), dtype=torch.int32, device=dev),
            row_w=torch.empty(max(R_max, 1), dtype=torch.float32, device=dev),
            slot_row=torch.empty((T, k + s), dtype=torch.int32, device=dev),
        )
        if xq is not None:
            _dev(xq, torch.uint8, "xq")
            _dev(xs, torch.uint8, "xs")
            out["xq_perm"] = torch.empty((max(R_max, 1), H), dtype=torch.uint8, device=dev)
            out["xs_perm"] = torch.empty((max(R_max, 1), H // 32), dtype=torch.uint8, device=dev)
        nws = int(lib.moe_permute_workspace_size(T, k, G))
        ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=dev)
        _check(lib.moe_permute(_p(topk_idx), _p(topk_w), T, k, e0, n_local, s, _p(xq), _p(xs), H,
                               _p(out["counts"]), _p(out["offsets"]), _p(out["offsets32"]),
                               _p(out["row_src"]), _p(out["row_w"]), _p(out["slot_row"]),
                               _p(out.get("xq_perm")), _p(out.get("xs_perm")), _p(ws), nws,
                               _stream()), "moe_permute")
    return out


# ----------------------------------------------------------------- grouped
def moe_transposed_ld(R_max: int, G: int) -> int:
    return int(lib.moe_transposed_ld(R_max, G))


def moe_grouped_w1(w1: PackedWeights, counts, offsets, row_w, xq, xs, I: int,
                   flags: int = 0, w1_shared: PackedWeights | None = None, offsets32=None,
                   hq=None, hs=None, hTq=None, hTs=None, row_src=None,
                   R_max: int | None = None, epi: Epilogue | None = None, stream=None):
    """xq/xs: the grouped rows [R_max, H] (row_src None) or the token rows
    [T, H] read through row_src (then R_max must be given). The launch
    configuration follows R_max / counts.shape[0] (see include/moe.h)."""
    H = xq.shape[1]
    if R_max is None:
        R_max = xq.shape[0]
    G = counts.shape[0]
    dev = xq.device
    with _on(stream):
        if hq is None:
            hq = torch.empty((R_max, I), dtype=torch.uint8, device=dev)
        if hs is None:
            hs = torch.empty((R_max, I // 32), dtype=torch.uint8, device=dev)
        if (flags & MOE_W1_WRITE_TRANSPOSE) and hTq is None:
            ld = moe_transposed_ld(R_max, G)
            hTq = torch.empty((I, ld), dtype=torch.uint8, device=dev)
            hTs = torch.empty((I, ld // 32), dtype=torch.uint8, device=dev)
        nws = int(lib.moe_grouped_workspace_size(R_max, G, 2 * I, H))
        ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=dev)
        _check(lib.moe_grouped_w1(w1.ref(), _wref(w1_shared), _p(counts), _p(offsets), _p(offsets32),
                                  _p(row_w), _p(xq), _p(xs), _p(row_src), xq.shape[0], R_max, H, I, G,
                                  _eref(epi), flags, _p(hq), _p(hs), _p(hTq), _p(hTs), _p(ws), nws,
                                  _stream()),
               "moe_grouped_w1")
    return hq, hs, hTq, hTs


def moe_grouped_w1_backward(w2t: PackedWeights, counts, offsets, row_w, dyq, dys, row_src, pre, I: int,
                            epi: Epilogue | None = None, flags: int = 0, offsets32=None,
                            w2t_shared: PackedWeights | None = None, want_dw: bool = True, stream=None):
    """The backward of the fused W1 epilogue: w2t holds W2^T per group (N = I,
    K = H), dyq/dys the layer output's gradient in token order [T, H] (E4M3 +
    E8M0), row_src the grouped rows' tokens, pre the saved BF16 pre-activation
    [R_max, 2I]. Returns a dict: dq [R_max, 2I], ds [R_max, 2I/32], dTq/dTs
    (with MOE_W1_WRITE_TRANSPOSE), dw [R_max] (with row_w and want_dw)."""
    R_max = pre.shape[0]
    H = dyq.shape[1]
    G = counts.shape[0]
    dev = dyq.device
    with _on(stream):
        out = dict(dq=torch.empty((R_max, 2 * I), dtype=torch.uint8, device=dev),
                   ds=torch.empty((R_max, 2 * I // 32), dtype=torch.uint8, device=dev),
                   dTq=None, dTs=None, dw=None)
        if flags & MOE_W1_WRITE_TRANSPOSE:
            ld = moe_transposed_ld(R_max, G)
            out["dTq"] = torch.zeros((2 * I, ld), dtype=torch.uint8, device=dev)
            out["dTs"] = torch.zeros((2 * I, ld // 32), dtype=torch.uint8, device=dev)
        if want_dw and row_w is not None:
            out["dw"] = torch.empty(R_max, dtype=torch.float32, device=dev)
        nws = int(lib.moe_backward_workspace_size(R_max, G, H, I))
        ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=dev)
        _check(lib.moe_grouped_w1_backward(
            w2t.ref(), _wref(w2t_shared), _p(counts), _p(offsets), _p(offsets32), _p(row_w), _p(dyq),
            _p(dys), _p(row_src), dyq.shape[0], _p(pre), R_max, H, I, G, _eref(epi), flags,
            _p(out["dq"]), _p(out["ds"]), _p(out["dTq"]), _p(out["dTs"]), _p(out["dw"]), _p(ws), nws,
            _stream()), "moe_grouped_w1_backward")
    return out


def moe_grouped_w2(w2: PackedWeights, counts, offsets, hq, hs, H: int,
                   w2_shared: PackedWeights | None = None, y=None, flags: int = 0, stream=None):
    R_max, I = hq.shape
    G = counts.shape[0]
    with _on(stream):
        if y is None:
            y = torch.empty((R_max, H), dtype=torch.uint16, device=hq.device)
        nws = int(lib.moe_grouped_workspace_size(R_max, G, H, I))
        ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=hq.device)
        _check(lib.moe_grouped_w2(w2.ref(), _wref(w2_shared), _p(counts), _p(offsets), _p(hq), _p(hs),
                                  R_max, H, I, G, flags, _p(y), _p(ws), nws, _stream()),
               "moe_grouped_w2")
    return y


# ----------------------------------------------------------------- combine
def moe_combine(y, slot_row, H: int, row_w=None, out=None, stream=None):
    """y: BF16 rows [R, H] (bfloat16, or their bits as uint16 or int16). Returns
    the tokens' sums, BF16 bits in uint16 [T, H]."""
    if y.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise MoeError(f"y must be BF16 (bfloat16, or its bits as uint16 or int16), got {y.dtype}")
    if not y.is_contiguous() or (y.dim() > 1 and y.shape[-1] != H):
        raise MoeError(f"y must be contiguous rows of {H}, got {tuple(y.shape)} with strides {y.stride()}")
    T, ks = slot_row.shape
    with _on(stream):
        if out is None:
            out = torch.empty((T, H), dtype=torch.uint16, device=y.device)
        _check(lib.moe_combine(_p(y), _p(slot_row), _p(row_w), T, ks, H, _p(out), _stream()),
               "moe_combine")
    return out


# ------------------------------------------------------------------- layer
_NAMES = ["topk_idx", "topk_w", "counts", "offsets", "offsets32", "row_src", "row_w", "slot_row",
          "hq", "hs", "y", "scratch", "ctrl"]


class LayerWorkspace:
    """Device workspace of moe_layer plus views of its intermediates."""

    def __init__(self, T, E_tot, k, E_loc, H, I, shared=False, flags=0, device="cuda"):
        s = int(bool(shared))
        self.shape = (T, E_tot, k, E_loc, H, I, s, flags)
        self.nbytes = int(lib.moe_layer_workspace_size(T, E_tot, k, E_loc, H, I, s, flags))
        self.buf = torch.empty(max(self.nbytes, 1), dtype=torch.uint8, device=device)
        offs = (C.c_size_t * len(_NAMES))()
        lib.moe_layer_workspace_offsets(T, E_tot, k, E_loc, H, I, s, flags, offs)
        self.offsets = list(offs)
        self.scratch_offset = self.offsets[_NAMES.index("scratch")]

    def view(self, name: str) -> torch.Tensor:
        T, E_tot, k, E_loc, H, I, s, _ = self.shape
        R = T * k + s * T
        G = E_loc + s
        shapes = {
            "topk_idx": ((T, k), torch.int32), "topk_w": ((T, k), torch.float32),
            "counts": ((G,), torch.int32), "offsets": ((G + 1,), torch.int32),
            "offsets32": ((G + 1,), torch.int32), "row_src": ((R,), torch.int32),
            "row_w": ((R,), torch.float32), "slot_row": ((T, k + s), torch.int32),
            "hq": ((R, I), torch.uint8), "hs": ((R, I // 32), torch.uint8),
            "y": ((R, H), torch.uint16),
            "ctrl": ((8 + G + H // 64,), torch.int32),
        }
        shp, dt = shapes[name]
        o = self.offsets[_NAMES.index(name)]
        n = 1
        for d in shp:
            n *= d
        nbytes = n * torch.tensor([], dtype=dt).element_size()
        return self.buf[o:o + nbytes].view(dt).view(shp)


def _layer_args(logits, xq, xs, w1, w2, k, e0, n_local, shared, flags, out, hTq, hTs, epi=None):
    T, E_tot = logits.shape
    H = xq.shape[1]
    args = moe_layer_args()
    args.logits, args.T, args.E_tot, args.k = _p(logits), T, E_tot, k
    args.e0, args.E_loc = e0, n_local
    args.xq, args.xs, args.H, args.I = _p(xq), _p(xs), H, w1.N // 2
    args.w1, args.w2 = C.pointer(w1.desc), C.pointer(w2.desc)
    if shared is not None:
        args.shared_w1, args.shared_w2 = C.pointer(shared[0].desc), C.pointer(shared[1].desc)
    args.flags = flags
    args.hTq, args.hTs = _p(hTq), _p(hTs)
    args.out = _p(out)
    if epi is not None:
        args.epi = C.pointer(epi.desc)
    return args


def moe_layer(logits, xq, xs, w1: PackedWeights, w2: PackedWeights, k: int, e0: int = 0,
              n_local: int | None = None, shared=None, flags: int = 0, out=None, ws=None,
              hTq=None, hTs=None, epi: Epilogue | None = None, stream=None):
    """Whole layer. shared = (PackedWeights W1, PackedWeights W2) or None.
    Returns out (bf16 bits as uint16 [T, H])."""
    _dev(logits, torch.float32, "logits")
    _dev(xq, torch.uint8, "xq")
    _dev(xs, torch.uint8, "xs")
    T, E_tot = logits.shape
    H = xq.shape[1]
    I = w1.N // 2
    n_local = w1.G if n_local is None else n_local
    s = 1 if shared is not None else 0
    with _on(stream):
        if out is None:
            out = torch.empty((T, H), dtype=torch.uint16, device=xq.device)
        if ws is None:
            ws = LayerWorkspace(T, E_tot, k, n_local, H, I, bool(s), flags, device=xq.device)
        args = _layer_args(logits, xq, xs, w1, w2, k, e0, n_local, shared, flags, out, hTq, hTs, epi)
        _check(lib.moe_layer(C.byref(args), _p(ws.buf), ws.nbytes, _stream()), "moe_layer")
    return out


def moe_layer_noalloc(logits, xq, xs, w1: PackedWeights, w2: PackedWeights, k: int, e0: int = 0,
                      n_local: int | None = None, shared=None, flags: int = 0, out=None,
                      hTq=None, hTs=None, stream=None):
    """moe_layer with the library's fixed per-GPU workspace (no workspace
    argument, nothing allocated by the library). `out` must be given when the
    call must not allocate either; calls overlapping on one GPU race."""
    _dev(logits, torch.float32, "logits")
    _dev(xq, torch.uint8, "xq")
    _dev(xs, torch.uint8, "xs")
    T = logits.shape[0]
    n_local = w1.G if n_local is None else n_local
    with _on(stream):
        if out is None:
            out = torch.empty((T, xq.shape[1]), dtype=torch.uint16, device=xq.device)
        args = _layer_args(logits, xq, xs, w1, w2, k, e0, n_local, shared, flags, out, hTq, hTs)
        _check(lib.moe_layer_noalloc(C.byref(args), _stream()), "moe_layer_noalloc")
    return out


def layer(xq, xs, logits, w1: PackedWeights, w2: PackedWeights, k: int, e0: int = 0,
          n_local: int | None = None, shared=None, flags: int = 0, out=None, **kw):
    """moe_layer with the argument order of the activation-first call form
    (x codes, x scales, router logits, weights, top-k)."""
    return moe_layer(logits, xq, xs, w1, w2, k, e0, n_local, shared, flags, out=out, **kw)


# ------------------------------------------- 16-bit and block-FP8 products
_T16 = {torch.bfloat16: MOE_T_BF16, torch.float16: MOE_T_F16}
_T_ANY = {**_T16, torch.float32: MOE_T_F32}


def _mat(t: torch.Tensor, types, name: str, device=None) -> torch.Tensor:
    """A 2-D device tensor whose rows are dense (its row stride may be larger)."""
    if t.device.type != "cuda":
        raise MoeError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise MoeError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in types:
        raise MoeError(f"{name} must be one of {[str(d) for d in types]}, got {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise MoeError(f"{name} must be 2-D with dense rows")
    return t


def _ld(t: torch.Tensor) -> int:
    """Leading dimension: the row stride (a single row's is not defined by its data)."""
    if t.shape[0] > 1:
        if t.stride(0) < t.shape[1]:
            raise MoeError("rows overlap")
        return t.stride(0)
    return t.shape[1]


def _dense(t, shape, dtype, name: str, device) -> None:
    """Check an optional dense device tensor of a known shape and type."""
    if t is None or (t.device == device and t.dtype == dtype and t.shape == shape and t.is_contiguous()):
        return
    if t.device != device:
        raise MoeError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise MoeError(f"{name} must be {dtype}, got {t.dtype}")
    raise MoeError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(t.shape)}")


class _Here:
    """The context of a call on the current device and stream: nothing to switch."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_HERE = _Here()


@contextlib.contextmanager
def _elsewhere(device, stream):
    if stream is not None and stream.device != device:
        raise MoeError(f"stream is on {stream.device}, expected {device}")
    with torch.cuda.device(device), _on(stream):
        yield


def _at(device, stream):
    """The operands' device made current, and `stream` (or that device's
    current stream) the one that allocates and launches. The usual case, both
    already current, costs no switch: a small call's time is host time."""
    if stream is None and device.index == torch.cuda.current_device():
        return _HERE
    return _elsewhere(device, stream)


def _raw_stream(device) -> int:
    """Handle of the device's current stream, without building a Stream object."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _ws(nbytes: int, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _offsets(offsets, G: int, device) -> None:
    _dense(offsets, (G + 1,), torch.int32, "offsets", device)


def _n_rows(src, t, name: str) -> int:
    """Rows that a call reads of t, directly or through src (whose type and
    device are checked once all operands give the same number)."""
    if src is None:
        return t.shape[0]
    if src.dim() != 1:
        raise MoeError(f"{name} must be 1-D, got {tuple(src.shape)}")
    return src.shape[0]


def moe_grouped_mm(x, w, offsets, w_kn: bool = False, row_src=None, out=None, stream=None):
    """y[r] = x[r] . W_g^T for the rows r of group g (offsets, int32 [G + 1] on
    the device): w [G, N, K], or [G, K, N] with w_kn. x [R, K], or [T, K] read
    through row_src (int32 [R]). bf16 or fp16; returns [R, N] of that type,
    rows of no group unwritten. Records no gradient: the rows' is this call with
    w_kn the other way, the weights' is moe_grouped_wgrad."""
    _mat(x, _T16, "x")
    dev, (T, K) = x.device, x.shape
    if w.dim() != 3 or w.shape[1 if w_kn else 2] != K:
        raise MoeError(f"w {tuple(w.shape)} does not fit rows of {K}")
    _dense(w, w.shape, x.dtype, "w", dev)
    G, N = w.shape[0], w.shape[2 if w_kn else 1]
    _offsets(offsets, G, dev)
    R = _n_rows(row_src, x, "row_src")
    _dense(row_src, (R,), torch.int32, "row_src", dev)
    with _at(dev, stream):
        if out is None:
            out = torch.empty((R, N), dtype=x.dtype, device=dev)
        elif _mat(out, (x.dtype,), "out", dev).shape != (R, N):
            raise MoeError(f"out must be [{R}, {N}], got {tuple(out.shape)}")
        nws = int(lib.moe_grouped_mm_workspace_size(R, G, N, K))
        ws = _ws(nws, dev)
        _check(lib.moe_grouped_mm(_p(x), T, _ld(x), _p(row_src), _p(w), _T16[x.dtype], _p(offsets), R, N, K, G,
                                  MOE_MM_W_KN if w_kn else 0, _p(out), _ld(out), _p(ws), nws, _raw_stream(dev)),
               "moe_grouped_mm")
    return out


def moe_grouped_wgrad(dy, x, offsets, dy_src=None, x_src=None, x_scales=None, out=None, accumulate: bool = False,
                      out_dtype=torch.float32, stream=None):
    """dW_g = dy^T x over the rows of each group: [G, N, K] in out_dtype
    (float32, or dy's type). dy [R, N] and x [R, K], or token-order arrays
    read through dy_src / x_src (int32 [R]). With x_scales, x is an 8-bit
    checkpoint (codes and scales of moe_quantize_block). accumulate adds to
    `out`, which must then be given. Records no gradient."""
    _mat(dy, _T16, "dy")
    dev, N = dy.device, dy.shape[1]
    _mat(x, (torch.uint8,) if x_scales is not None else (dy.dtype,), "x", dev)
    K = x.shape[1]
    _dense(x_scales, (x.shape[0], -(-K // 128)), torch.float32, "x_scales", dev)
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise MoeError(f"offsets must be 1-D with at least 2 elements, got {tuple(offsets.shape)}")
    G = offsets.shape[0] - 1
    _offsets(offsets, G, dev)
    n = {_n_rows(dy_src, dy, "dy_src"), _n_rows(x_src, x, "x_src")}
    if len(n) != 1:
        raise MoeError(f"dy and x give different numbers of rows: {sorted(n)}")
    R = n.pop()
    _dense(dy_src, (R,), torch.int32, "dy_src", dev)
    _dense(x_src, (R,), torch.int32, "x_src", dev)
    if out_dtype not in (torch.float32, dy.dtype):
        raise MoeError(f"out_dtype must be float32 or {dy.dtype}, got {out_dtype}")
    if accumulate and out is None:
        raise MoeError("accumulate needs out")
    flags = (MOE_WGRAD_ACCUMULATE if accumulate else 0) | (MOE_WGRAD_F32 if out_dtype == torch.float32 else 0)
    with _at(dev, stream):
        if out is None:
            out = torch.empty((G, N, K), dtype=out_dtype, device=dev)
        _dense(out, (G, N, K), out_dtype, "out", dev)
        nws = int(lib.moe_grouped_wgrad_workspace_size(R, G, N, K))
        ws = _ws(nws, dev)
        _check(lib.moe_grouped_wgrad(_p(dy), dy.shape[0], _ld(dy), _p(dy_src), _p(x), x.shape[0], _ld(x), _p(x_src),
                                     _p(x_scales), _T16[dy.dtype], _p(offsets), R, N, K, G, flags, _p(out), _p(ws),
                                     nws, _raw_stream(dev)), "moe_grouped_wgrad")
    return out


def moe_grouped_mm_plan(R_max: int, G: int, N: int, K: int, fp8: bool = False) -> tuple[int, int]:
    """(rows of a tile, parts of the reduction axis) of a grouped product of these sizes."""
    rows, parts = C.c_int32(), C.c_int32()
    _check(lib.moe_grouped_mm_plan(R_max, G, N, K, int(fp8), C.byref(rows), C.byref(parts)), "moe_grouped_mm_plan")
    return rows.value, parts.value


def moe_grouped_wgrad_plan(R_max: int, G: int, N: int, K: int) -> int:
    """Rows of a part of a weight gradient's groups (0: no group can be longer)."""
    rows = C.c_int32()
    _check(lib.moe_grouped_wgrad_plan(R_max, G, N, K, C.byref(rows)), "moe_grouped_wgrad_plan")
    return rows.value


def moe_quantize_block(x, n_rows=None, codes=None, scales=None, stream=None):
    """Rows of x (bf16, fp16 or fp32 [R, K]) to E4M3 codes uint8 [R, K] and
    power-of-two scales f32 [R, ceil(K/128)]. n_rows: an int32 device tensor
    of one element; rows from it on are left unwritten. Records no gradient."""
    _mat(x, _T_ANY, "x")
    dev, (R, K) = x.device, x.shape
    _dense(n_rows, () if n_rows is not None and n_rows.dim() == 0 else (1,), torch.int32, "n_rows", dev)
    with _at(dev, stream):
        if codes is None:
            codes = torch.empty((R, K), dtype=torch.uint8, device=dev)
        if scales is None:
            scales = torch.empty((R, -(-K // 128)), dtype=torch.float32, device=dev)
        _dense(codes, (R, K), torch.uint8, "codes", dev)
        _dense(scales, (R, -(-K // 128)), torch.float32, "scales", dev)
        _check(lib.moe_quantize_block(_p(x), _T_ANY[x.dtype], R, K, _ld(x), _p(n_rows), _p(codes), _p(scales),
                                      _raw_stream(dev)), "moe_quantize_block")
    return codes, scales


def moe_quantize_block_weights(w, codes=None, scales=None, stream=None):
    """w [G, N, K] (bf16, fp16 or fp32) to E4M3 codes uint8 [G, N, K] and
    power-of-two scales f32 [G, ceil(N/128), ceil(K/128)]. Records no gradient."""
    if w.device.type != "cuda" or w.dtype not in _T_ANY or w.dim() != 3 or not w.is_contiguous():
        raise MoeError("w must be a contiguous 3-D device tensor of bf16, fp16 or fp32")
    dev, (G, N, K) = w.device, w.shape
    shp = (G, -(-N // 128), -(-K // 128))
    with _at(dev, stream):
        if codes is None:
            codes = torch.empty((G, N, K), dtype=torch.uint8, device=dev)
        if scales is None:
            scales = torch.empty(shp, dtype=torch.float32, device=dev)
        _dense(codes, (G, N, K), torch.uint8, "codes", dev)
        _dense(scales, shp, torch.float32, "scales", dev)
        _check(lib.moe_quantize_block_weights(_p(w), _T_ANY[w.dtype], G, N, K, _p(codes), _p(scales), _raw_stream(dev)),
               "moe_quantize_block_weights")
    return codes, scales


def moe_grouped_mm_fp8(xq, xs, wq, ws, offsets, row_src=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """Grouped product of block-scaled FP8 operands: xq uint8 [R, K] (or [T, K]
    read through row_src) with xs f32 [.., ceil(K/128)], wq uint8 [G, N, K]
    with ws f32 [G, ceil(N/128), ceil(K/128)]. Returns [R, N] bf16 or fp16.
    Records no gradient."""
    if xq.device.type != "cuda" or xq.dim() != 2 or wq.dim() != 3 or wq.shape[2] != xq.shape[1]:
        raise MoeError("xq must be a 2-D device tensor and wq [G, N, K] of the same K")
    dev, (T, K) = xq.device, xq.shape
    G, N = wq.shape[0], wq.shape[1]
    kb = -(-K // 128)
    _dense(xq, (T, K), torch.uint8, "xq", dev)
    _dense(xs, (T, kb), torch.float32, "xs", dev)
    _dense(wq, (G, N, K), torch.uint8, "wq", dev)
    _dense(ws, (G, -(-N // 128), kb), torch.float32, "ws", dev)
    _offsets(offsets, G, dev)
    R = _n_rows(row_src, xq, "row_src")
    _dense(row_src, (R,), torch.int32, "row_src", dev)
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _T16:
        raise MoeError(f"out_dtype must be bf16 or fp16, got {out_dtype}")
    with _at(dev, stream):
        if out is None:
            out = torch.empty((R, N), dtype=out_dtype, device=dev)
        elif _mat(out, _T16, "out", dev).shape != (R, N):
            raise MoeError(f"out must be [{R}, {N}], got {tuple(out.shape)}")
        nws = int(lib.moe_grouped_mm_fp8_workspace_size(R, G, N, K))
        wsp = _ws(nws, dev)
        _check(lib.moe_grouped_mm_fp8(_p(xq), _p(xs), T, _p(row_src), _p(wq), _p(ws), _p(offsets), R, N, K, G,
                                      _T16[out_dtype], _p(out), _ld(out), _p(wsp), nws, _raw_stream(dev)),
               "moe_grouped_mm_fp8")
    return out


def moe_glu_checkpoint(pre, row_w=None, n_rows=None, epi: Epilogue | None = None, keep: bool = True, h=None,
                       codes=None, scales=None, stream=None):
    """pre = [gate | up] rows [R, 2I] (bf16 or fp16) to h = act(gate) * up * w
    [R, I] and, with keep, pre in 8 bits: codes uint8 [R, 2I], scales f32
    [R, 2, ceil(I/128)]. Returns (h, codes, scales). Records no gradient: that is
    moe_glu_checkpoint_backward."""
    _mat(pre, _T16, "pre")
    dev, R, I = pre.device, pre.shape[0], pre.shape[1] // 2
    if pre.shape[1] % 2:
        raise MoeError("pre must have an even number of columns")
    if not keep and (codes is not None or scales is not None):
        raise MoeError("codes and scales are written only with keep")
    shp = (R, 2, -(-I // 128))
    _dense(row_w, (R,), torch.float32, "row_w", dev)
    _dense(n_rows, () if n_rows is not None and n_rows.dim() == 0 else (1,), torch.int32, "n_rows", dev)
    with _at(dev, stream):
        if h is None:
            h = torch.empty((R, I), dtype=pre.dtype, device=dev)
        if keep and codes is None:
            codes = torch.empty((R, 2 * I), dtype=torch.uint8, device=dev)
        if keep and scales is None:
            scales = torch.empty(shp, dtype=torch.float32, device=dev)
        _dense(h, (R, I), pre.dtype, "h", dev)
        _dense(codes, (R, 2 * I), torch.uint8, "codes", dev)
        _dense(scales, shp, torch.float32, "scales", dev)
        _check(lib.moe_glu_checkpoint(_p(pre), _T16[pre.dtype], R, I, _ld(pre), _p(row_w), _p(n_rows), _eref(epi),
                                      _p(h), _p(codes), _p(scales), _raw_stream(dev)), "moe_glu_checkpoint")
    return h, codes, scales


def moe_glu_checkpoint_backward(codes, scales, dh, row_w=None, n_rows=None, epi: Epilogue | None = None,
                                want_h: bool = True, want_dw: bool = True, stream=None):
    """The backward of moe_glu_checkpoint from its 8-bit codes and scales and
    dh [R, I] (bf16 or fp16). Returns a dict: dpre [R, 2I], h [R, I] (the
    forward's product, recomputed) and dw f32 [R] (None where not wanted)."""
    _mat(dh, _T16, "dh")
    dev, (R, I) = dh.device, dh.shape
    _dense(codes, (R, 2 * I), torch.uint8, "codes", dev)
    _dense(scales, (R, 2, -(-I // 128)), torch.float32, "scales", dev)
    _dense(row_w, (R,), torch.float32, "row_w", dev)
    _dense(n_rows, () if n_rows is not None and n_rows.dim() == 0 else (1,), torch.int32, "n_rows", dev)
    with _at(dev, stream):
        out = dict(dpre=torch.empty((R, 2 * I), dtype=dh.dtype, device=dev),
                   h=torch.empty((R, I), dtype=dh.dtype, device=dev) if want_h else None,
                   dw=torch.empty(R, dtype=torch.float32, device=dev) if want_dw else None)
        _check(lib.moe_glu_checkpoint_backward(_p(codes), _p(scales), _p(dh), _T16[dh.dtype], R, I, _ld(dh),
                                               _p(row_w), _p(n_rows), _eref(epi), _p(out["dpre"]), _p(out["h"]),
                                               _p(out["dw"]), _raw_stream(dev)), "moe_glu_checkpoint_backward")
    return out
