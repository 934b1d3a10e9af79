"""Python binding of libs2r: sparse-sketch gradient aggregation on MI355X (gfx950).

Thin ctypes marshalling over the C ABI in include/s2r.h -- the functions below carry the
same names as the C entry points, take torch tensors (device memory) and the current torch
stream, and do no arithmetic of their own.  Every step of the path runs in the HIP kernels
of libs2r.so; there is no CPU or PyTorch fallback: if the library is not built, importing
the binding's entry points raises.

The method is the data-parallel hot path of S2 Reducer (arXiv 2110.02140, Section 3.1 and
Algorithm 1): encode (bitmap + count-sketch per worker), reduce (sum of sketches, OR of
bitmaps) and decode (median over rows at every set bit).
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libs2r.so")
MAX_ROWS = 16

(S2R_OK, S2R_ERR_NULL, S2R_ERR_DIM, S2R_ERR_ALIGN, S2R_ERR_WORKSPACE, S2R_ERR_HIP,
 S2R_ERR_SCRATCH) = range(7)
NOALLOC_SCRATCH_BYTES = 256 << 20


class S2RError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class s2r_params(ctypes.Structure):
    """Mirror of ``s2r_params`` in include/s2r.h."""

    _fields_ = [
        ("d", ctypes.c_uint32),
        ("log2_w", ctypes.c_uint32),
        ("log2_part", ctypes.c_uint32),
        ("log2_block", ctypes.c_uint32),
        ("pA", ctypes.c_uint64),
        ("pB", ctypes.c_uint64),
        ("hA", ctypes.c_uint64 * MAX_ROWS),
        ("hB", ctypes.c_uint64 * MAX_ROWS),
        ("sA", ctypes.c_uint64 * MAX_ROWS),
        ("sB", ctypes.c_uint64 * MAX_ROWS),
    ]

    @property
    def w(self) -> int:
        return 1 << self.log2_w

    def as_dict(self) -> dict:
        d = self.d
        return {
            "d": d, "log2_w": self.log2_w, "log2_part": self.log2_part,
            "log2_block": self.log2_block, "pA": self.pA, "pB": self.pB,
            "hA": list(self.hA)[:d], "hB": list(self.hB)[:d],
            "sA": list(self.sA)[:d], "sB": list(self.sB)[:d],
        }


S2R_BF16, S2R_F16, S2R_F32 = range(3)
S2R_E4M3, S2R_E5M2 = range(2)
S2R_ACT_SILU, S2R_ACT_GELU, S2R_ACT_GELU_TANH = range(3)
_FORMATS = {"e4m3": S2R_E4M3, "e5m2": S2R_E5M2}
_ACTS = {"silu": S2R_ACT_SILU, "gelu": S2R_ACT_GELU, "gelu_tanh": S2R_ACT_GELU_TANH}


class s2r_mat(ctypes.Structure):
    """Mirror of ``s2r_mat`` in include/s2r_q8.h; made from a tensor by mat()."""

    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_uint64), ("dtype", ctypes.c_uint32)]


class s2r_q8_mat(ctypes.Structure):
    """Mirror of ``s2r_q8_mat`` in include/s2r_q8.h; made from tensors by q8_mat() or alloc_q8()."""

    _fields_ = [("q", ctypes.c_void_p), ("ld", ctypes.c_uint64), ("scale", ctypes.c_void_p),
                ("lds", ctypes.c_uint64), ("format", ctypes.c_uint32)]


class s2r_q4_mat(ctypes.Structure):
    """Mirror of ``s2r_q4_mat`` in include/s2r_q4.h; made from tensors by q4_mat() or alloc_q4()."""

    _fields_ = [("q", ctypes.c_void_p), ("ld", ctypes.c_uint64), ("scale", ctypes.c_void_p),
                ("lds", ctypes.c_uint64)]


class s2r_experts(ctypes.Structure):
    """Mirror of ``s2r_experts`` in include/s2r_moe.h; made from tensors by experts()."""

    _fields_ = [("first", ctypes.c_void_p), ("rows", ctypes.c_void_p), ("experts", ctypes.c_uint32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libs2r.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"libs2r.so not found at {LIB_PATH}: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        vp, u64, u32, sz = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_size_t
        st = ctypes.c_int
        L.s2r_params_from_seed.argtypes = [u64, u32, u32, u32, P(s2r_params)]
        L.s2r_params_from_seed.restype = st
        L.s2r_default_log2_part.argtypes = [u32, u32]
        L.s2r_default_log2_part.restype = u32
        L.s2r_sketch_lambda.argtypes = [u32, u32, u64, ctypes.c_int]
        L.s2r_sketch_lambda.restype = ctypes.c_double
        L.s2r_log2_w_for_lambda.argtypes = [u32, u64, ctypes.c_double, ctypes.c_int]
        L.s2r_log2_w_for_lambda.restype = u32
        L.s2r_bitmap_words.argtypes = [u64]
        L.s2r_bitmap_words.restype = u64
        L.s2r_block_bitmap_words.argtypes = [u64, u32]
        L.s2r_block_bitmap_words.restype = u64
        L.s2r_encode_workspace_bytes.argtypes = [P(s2r_params), u32, u64, u64]
        L.s2r_encode_workspace_bytes.restype = sz
        L.s2r_encode.argtypes = [P(s2r_params), u32, vp, u64, u64, vp, vp, vp, vp, u64, vp, vp, sz,
                                 vp]
        L.s2r_encode.restype = st
        L.s2r_encode_noalloc.argtypes = [P(s2r_params), u32, vp, u64, u64, vp, vp, vp, vp, u64,
                                         vp, vp]
        L.s2r_encode_noalloc.restype = st
        L.s2r_reduce.argtypes = [P(s2r_params), u32, u64, vp, vp, vp, vp, vp]
        L.s2r_reduce.restype = st
        L.s2r_decode_workspace_bytes.argtypes = [P(s2r_params), u64, u64]
        L.s2r_decode_workspace_bytes.restype = sz
        L.s2r_decode.argtypes = [P(s2r_params), u64, vp, vp, vp, u64, vp, sz, vp]
        L.s2r_decode.restype = st
        L.s2r_hash.argtypes = [P(s2r_params), vp, u64, vp, vp, vp]
        L.s2r_hash.restype = st
        L.s2r_gather_sum.argtypes = [u32, vp, vp, u64, vp, u64, vp, vp]
        L.s2r_gather_sum.restype = st
        L.s2r_diag_trace_attach.argtypes = [vp]
        L.s2r_diag_trace_attach.restype = st
        L.s2r_topk_workspace_bytes.argtypes = [u32, u64, u64]
        L.s2r_topk_workspace_bytes.restype = sz
        L.s2r_topk_ef.argtypes = [u32, vp, vp, u64, u64, u64, u64, vp, vp, vp, sz, vp]
        L.s2r_topk_ef.restype = st
        L.s2r_diag_stream_write.argtypes = [vp, sz, ctypes.c_float, vp]
        L.s2r_diag_stream_write.restype = st
        L.s2r_diag_stream_read.argtypes = [vp, sz, vp, vp]
        L.s2r_diag_stream_read.restype = st
        pm, pq = P(s2r_mat), P(s2r_q8_mat)
        L.s2r_q8_save.argtypes = [u64, u64, pm, pq, vp]
        L.s2r_q8_load.argtypes = [u64, u64, pq, pm, vp]
        L.s2r_q8_weight.argtypes = [u64, u64, pm, pq, pq, vp]
        L.s2r_q8_gemm_workspace_bytes.argtypes = [u64, u64, u64]
        L.s2r_q8_gemm_workspace_bytes.restype = sz
        L.s2r_q8_gemm.argtypes = [u64, u64, u64, pq, pq, pm, vp, sz, vp]
        L.s2r_q8_gemm_fast.argtypes = L.s2r_q8_gemm.argtypes
        L.s2r_q8_wgrad_workspace_bytes.argtypes = [u64, u64, u64]
        L.s2r_q8_wgrad_workspace_bytes.restype = sz
        L.s2r_q8_wgrad.argtypes = [u64, u64, u64, pm, pq, pq, vp, u64, ctypes.c_int, vp, sz, vp]
        L.s2r_q8_glu.argtypes = [u64, u64, ctypes.c_int, pm, pm, pq, pq, pm, pq, vp]
        L.s2r_q8_glu_grad.argtypes = [u64, u64, ctypes.c_int, pq, pq, pm, pm, pm, pq, pq, vp]
        for f in (L.s2r_q8_save, L.s2r_q8_load, L.s2r_q8_weight, L.s2r_q8_gemm, L.s2r_q8_gemm_fast,
                  L.s2r_q8_wgrad, L.s2r_q8_glu, L.s2r_q8_glu_grad):
            f.restype = st
        pe, p4, ci = P(s2r_experts), P(s2r_q4_mat), ctypes.c_int
        L.s2r_moe_rows.argtypes = [u64, u32, u32]
        L.s2r_moe_rows.restype = u64
        L.s2r_moe_route_workspace_bytes.argtypes = [u64, u32, u32]
        L.s2r_moe_route_workspace_bytes.restype = sz
        L.s2r_moe_route.argtypes = [u64, u32, u32, vp, vp, vp, vp, vp, sz, vp]
        L.s2r_moe_gather.argtypes = [u64, u32, u64, pm, vp, u64, pm, pq, vp]
        L.s2r_moe_combine.argtypes = [u64, u32, u64, pm, u64, vp, vp, pm, vp]
        L.s2r_moe_combine_grad.argtypes = [u64, u32, u64, pm, vp, u64, vp, pm, pm, pq, vp, vp]
        L.s2r_q8_gemm_experts.argtypes = [u64, u64, u64, pe, pq, pq, u64, u64, pm, vp]
        L.s2r_q8_wgrad_experts.argtypes = [u64, u64, u64, pe, pm, pq, pq, vp, u64, u64, ci, vp]
        L.s2r_q4_save.argtypes = [u64, u64, pm, p4, p4, vp]
        L.s2r_q4_load.argtypes = [u64, u64, p4, pm, vp]
        L.s2r_q4_gemm_workspace_bytes.argtypes = [u64, u64, u64]
        L.s2r_q4_gemm_workspace_bytes.restype = sz
        L.s2r_q4_gemm.argtypes = [u64, u64, u64, p4, p4, pm, vp, sz, vp]
        for f in (L.s2r_moe_route, L.s2r_moe_gather, L.s2r_moe_combine, L.s2r_moe_combine_grad,
                  L.s2r_q8_gemm_experts, L.s2r_q8_wgrad_experts, L.s2r_q4_save, L.s2r_q4_load,
                  L.s2r_q4_gemm):
            f.restype = st
        L.s2r_status_string.argtypes = [st]
        L.s2r_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().s2r_status_string(status).decode()


def _check(status: int, where: str) -> None:
    if status != S2R_OK:
        raise S2RError(status, where)


def _ptr(t) -> int | None:
    """Device pointer of a tensor (None for None), or an int passed through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    # the current stream's handle without a Stream object around it, which costs as much as a short call,
    # where this torch has such a call: it is none of its public ones
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream().cuda_stream if raw is None else raw(torch.cuda.current_device())


# ---------------------------------------------------------------------------------------
# entry points (same names as the C ABI)


def s2r_params_from_seed(seed: int, d: int, log2_w: int, log2_part: int | None = None,
                         log2_block: int = 0) -> s2r_params:
    """Hash constants from a seed (SplitMix64).  log2_part defaults to the largest partition
    that fits the LDS accumulator (s2r_default_log2_part); log2_part == log2_w gives
    independent rows.  log2_block sets the bitmap granularity (one bit per 2^log2_block
    elements; 0 = per element)."""
    if log2_part is None:
        log2_part = s2r_default_log2_part(d, log2_w)
    p = s2r_params()
    _check(lib().s2r_params_from_seed(seed, d, log2_w, log2_part, ctypes.byref(p)),
           "s2r_params_from_seed")
    p.log2_block = log2_block
    return p


def s2r_default_log2_part(d: int, log2_w: int) -> int:
    return int(lib().s2r_default_log2_part(d, log2_w))


def s2r_sketch_lambda(rows: int, log2_w: int, nnz: int, per_row: bool = False) -> float:
    """Sketch size over the non-zero count: rows * 2^log2_w / nnz, or 2^log2_w / nnz with
    per_row (see include/s2r.h)."""
    return float(lib().s2r_sketch_lambda(rows, log2_w, nnz, 1 if per_row else 0))


def s2r_log2_w_for_lambda(rows: int, nnz: int, lam: float, per_row: bool = False) -> int:
    """Smallest log2_w reaching the ratio `lam`; 2^32 - 1 when none can."""
    return int(lib().s2r_log2_w_for_lambda(rows, nnz, lam, 1 if per_row else 0))


def s2r_bitmap_words(n: int) -> int:
    return int(lib().s2r_bitmap_words(n))


def s2r_block_bitmap_words(n: int, log2_block: int) -> int:
    return int(lib().s2r_block_bitmap_words(n, log2_block))


def s2r_encode_workspace_bytes(p: s2r_params, W: int, n: int, cap: int) -> int:
    return int(lib().s2r_encode_workspace_bytes(ctypes.byref(p), W, n, cap))


def s2r_encode(p: s2r_params, W: int, grad, n: int, ld: int, bitmaps, sketches, idx, val, cap: int,
               nnz, workspace, ws_bytes: int | None = None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().s2r_encode(ctypes.byref(p), W, _ptr(grad), n, ld, _ptr(bitmaps), _ptr(sketches),
                            _ptr(idx), _ptr(val), cap, _ptr(nnz), _ptr(workspace), ws_bytes,
                            _stream(stream)), "s2r_encode")


def s2r_encode_noalloc(p: s2r_params, W: int, grad, n: int, ld: int, bitmaps, sketches, idx, val,
                       cap: int, nnz, stream=None) -> None:
    """s2r_encode with the library's static scratch as its workspace (allocates nothing)."""
    _check(lib().s2r_encode_noalloc(ctypes.byref(p), W, _ptr(grad), n, ld, _ptr(bitmaps),
                                    _ptr(sketches), _ptr(idx), _ptr(val), cap, _ptr(nnz),
                                    _stream(stream)), "s2r_encode_noalloc")


def s2r_reduce(p: s2r_params, W: int, n: int, bitmaps, sketches, bitmap_out, sketch_out,
               stream=None) -> None:
    _check(lib().s2r_reduce(ctypes.byref(p), W, n, _ptr(bitmaps), _ptr(sketches), _ptr(bitmap_out),
                            _ptr(sketch_out), _stream(stream)), "s2r_reduce")


def s2r_decode_workspace_bytes(p: s2r_params, n: int, max_set: int) -> int:
    return int(lib().s2r_decode_workspace_bytes(ctypes.byref(p), n, max_set))


def s2r_decode(p: s2r_params, n: int, bitmap, sketch, out, max_set: int = 0, workspace=None,
               ws_bytes: int | None = None, stream=None) -> None:
    """workspace=None selects direct gathers; otherwise pass a buffer of
    s2r_decode_workspace_bytes(p, n, max_set) bytes (see include/s2r.h)."""
    if ws_bytes is None:
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().s2r_decode(ctypes.byref(p), n, _ptr(bitmap), _ptr(sketch), _ptr(out), max_set,
                            _ptr(workspace), ws_bytes, _stream(stream)), "s2r_decode")


def s2r_hash(p: s2r_params, keys, m: int, buckets, signs, stream=None) -> None:
    _check(lib().s2r_hash(ctypes.byref(p), _ptr(keys), m, _ptr(buckets), _ptr(signs),
                          _stream(stream)), "s2r_hash")


def s2r_gather_sum(W: int, idx, val, cap: int, nnz, n: int, out, stream=None) -> None:
    """Exact sum of the workers' (index, value) lists into dense out[n] (worker order)."""
    _check(lib().s2r_gather_sum(W, _ptr(idx), _ptr(val), cap, _ptr(nnz), n, _ptr(out),
                                _stream(stream)), "s2r_gather_sum")


def s2r_topk_workspace_bytes(W: int, n: int, block: int) -> int:
    return int(lib().s2r_topk_workspace_bytes(W, n, block))


def s2r_topk_ef(W: int, grad, residual, n: int, ld: int, block: int, K: int, out, selected,
                workspace, ws_bytes: int | None = None, stream=None) -> None:
    """Block-wise Top-K with error feedback (residual may be None: no error feedback;
    selected may be None)."""
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().s2r_topk_ef(W, _ptr(grad), _ptr(residual), n, ld, block, K, _ptr(out),
                             _ptr(selected), _ptr(workspace), ws_bytes, _stream(stream)),
           "s2r_topk_ef")


# ---------------------------------------------------------------------------------------
# training in 8 bits (include/s2r_q8.h)


def mat(t) -> s2r_mat:
    """Descriptor of a 2-D bf16, fp16 or fp32 tensor with unit stride along its rows; keeps
    the tensor alive."""
    import torch
    codes = {torch.bfloat16: S2R_BF16, torch.float16: S2R_F16, torch.float32: S2R_F32}
    if t.dim() != 2 or t.dtype not in codes or (t.shape[1] > 1 and t.stride(1) != 1):
        raise S2RError(S2R_ERR_DIM, "mat")
    ld = max(t.stride(0), t.shape[1]) if t.shape[0] <= 1 else t.stride(0)
    m = s2r_mat(t.data_ptr(), ld, codes[t.dtype])
    m.tensor = t
    return m


def q8_mat(q, scale, fmt: str = "e4m3") -> s2r_q8_mat:
    """Descriptor of an 8-bit matrix: q [rows][ld] and scale [ceil(cols / 128)][lds], one byte
    each, in format "e4m3" or "e5m2"; keeps the tensors alive."""
    for t in (q, scale):
        if t.dim() != 2 or t.element_size() != 1 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise S2RError(S2R_ERR_DIM, "q8_mat")
    if fmt not in _FORMATS:
        raise S2RError(S2R_ERR_DIM, "q8_mat")
    ld, lds = (max(t.stride(0), t.shape[1]) if t.shape[0] <= 1 else t.stride(0) for t in (q, scale))
    m = s2r_q8_mat(q.data_ptr(), ld, scale.data_ptr(), lds, _FORMATS[fmt])
    m.codes, m.scales = q, scale
    return m


def alloc_q8(rows: int, cols: int, fmt: str = "e4m3", square: bool = False,
             device="cuda") -> s2r_q8_mat:
    """An 8-bit matrix on new tensors (.codes, .scales), row blocks or with `square` 128 x 128
    blocks, padded as the calls need it."""
    import torch
    up = lambda n, m: -(-n // m) * m
    sr = up(rows, 128) // 128 if square else rows
    return q8_mat(torch.empty((rows, up(max(cols, 1), 16)), dtype=torch.uint8, device=device),
                  torch.empty((up(cols, 128) // 128, up(max(sr, 1), 4)), dtype=torch.uint8,
                              device=device), fmt)


def _ref(m):
    return None if m is None else ctypes.byref(m)


def _ws(workspace, ws_bytes):
    if ws_bytes is None:
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _ptr(workspace), ws_bytes


def _act(act) -> int:
    return _ACTS.get(act, -1) if isinstance(act, str) else act


def s2r_q8_save(M: int, K: int, x: s2r_mat, out: s2r_q8_mat, stream=None) -> None:
    """x [M][K] to 8 bits, one scale per 128 elements of a row."""
    _check(lib().s2r_q8_save(M, K, _ref(x), _ref(out), _stream(stream)), "s2r_q8_save")


def s2r_q8_load(M: int, K: int, q: s2r_q8_mat, x: s2r_mat, stream=None) -> None:
    """The stored values of q [M][K] into x."""
    _check(lib().s2r_q8_load(M, K, _ref(q), _ref(x), _stream(stream)), "s2r_q8_load")


def s2r_q8_weight(N: int, K: int, w: s2r_mat, out: s2r_q8_mat, out_t: s2r_q8_mat | None = None,
                  stream=None) -> None:
    """w [N][K] to 8 bits, one scale per 128 x 128 block, and its transpose into out_t."""
    _check(lib().s2r_q8_weight(N, K, _ref(w), _ref(out), _ref(out_t), _stream(stream)),
           "s2r_q8_weight")


def s2r_q8_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().s2r_q8_gemm_workspace_bytes(M, N, K))


def s2r_q8_gemm(M: int, N: int, K: int, a: s2r_q8_mat, b: s2r_q8_mat, c: s2r_mat, workspace=None,
                ws_bytes: int | None = None, stream=None) -> None:
    """c [M][N] = a [M][K] b [N][K]^T (a in row blocks, b in square blocks)."""
    ws, nb = _ws(workspace, ws_bytes)
    _check(lib().s2r_q8_gemm(M, N, K, _ref(a), _ref(b), _ref(c), ws, nb, _stream(stream)),
           "s2r_q8_gemm")


def s2r_q8_gemm_fast(M: int, N: int, K: int, a: s2r_q8_mat, b: s2r_q8_mat, c: s2r_mat, workspace=None,
                     ws_bytes: int | None = None, stream=None) -> None:
    """s2r_q8_gemm through the 8-bit matrix instruction: faster, with products cut short (the bound
    is in include/s2r_q8.h)."""
    ws, nb = _ws(workspace, ws_bytes)
    _check(lib().s2r_q8_gemm_fast(M, N, K, _ref(a), _ref(b), _ref(c), ws, nb, _stream(stream)),
           "s2r_q8_gemm_fast")


def s2r_q8_wgrad_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().s2r_q8_wgrad_workspace_bytes(M, N, K))


def s2r_q8_wgrad(M: int, N: int, K: int, dy, x: s2r_q8_mat, dw, lddw: int,
                 accumulate: bool = False, workspace=None, ws_bytes: int | None = None,
                 stream=None) -> None:
    """dw [N][lddw] (+)= dy^T x, dy a bf16 s2r_mat or an s2r_q8_mat; dw fp32, a tensor or an
    address within a worker's gradient row."""
    ws, nb = _ws(workspace, ws_bytes)
    wide = isinstance(dy, s2r_mat)
    _check(lib().s2r_q8_wgrad(M, N, K, _ref(dy) if wide else None, None if wide else _ref(dy),
                              _ref(x), _ptr(dw), lddw, 1 if accumulate else 0, ws, nb,
                              _stream(stream)), "s2r_q8_wgrad")


def s2r_q8_glu(M: int, F: int, act, g: s2r_mat, u: s2r_mat | None = None,
               gq: s2r_q8_mat | None = None, uq: s2r_q8_mat | None = None,
               y: s2r_mat | None = None, yq: s2r_q8_mat | None = None, stream=None) -> None:
    """act(g) * u, or act(g) without u; act is "silu", "gelu" or "gelu_tanh"."""
    _check(lib().s2r_q8_glu(M, F, _act(act), _ref(g), _ref(u), _ref(gq), _ref(uq), _ref(y),
                            _ref(yq), _stream(stream)), "s2r_q8_glu")


def s2r_q8_glu_grad(M: int, F: int, act, gq: s2r_q8_mat, uq: s2r_q8_mat | None, dy: s2r_mat,
                    dg: s2r_mat | None = None, du: s2r_mat | None = None,
                    dgq: s2r_q8_mat | None = None, duq: s2r_q8_mat | None = None,
                    stream=None) -> None:
    """The gradients of s2r_q8_glu's g and u from their checkpoints."""
    _check(lib().s2r_q8_glu_grad(M, F, _act(act), _ref(gq), _ref(uq), _ref(dy), _ref(dg), _ref(du),
                                 _ref(dgq), _ref(duq), _stream(stream)), "s2r_q8_glu_grad")


# ---------------------------------------------------------------------------------------
# layers of experts (include/s2r_moe.h)


_DTYPES: dict = {}  # torch's types by name, once torch is there


def _dense(t, shape: tuple, kind: str, where: str):
    """Device pointer of a dense tensor of `shape` and of the types "ints" or "floats" (None and
    addresses pass through)."""
    if t is None or type(t) is int:
        return t
    if not _DTYPES:
        import torch
        _DTYPES.update(ints=(torch.int32, torch.uint32), floats=(torch.float32,))
    if t.dtype not in _DTYPES[kind] or t.shape != shape or not t.is_contiguous():
        raise S2RError(S2R_ERR_DIM, where)
    return t.data_ptr()


def _ints(t, shape: tuple, where: str):
    return _dense(t, shape, "ints", where)


def _floats(t, shape: tuple, where: str):
    return _dense(t, shape, "floats", where)


def experts(first, rows) -> s2r_experts:
    """Descriptor of the experts' rows, two int32 tensors [E]; keeps them alive.  Every element of `first` is a
    multiple of 4: nothing on the host can see whether it is, and scales of other rows may be taken where it is not."""
    E = rows.numel()
    e = s2r_experts(_ints(first, (E,), "experts"), _ints(rows, (E,), "experts"), E)
    e.tensors = first, rows
    return e


def s2r_moe_rows(T: int, K: int, E: int) -> int:
    """Rows that always hold the K choices of T tokens among E experts."""
    return int(lib().s2r_moe_rows(T, K, E))


def s2r_moe_route_workspace_bytes(T: int, K: int, E: int) -> int:
    return int(lib().s2r_moe_route_workspace_bytes(T, K, E))


def s2r_moe_route(T: int, K: int, E: int, expert, first, rows, place, workspace=None,
                  ws_bytes: int | None = None, stream=None) -> None:
    """expert [T][K] -> first [E] and rows [E] of every expert, place [T][K] of every choice
    (int32, dense; -1: none)."""
    w = "s2r_moe_route"
    ws, nb = _ws(workspace, ws_bytes)
    _check(lib().s2r_moe_route(T, K, E, _ints(expert, (T, K), w), _ints(first, (E,), w), _ints(rows, (E,), w),
                               _ints(place, (T, K), w), ws, nb, _stream(stream)), w)


def s2r_moe_gather(T: int, K: int, D: int, x: s2r_mat, place, R: int, out: s2r_mat | None = None,
                   outq: s2r_q8_mat | None = None, stream=None) -> None:
    """Every token of x [T][D] to its choices' rows of out and, in 8 bits, of outq [R][D]."""
    w = "s2r_moe_gather"
    _check(lib().s2r_moe_gather(T, K, D, _ref(x), _ints(place, (T, K), w), R, _ref(out), _ref(outq),
                                _stream(stream)), w)


def s2r_moe_combine(T: int, K: int, D: int, rows: s2r_mat, R: int, place, weight, y: s2r_mat,
                    stream=None) -> None:
    """y [T][D] = the sum of every token's rows of rows [R][D], with weight [T][K] (None: ones)."""
    w = "s2r_moe_combine"
    _check(lib().s2r_moe_combine(T, K, D, _ref(rows), R, _ints(place, (T, K), w), _floats(weight, (T, K), w),
                                 _ref(y), _stream(stream)), w)


def s2r_moe_combine_grad(T: int, K: int, D: int, dy: s2r_mat, place, R: int, weight=None,
                         rows: s2r_mat | None = None, drows: s2r_mat | None = None,
                         drowsq: s2r_q8_mat | None = None, dweight=None, stream=None) -> None:
    """The gradients of s2r_moe_combine's rows (drows, and drowsq in 8 bits) and weights (dweight
    [T][K], from rows)."""
    w = "s2r_moe_combine_grad"
    _check(lib().s2r_moe_combine_grad(T, K, D, _ref(dy), _ints(place, (T, K), w), R, _floats(weight, (T, K), w),
                                      _ref(rows), _ref(drows), _ref(drowsq), _floats(dweight, (T, K), w),
                                      _stream(stream)), w)


def s2r_q8_gemm_experts(M: int, N: int, K: int, e: s2r_experts, a: s2r_q8_mat, b: s2r_q8_mat, b_step: int,
                        b_scale_step: int, c: s2r_mat, stream=None) -> None:
    """c = a b_e^T for the rows of every expert; b is expert 0's [N][K], expert e's is e * b_step and
    e * b_scale_step bytes further on."""
    _check(lib().s2r_q8_gemm_experts(M, N, K, _ref(e), _ref(a), _ref(b), b_step, b_scale_step, _ref(c),
                                     _stream(stream)), "s2r_q8_gemm_experts")


def s2r_q8_wgrad_experts(M: int, N: int, K: int, e: s2r_experts, dy, x: s2r_q8_mat, dw, lddw: int, dw_step: int,
                         accumulate: bool = False, stream=None) -> None:
    """dw + e * dw_step [N][lddw] (+)= dy^T x over the rows of every expert e, as s2r_q8_wgrad."""
    wide = isinstance(dy, s2r_mat)
    _check(lib().s2r_q8_wgrad_experts(M, N, K, _ref(e), _ref(dy) if wide else None, None if wide else _ref(dy),
                                      _ref(x), _ptr(dw), lddw, dw_step, 1 if accumulate else 0,
                                      _stream(stream)), "s2r_q8_wgrad_experts")


# ---------------------------------------------------------------------------------------
# matrices in 4 bits (include/s2r_q4.h)


def q4_mat(q, scale) -> s2r_q4_mat:
    """Descriptor of a 4-bit matrix: q [rows][ld] bytes of two codes and scale [rows][lds] bytes; keeps
    the tensors alive."""
    for t in (q, scale):
        if t.dim() != 2 or t.element_size() != 1 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise S2RError(S2R_ERR_DIM, "q4_mat")
    ld, lds = (max(t.stride(0), t.shape[1]) if t.shape[0] <= 1 else t.stride(0) for t in (q, scale))
    m = s2r_q4_mat(q.data_ptr(), ld, scale.data_ptr(), lds)
    m.codes, m.scales = q, scale
    return m


def alloc_q4(rows: int, cols: int, device="cuda") -> s2r_q4_mat:
    """A 4-bit matrix on new tensors (.codes, .scales), padded as the calls need it."""
    import torch
    up = lambda n, m: -(-n // m) * m
    return q4_mat(torch.empty((rows, up(max(cols, 1), 32) // 2), dtype=torch.uint8, device=device),
                  torch.empty((rows, up(max(cols, 1), 256) // 32), dtype=torch.uint8, device=device))


def s2r_q4_save(R: int, C: int, x: s2r_mat, out: s2r_q4_mat | None = None, out_t: s2r_q4_mat | None = None,
                stream=None) -> None:
    """x [R][C] to 4 bits, and its transpose [C][R], one scale per 32 elements of their rows."""
    _check(lib().s2r_q4_save(R, C, _ref(x), _ref(out), _ref(out_t), _stream(stream)), "s2r_q4_save")


def s2r_q4_load(R: int, C: int, q: s2r_q4_mat, x: s2r_mat, stream=None) -> None:
    """The stored values of q [R][C] into x."""
    _check(lib().s2r_q4_load(R, C, _ref(q), _ref(x), _stream(stream)), "s2r_q4_load")


def s2r_q4_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().s2r_q4_gemm_workspace_bytes(M, N, K))


def s2r_q4_gemm(M: int, N: int, K: int, a: s2r_q4_mat, b: s2r_q4_mat, c: s2r_mat, workspace=None,
                ws_bytes: int | None = None, stream=None) -> None:
    """c [M][N] = a [M][K] b [N][K]^T."""
    ws, nb = _ws(workspace, ws_bytes)
    _check(lib().s2r_q4_gemm(M, N, K, _ref(a), _ref(b), _ref(c), ws, nb, _stream(stream)), "s2r_q4_gemm")


TRACE_MAX = 64


class s2r_trace(ctypes.Structure):
    """Mirror of ``s2r_trace`` in include/s2r_diag.h."""

    _fields_ = [
        ("capacity", ctypes.c_uint32),
        ("count", ctypes.c_uint32),
        ("events", ctypes.c_void_p * TRACE_MAX),
        ("names", ctypes.c_char_p * TRACE_MAX),
    ]


def s2r_diag_trace_attach(trace) -> None:
    """Attach an s2r_trace (or None to detach) to the calling thread (include/s2r_diag.h)."""
    _check(lib().s2r_diag_trace_attach(None if trace is None else ctypes.addressof(trace)),
           "s2r_diag_trace_attach")


def s2r_diag_stream_write(buf, nbytes: int, value: float = 0.0, stream=None) -> None:
    """Measurement helper (include/s2r_diag.h): fill `nbytes` of `buf` with `value` once."""
    _check(lib().s2r_diag_stream_write(_ptr(buf), nbytes, value, _stream(stream)),
           "s2r_diag_stream_write")


def s2r_diag_stream_read(buf, nbytes: int, sink, stream=None) -> None:
    """Measurement helper (include/s2r_diag.h): stream `nbytes` of `buf` once."""
    _check(lib().s2r_diag_stream_read(_ptr(buf), nbytes, _ptr(sink), _stream(stream)),
           "s2r_diag_stream_read")


# ---------------------------------------------------------------------------------------
# allocation helper (torch supplies device memory; no arithmetic here)


def alloc_decode_workspace(p: s2r_params, n: int, max_set: int, device="cuda"):
    """A workspace tensor for the partitioned decode, or None when it does not apply."""
    import torch
    nb = s2r_decode_workspace_bytes(p, n, max_set)
    return torch.empty((nb,), dtype=torch.uint8, device=device) if nb else None


def alloc_encode_buffers(p: s2r_params, W: int, n: int, cap: int, device="cuda") -> dict:
    """torch tensors for every s2r_encode output plus its workspace."""
    import torch
    words = s2r_block_bitmap_words(n, p.log2_block)
    ws = s2r_encode_workspace_bytes(p, W, n, cap)
    if ws == 0:
        raise S2RError(S2R_ERR_DIM, "s2r_encode_workspace_bytes")
    return {
        "bitmaps": torch.empty((W, max(words, 1)), dtype=torch.int64, device=device),
        "sketches": torch.empty((W, p.d, p.w), dtype=torch.float32, device=device),
        "idx": torch.empty((W, max(cap, 1)), dtype=torch.int32, device=device),
        "val": torch.empty((W, max(cap, 1)), dtype=torch.float32, device=device),
        "nnz": torch.empty((W,), dtype=torch.int64, device=device),
        "workspace": torch.empty((ws,), dtype=torch.uint8, device=device),
    }


__all__ = [
    "s2r_params", "S2RError", "s2r_params_from_seed", "s2r_default_log2_part", "s2r_bitmap_words",
    "s2r_sketch_lambda", "s2r_log2_w_for_lambda",
    "s2r_block_bitmap_words",
    "s2r_encode_workspace_bytes", "s2r_encode", "s2r_encode_noalloc", "s2r_reduce", "s2r_decode_workspace_bytes",
    "s2r_decode", "s2r_hash", "s2r_gather_sum", "s2r_topk_workspace_bytes", "s2r_topk_ef",
    "s2r_mat", "s2r_q8_mat", "mat", "q8_mat", "alloc_q8", "s2r_q8_save", "s2r_q8_load",
    "s2r_q8_weight", "s2r_q8_gemm_workspace_bytes", "s2r_q8_gemm", "s2r_q8_gemm_fast",
    "s2r_q8_wgrad_workspace_bytes", "s2r_q8_wgrad", "s2r_q8_glu", "s2r_q8_glu_grad",
    "s2r_experts", "experts", "s2r_moe_rows", "s2r_moe_route_workspace_bytes", "s2r_moe_route", "s2r_moe_gather",
    "s2r_moe_combine", "s2r_moe_combine_grad", "s2r_q8_gemm_experts", "s2r_q8_wgrad_experts",
    "s2r_q4_mat", "q4_mat", "alloc_q4", "s2r_q4_save", "s2r_q4_load", "s2r_q4_gemm_workspace_bytes", "s2r_q4_gemm",
    "s2r_trace", "s2r_diag_trace_attach",
    "alloc_encode_buffers", "status_string", "lib",
]
