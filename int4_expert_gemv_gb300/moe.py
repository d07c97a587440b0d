"""Thin Python binding of the C ABI in include/moe.h (ctypes).

Argument marshalling only: every function forwards device pointers, sizes and
the current CUDA stream to libmoe.so, which does all of the work.  Tensors are
PyTorch CUDA tensors (PyTorch supplies device memory and streams); raw integer
pointers are accepted wherever a tensor is.  A non-zero status raises
MoEError.  There is no fallback: if libmoe.so is missing the import of the
library fails loudly.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_ECUDA, MOE_ETIMEOUT, MOE_ENOSPACE = range(6)
MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_E4M3 = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_ROTARY_HALF, MOE_ROTARY_INTERLEAVED = 0, 1
MOE_ROTARY_PLAIN, MOE_ROTARY_LINEAR, MOE_ROTARY_BASE, MOE_ROTARY_YARN, MOE_ROTARY_BANDS = range(5)
MOE_PREC_AFFINE4, MOE_PREC_FP16 = 4, 16

_lock = threading.Lock()
_lib = None


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {status_string(status)}: {detail}")
        self.status = status


# ------------------------------------------------------------------ structs
class HeadDesc(C.Structure):
    _fields_ = [("d", C.c_int), ("E", C.c_int), ("H", C.c_int), ("prec", C.c_int),
                ("fc1x", C.c_void_p), ("fc1_tab", C.c_void_p), ("b1", C.c_void_p),
                ("fc2", C.c_void_p), ("b2", C.c_void_p),
                ("lx", C.c_void_p), ("l_tab", C.c_void_p), ("bl", C.c_void_p)]


class LoraDesc(C.Structure):
    _fields_ = [("r", C.c_int), ("scale", C.c_float), ("A", C.c_void_p), ("B", C.c_void_p),
                ("a_stride", C.c_size_t), ("b_stride", C.c_size_t)]


class ExpertsDesc(C.Structure):
    _fields_ = [("d", C.c_int), ("F", C.c_int), ("E", C.c_int), ("bits", C.c_int),
                ("pool", C.c_void_p), ("expert_stride", C.c_size_t), ("shared", C.c_void_p),
                ("lora", LoraDesc * 3), ("shared_lora", LoraDesc * 3)]


class StackDesc(C.Structure):
    _fields_ = [("experts", C.c_void_p), ("routers", C.c_void_p), ("heads", C.c_void_p),
                ("n_layers", C.c_int), ("depth", C.c_int), ("K", C.c_int),
                ("self_predict", C.c_int), ("timeout_ns", C.c_ulonglong),
                ("debug_unset_wait", C.c_int), ("debug_trace", C.c_void_p),
                ("inflight_bytes", C.c_uint), ("slot_map", C.c_void_p),
                ("layer_ready", C.c_void_p), ("free_sms", C.c_int)]


class ChainInfo(C.Structure):
    _fields_ = [("smem_a", C.c_size_t), ("smem_b", C.c_size_t), ("threads", C.c_int),
                ("regs_a", C.c_int), ("regs_b", C.c_int),
                ("local_bytes_a", C.c_int), ("local_bytes_b", C.c_int),
                ("ctas_a", C.c_int), ("ctas_b", C.c_int), ("coresident", C.c_int)]


class RouteDesc(C.Structure):
    _fields_ = [("E", C.c_int), ("K", C.c_int), ("score", C.c_int), ("n_group", C.c_int),
                ("keep_group", C.c_int), ("group_best", C.c_int), ("renorm", C.c_int),
                ("factor", C.c_float), ("bias", C.c_void_p)]


class KVDesc(C.Structure):
    _fields_ = [("n_pages", C.c_int), ("page", C.c_int), ("Hkv", C.c_int), ("D", C.c_int),
                ("dtype", C.c_int), ("k", C.c_void_p), ("v", C.c_void_p),
                ("page_stride", C.c_size_t), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p)]


class NormDesc(C.Structure):
    _fields_ = [("d", C.c_int), ("eps", C.c_float), ("weight", C.c_void_p), ("w_dtype", C.c_int),
                ("pow2", C.c_int)]


class ScaledMatrixDesc(C.Structure):
    _fields_ = [("N", C.c_int), ("K", C.c_int), ("w", C.c_void_p), ("w_stride", C.c_size_t),
                ("scales", C.c_void_p), ("scale_stride", C.c_size_t)]


class RotaryDesc(C.Structure):
    _fields_ = [("D", C.c_int), ("rot", C.c_int), ("first", C.c_int), ("layout", C.c_int),
                ("scaling", C.c_int), ("trained", C.c_int), ("base", C.c_double),
                ("factor", C.c_double), ("low", C.c_double), ("high", C.c_double),
                ("amplitude", C.c_float)]


# ------------------------------------------------------------------ loading
def lib():
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is missing: build it with "
                                  "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = C.CDLL(LIB_PATH)
            P, I, S = C.c_void_p, C.c_int, C.c_size_t
            sigs = {
                "moe_status_string": (C.c_char_p, [I]),
                "moe_last_error": (C.c_char_p, []),
                "moe_record_bytes": (S, [I, I]),
                "moe_packed_matrix_bytes": (S, [I, I, I]),
                "moe_pool_expert_bytes": (S, [I, I, I, I]),
                "moe_pack_matrix": (I, [P, P, P, I, I, I, P, P]),
                "moe_merge_lora": (I, [P, S, I, I, I, P, P, I, C.c_float, P, S, P]),
                "moe_gather_experts": (I, [P, S, I, P, I, S, P, S, P, P]),
                "moe_cache_experts": (I, [P, S, I, P, I, S, P, S, I, P, P, P, P, P, P, P]),
                "moe_pack_experts": (I, [I, I, I, I, P, P, P, P, P, P, P, P, P, P, S, P]),
                "moe_debug_dequant": (I, [P, I, I, I, I, P, P]),
                "moe_debug_batched_waits": (I, [C.c_ulonglong, I]),
                "moe_debug_batched_engine": (I, [I]),
                "moe_debug_batched_trace": (I, [P]),
                "moe_prerouter_head_workspace_bytes": (S, [C.POINTER(HeadDesc), I]),
                "moe_prerouter_head": (I, [C.POINTER(HeadDesc), P, I, P, P, I, I, P, P, S, P]),
                "moe_topk_route": (I, [P, I, I, I, P, P, P, P]),
                "moe_scored_route": (I, [C.POINTER(RouteDesc), P, I, S, I, P, P, P]),
                "moe_kv_plan": (I, [P, P, I, P, I, I, P, I, P, P, P, P, P, I, P, P, P]),
                "moe_kv_append": (I, [C.POINTER(KVDesc), P, S, P, S, I, P, I, P]),
                "moe_paged_attention_workspace_bytes": (S, [C.POINTER(KVDesc), I, I]),
                "moe_paged_attention": (I, [C.POINTER(KVDesc), P, I, S, I, I, P, P, I, C.c_float, I,
                                            P, S, P, P, S, P]),
                "moe_quantise_e4m3": (I, [P, I, S, I, I, I, I, P, S, P, S, P]),
                "moe_add_rms_norm": (I, [C.POINTER(NormDesc), P, I, S, P, I, S, I, P, S, P, I, S,
                                         P, S, P]),
                "moe_scaled_product_workspace_bytes": (S, [C.POINTER(ScaledMatrixDesc), I]),
                "moe_scaled_product": (I, [C.POINTER(ScaledMatrixDesc), P, S, P, S, I, P, I, S, P,
                                           S, P]),
                "moe_rotary_table": (I, [C.POINTER(RotaryDesc), P, P]),
                "moe_rotary": (I, [C.POINTER(RotaryDesc), P, P, I, I, P, S, I, P, S, P, S, I, P, S,
                                   P]),
                "moe_expert_ffn_workspace_bytes": (S, [C.POINTER(ExpertsDesc), I, I]),
                "moe_expert_ffn_int4": (I, [C.POINTER(ExpertsDesc), P, I, P, I, I, P, P, S, P]),
                "moe_combine_residual": (I, [P, P, I, I, I, I, P, P, P, P]),
                "moe_expert_ffn_int4_noalloc": (I, [C.POINTER(ExpertsDesc), P, I, P, I, I, P, P]),
                "moe_expert_ffn_noalloc_status": (I, [C.POINTER(C.c_int), P]),
                "moe_decode_step_workspace_bytes": (S, [C.POINTER(StackDesc)]),
                "moe_decode_step": (I, [C.POINTER(StackDesc), P, P, P, P, P, I, P, S, P]),
                "moe_decode_step_status": (I, [P, C.POINTER(C.c_int), P]),
                "moe_decode_step_chain_workspace_bytes": (S, [C.POINTER(StackDesc)]),
                "moe_decode_step_chain": (I, [C.POINTER(StackDesc), P, P, P, P, P, I, P, S, P]),
                "moe_decode_step_chain_info": (I, [C.POINTER(StackDesc), C.POINTER(ChainInfo)]),
                "moe_decode_step_chain_variant": (I, [I, I]),
                "moe_decode_step_chain_cache": (I, [I]),
            }
            for name, (res, args) in sigs.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def last_error() -> str:
    return lib().moe_last_error().decode()


def _ptr(t):
    try:
        return t.data_ptr()
    except AttributeError:
        if t is None or isinstance(t, int):      # an address
            return t
        raise


_current = None


def _stream(stream):
    if stream is None:
        # torch.cuda.current_stream() without making a Stream object (2.9 us
        # a call on the GPU's host, against 0.2)
        global _current
        if _current is None:
            import torch
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            device = getattr(torch._C, "_cuda_getDevice", None)
            if raw and device and torch.cuda.is_initialized():
                _current = lambda: raw(device())  # noqa: E731
            else:
                return torch.cuda.current_stream().cuda_stream
        return _current()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoEError(rc, where, last_error())


def _nbytes(t):
    return 0 if t is None else (t.numel() * t.element_size() if not isinstance(t, int) else 0)


_dtypes = None


def _dtype_code(x) -> int:
    global _dtypes
    if _dtypes is None:
        import torch
        _dtypes = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16}
    try:
        return _dtypes[x.dtype]
    except KeyError:
        raise TypeError(f"activations must be float32 or bfloat16, got {x.dtype}") from None


# ------------------------------------------------------------------ sizes
def moe_record_bytes(cols: int, bits: int) -> int:
    return lib().moe_record_bytes(cols, bits)


def moe_packed_matrix_bytes(rows: int, cols: int, bits: int) -> int:
    return lib().moe_packed_matrix_bytes(rows, cols, bits)


def moe_pool_expert_bytes(d: int, F: int, bits: int, group: int = 64) -> int:
    return lib().moe_pool_expert_bytes(d, F, bits, group)


def moe_prerouter_head_workspace_bytes(hd: HeadDesc, T: int) -> int:
    return lib().moe_prerouter_head_workspace_bytes(C.byref(hd), T)


def moe_expert_ffn_workspace_bytes(ed: ExpertsDesc, T: int, K: int) -> int:
    return lib().moe_expert_ffn_workspace_bytes(C.byref(ed), T, K)


# ------------------------------------------------------------------ calls
def moe_pack_matrix(q, s, b, rows: int, cols: int, bits: int, out, stream=None):
    _check(lib().moe_pack_matrix(_ptr(q), _ptr(s), _ptr(b), rows, cols, bits, _ptr(out),
                                 _stream(stream)), "moe_pack_matrix")


def moe_merge_lora(src, src_stride: int, rows: int, cols: int, bits: int, A, B, r: int,
                   scale: float, dst, dst_stride: int, stream=None):
    """W' = requantise(W + scale B A) on packed records (see include/moe.h).
    src / dst: tensors or device addresses (ints) of the first record."""
    _check(lib().moe_merge_lora(_ptr(src), src_stride, rows, cols, bits, _ptr(A), _ptr(B), r,
                                scale, _ptr(dst), dst_stride, _stream(stream)), "moe_merge_lora")


def moe_gather_experts(pool, expert_stride: int, E: int, idx, n: int, blob_bytes: int, slots,
                       slot_stride: int, slot_idx, stream=None):
    """Routed experts' blobs from a pool (HBM or pinned host memory) into HBM
    slots, route rewritten to the slots (see include/moe.h)."""
    _check(lib().moe_gather_experts(_ptr(pool), expert_stride, E, _ptr(idx), n, blob_bytes,
                                    _ptr(slots), slot_stride, _ptr(slot_idx), _stream(stream)),
           "moe_gather_experts")


def moe_cache_experts(pool, expert_stride: int, E: int, idx, n: int, blob_bytes: int, cache,
                      slot_stride: int, C: int, tags, ages, clock, slot_idx, plan, stats=None,
                      stream=None):
    """Route idx's experts through an HBM cache of C slots (LRU); slot_idx
    receives each entry's slot (the chain's slot map)."""
    _check(lib().moe_cache_experts(_ptr(pool), expert_stride, E, _ptr(idx), n, blob_bytes,
                                   _ptr(cache), slot_stride, C, _ptr(tags), _ptr(ages), _ptr(clock),
                                   _ptr(slot_idx), _ptr(plan), _ptr(stats), _stream(stream)),
           "moe_cache_experts")


def moe_pack_experts(d, F, E, bits, gate_q, gate_s, gate_b, up_q, up_s, up_b, down_q, down_s,
                     down_b, pool, expert_stride: int, stream=None):
    _check(lib().moe_pack_experts(d, F, E, bits, _ptr(gate_q), _ptr(gate_s), _ptr(gate_b),
                                  _ptr(up_q), _ptr(up_s), _ptr(up_b), _ptr(down_q),
                                  _ptr(down_s), _ptr(down_b), _ptr(pool), expert_stride,
                                  _stream(stream)), "moe_pack_experts")


def moe_debug_batched_waits(timeout_ns: int, stall: bool) -> None:
    """Test hook: the batched engine's wait bound (0 = 1 s) and a wait that
    nothing satisfies in every later launch (stall)."""
    _check(lib().moe_debug_batched_waits(int(timeout_ns), int(bool(stall))),
           "moe_debug_batched_waits")


def moe_debug_batched_engine(mode: int) -> None:
    """Which engine runs the batched GEMMs: 0 by size, 1 register
    (mma.sync), 2 tensor memory (tcgen05)."""
    _check(lib().moe_debug_batched_engine(int(mode)), "moe_debug_batched_engine")


def moe_debug_batched_trace(buf) -> None:
    """Profiling hook: stamps of CTA 0 of later tensor-memory engine launches
    into buf (device u64 [64 * 16]), or off (None)."""
    _check(lib().moe_debug_batched_trace(_ptr(buf)), "moe_debug_batched_trace")


def moe_debug_dequant(blob, d: int, F: int, bits: int, which: int, out, stream=None):
    _check(lib().moe_debug_dequant(_ptr(blob), d, F, bits, which, _ptr(out), _stream(stream)),
           "moe_debug_dequant")


def moe_prerouter_head(hd: HeadDesc, x, cur_idx, prev_idx, K: int, T: int, logits, ws,
                       stream=None, x_dtype: int | None = None):
    xd = _dtype_code(x) if x_dtype is None else x_dtype
    _check(lib().moe_prerouter_head(C.byref(hd), _ptr(x), xd, _ptr(cur_idx), _ptr(prev_idx), K,
                                    T, _ptr(logits), _ptr(ws), _nbytes(ws), _stream(stream)),
           "moe_prerouter_head")


def moe_topk_route(logits, T: int, E: int, K: int, idx, w, margin=None, stream=None):
    _check(lib().moe_topk_route(_ptr(logits), T, E, K, _ptr(idx), _ptr(w), _ptr(margin),
                                _stream(stream)), "moe_topk_route")


def _row_stride(t) -> int:
    """Elements between the rows of a tensor whose rows are contiguous."""
    if t.is_contiguous():
        return t.numel() // max(1, t.shape[0])
    if t.dim() == 2 and t.stride(1) == 1:
        return t.stride(0)
    inner = 1
    for n, st in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and st != inner:
            raise ValueError(f"rows must be contiguous: shape {tuple(t.shape)}, strides {t.stride()}")
        inner *= n
    return inner if t.shape[0] <= 1 else t.stride(0)


def moe_scored_route(rd: RouteDesc, logits, T: int, idx, w, stream=None):
    """Top-K experts by softmax or sigmoid scores with a balance bias and
    groups; logits fp32 or bf16 [T][E], rows may be strided."""
    _check(lib().moe_scored_route(C.byref(rd), _ptr(logits), _dtype_code(logits),
                                  _row_stride(logits), T, _ptr(idx), _ptr(w), _stream(stream)),
           "moe_scored_route")


def moe_kv_plan(seq_len, new_len, R: int, block_table, max_blocks: int, page: int, ring,
                n_pages: int, pool, seq_out, first, slots, places, cap: int, pool_out, status,
                stream=None):
    """Block tables, slots and places of a scheduler step's new tokens, pages
    taken from and given back to the ring of free ones (see include/moe.h)."""
    _check(lib().moe_kv_plan(_ptr(seq_len), _ptr(new_len), R, _ptr(block_table), max_blocks, page,
                             _ptr(ring), n_pages, _ptr(pool), _ptr(seq_out), _ptr(first),
                             _ptr(slots), _ptr(places), cap, _ptr(pool_out), _ptr(status),
                             _stream(stream)), "moe_kv_plan")


def moe_kv_append(kv: KVDesc, k, v, slots, N: int, stream=None):
    """Keys and values of N tokens into the paged cache at their slots;
    k, v: fp32 or bf16 [N][Hkv][D] or [N][Hkv * D], tokens may be strided."""
    if k.dtype != v.dtype:
        raise TypeError(f"k and v must have one type, got {k.dtype} and {v.dtype}")
    _check(lib().moe_kv_append(C.byref(kv), _ptr(k), _row_stride(k), _ptr(v), _row_stride(v),
                               _dtype_code(k), _ptr(slots), N, _stream(stream)), "moe_kv_append")


def moe_paged_attention_workspace_bytes(kv: KVDesc, B: int, Hq: int) -> int:
    return lib().moe_paged_attention_workspace_bytes(C.byref(kv), B, Hq)


def moe_paged_attention(kv: KVDesc, q, B: int, Hq: int, seq_len, block_table, max_blocks: int,
                        scale: float, out, ws, lse=None, window: int = 0, stream=None):
    """Attention of one new token per request over the paged cache; q and out
    fp32 or bf16 (one type) [B][Hq][D], rows may be strided."""
    if q.dtype != out.dtype:
        raise TypeError(f"q and out must have one type, got {q.dtype} and {out.dtype}")
    _check(lib().moe_paged_attention(C.byref(kv), _ptr(q), _dtype_code(q), _row_stride(q), B, Hq,
                                     _ptr(seq_len), _ptr(block_table), max_blocks, scale, window,
                                     _ptr(out), _row_stride(out), _ptr(lse), _ptr(ws), _nbytes(ws),
                                     _stream(stream)), "moe_paged_attention")


_kinds = None


def _kind(t) -> int:
    """The type of numbers that may be in 8 bits (codes as uint8, too)."""
    global _kinds
    if _kinds is None:
        import torch
        _kinds = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16,
                  torch.float8_e4m3fn: MOE_DTYPE_E4M3, torch.uint8: MOE_DTYPE_E4M3}
    try:
        return _kinds[t.dtype]
    except KeyError:
        raise TypeError(f"numbers must be float32, bfloat16 or float8_e4m3fn, got {t.dtype}") from None


def _stride0(t) -> int:
    """_row_stride, at once for the rows of a matrix."""
    st = t.stride()
    return st[0] if len(st) == 2 and st[1] == 1 else _row_stride(t)


def _code_rows(t, what: str) -> int:
    if _kind(t) != MOE_DTYPE_E4M3:
        raise TypeError(f"{what} must be float8_e4m3fn (or uint8), got {t.dtype}")
    return _stride0(t)


def _f32(t, what: str) -> int:
    if _kind(t) != MOE_DTYPE_F32:
        raise TypeError(f"{what} must be float32, got {t.dtype}")
    return _stride0(t)


def moe_quantise_e4m3(x, rows: int, cols: int, codes, scales, block_rows: int = 1,
                      pow2: bool = False, stream=None):
    """x fp32 or bf16 [rows][cols] as e4m3 codes with a fp32 scale for each
    block of block_rows (1 or 128) x 128; rows may be strided."""
    _check(lib().moe_quantise_e4m3(_ptr(x), _dtype_code(x), _stride0(x), rows, cols, block_rows,
                                   int(bool(pow2)), _ptr(codes), _code_rows(codes, "codes"),
                                   _ptr(scales), _f32(scales, "scales"), _stream(stream)),
           "moe_quantise_e4m3")


def moe_add_rms_norm(nd: NormDesc, x, T: int, y, res=None, sum=None, scales=None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight of h = x + res (res None: x), and
    h itself into sum (of res's type; may be res).  y fp32, bf16 or e4m3 codes
    with their scales; rows may be strided."""
    yd = _kind(y)
    if sum is not None and res is not None and sum.dtype != res.dtype:
        raise TypeError(f"sum and res must have one type, got {sum.dtype} and {res.dtype}")
    _check(lib().moe_add_rms_norm(
        C.byref(nd), _ptr(x), _dtype_code(x), _stride0(x), _ptr(res),
        MOE_DTYPE_F32 if res is None else _dtype_code(res), 0 if res is None else _stride0(res),
        T, _ptr(sum), 0 if sum is None else _stride0(sum), _ptr(y), yd, _stride0(y),
        _ptr(scales), 0 if scales is None else _f32(scales, "scales"), _stream(stream)),
        "moe_add_rms_norm")


def moe_scaled_product_workspace_bytes(wd: ScaledMatrixDesc, T: int) -> int:
    return lib().moe_scaled_product_workspace_bytes(C.byref(wd), T)


def moe_scaled_product(wd: ScaledMatrixDesc, x, x_scales, T: int, out, ws, stream=None):
    """out [T][N] (fp32 or bf16) = x W^T of e4m3 codes x [T][K] with scales for
    each 128 of a row; ws: zeroed once, its word 0 is the status."""
    _check(lib().moe_scaled_product(C.byref(wd), _ptr(x), _code_rows(x, "x"), _ptr(x_scales),
                                    _f32(x_scales, "x_scales"), T, _ptr(out), _dtype_code(out),
                                    _stride0(out), _ptr(ws), _nbytes(ws), _stream(stream)),
           "moe_scaled_product")


def moe_rotary_table(rd: RotaryDesc, turns, stream=None):
    """The frequencies of a rotary embedding, int64 (or uint64) [rot / 2]."""
    _check(lib().moe_rotary_table(C.byref(rd), _ptr(turns), _stream(stream)), "moe_rotary_table")


def moe_rotary(rd: RotaryDesc, turns, places, T: int, q, Hq: int, q_out, k=None, Hk: int = 0,
               k_out=None, stream=None):
    """q and k, [T][H][D] or [T][H * D], fp32 or bf16, turned by their places
    (int32 [T]) into q_out and k_out, which may be q and k; tokens may be
    strided."""
    dt = (q if q is not None else k).dtype
    for t in (q, q_out, k, k_out):
        if t is not None and t.dtype != dt:
            raise TypeError(f"q, k and their results must have one type, got {dt} and {t.dtype}")
    row = lambda t: 0 if t is None else _stride0(t)  # noqa: E731
    _check(lib().moe_rotary(C.byref(rd), _ptr(turns), _ptr(places), T,
                            _dtype_code(q if q is not None else k), _ptr(q),
                            row(q), Hq, _ptr(q_out), row(q_out), _ptr(k), row(k), Hk, _ptr(k_out),
                            row(k_out), _stream(stream)), "moe_rotary")


def moe_expert_ffn_int4(ed: ExpertsDesc, x, idx, T: int, K: int, y_slots, ws, stream=None,
                        x_dtype: int | None = None):
    xd = _dtype_code(x) if x_dtype is None else x_dtype
    _check(lib().moe_expert_ffn_int4(C.byref(ed), _ptr(x), xd, _ptr(idx), T, K, _ptr(y_slots),
                                     _ptr(ws), _nbytes(ws), _stream(stream)),
           "moe_expert_ffn_int4")


def moe_combine_residual(y_slots, w, T: int, K: int, has_shared: bool, d: int, residual, out,
                         x_next=None, stream=None):
    _check(lib().moe_combine_residual(_ptr(y_slots), _ptr(w), T, K, int(has_shared), d,
                                      _ptr(residual), _ptr(out), _ptr(x_next),
                                      _stream(stream)), "moe_combine_residual")


MOE_FFN_STATIC_SCRATCH_BYTES = 4 << 20


def moe_expert_ffn_int4_noalloc(ed: ExpertsDesc, x, idx, T: int, K: int, y_slots, stream=None,
                                x_dtype: int | None = None):
    """moe_expert_ffn_int4 for callers that cannot allocate: the library's
    fixed static device scratch stands in for the workspace."""
    xd = _dtype_code(x) if x_dtype is None else x_dtype
    _check(lib().moe_expert_ffn_int4_noalloc(C.byref(ed), _ptr(x), xd, _ptr(idx), T, K,
                                             _ptr(y_slots), _stream(stream)),
           "moe_expert_ffn_int4_noalloc")


def moe_expert_ffn_noalloc_status(stream=None) -> int:
    """Status word of the last allocation-free expert call on the current
    device (synchronises the stream): MOE_OK or MOE_ETIMEOUT."""
    st = C.c_int(0)
    _check(lib().moe_expert_ffn_noalloc_status(C.byref(st), _stream(stream)),
           "moe_expert_ffn_noalloc_status")
    return st.value


# ------------------------------------------------------------------ stack
def moe_decode_step_workspace_bytes(sd: StackDesc) -> int:
    return lib().moe_decode_step_workspace_bytes(C.byref(sd))


def moe_decode_step(sd: StackDesc, x0, out, route_idx, route_w, route_margin, t: int, ws,
                    stream=None):
    _check(lib().moe_decode_step(C.byref(sd), _ptr(x0), _ptr(out), _ptr(route_idx),
                                 _ptr(route_w), _ptr(route_margin), t, _ptr(ws), _nbytes(ws),
                                 _stream(stream)), "moe_decode_step")


def moe_decode_step_chain_workspace_bytes(sd: StackDesc) -> int:
    return lib().moe_decode_step_chain_workspace_bytes(C.byref(sd))


def moe_decode_step_chain(sd: StackDesc, x0, out, route_idx, route_w, route_margin, t: int, ws,
                          stream=None):
    _check(lib().moe_decode_step_chain(C.byref(sd), _ptr(x0), _ptr(out), _ptr(route_idx),
                                       _ptr(route_w), _ptr(route_margin), t, _ptr(ws), _nbytes(ws),
                                       _stream(stream)), "moe_decode_step_chain")


def moe_decode_step_chain_variant(variant: int, prefetch_l2: bool = True) -> None:
    """0: the library's choice, 1: two kernels per layer, 2: one cluster
    kernel per layer (process-wide; read when a step is enqueued)."""
    _check(lib().moe_decode_step_chain_variant(int(variant), int(bool(prefetch_l2))),
           "moe_decode_step_chain_variant")


def moe_decode_step_chain_cache(max_graphs: int) -> None:
    """Graphs moe_decode_step_chain keeps for repeated calls (0: none)."""
    _check(lib().moe_decode_step_chain_cache(int(max_graphs)), "moe_decode_step_chain_cache")


def moe_decode_step_chain_info(sd: StackDesc) -> dict:
    """How the chain's two per-layer kernels sit on an SM of the current
    device (shared memory, registers, CTAs per SM, co-residency)."""
    info = ChainInfo()
    _check(lib().moe_decode_step_chain_info(C.byref(sd), C.byref(info)),
           "moe_decode_step_chain_info")
    return {k: getattr(info, k) for k, _ in ChainInfo._fields_}


def moe_decode_step_status(ws, stream=None) -> int:
    st = C.c_int(0)
    _check(lib().moe_decode_step_status(_ptr(ws), C.byref(st), _stream(stream)),
           "moe_decode_step_status")
    return st.value
