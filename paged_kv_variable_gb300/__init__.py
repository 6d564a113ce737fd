"""Python binding of the pkv C ABI (``include/pkv.h``): argument marshalling only.

Every step of the attention call runs in the CUDA library ``_lib/libpkv.so``;
this module only turns PyTorch tensors into pointers, strides and sizes.  If
the library has not been built, importing works but every call raises
``RuntimeError`` -- there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpkv.so")

PKV_BF16 = 0
PKV_FP8_E4M3 = 1

STATUS_NAMES = {
    0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED", 3: "PKV_ERR_WORKSPACE_TOO_SMALL",
    4: "PKV_ERR_CUDA", 5: "PKV_ERR_DEVICE_TIMEOUT", 6: "PKV_ERR_DEVICE_BOUNDS", 7: "PKV_ERR_PLAN_MISMATCH",
}

# every symbol the header declares
EXPORTED = ["pkv_plan", "pkv_plan_upload", "pkv_plan_get_stats", "pkv_plan_get_items", "pkv_attn_varlen_kvcache_fwd", "pkv_kv_append",
            "pkv_get_status", "pkv_plan_destroy", "pkv_last_error", "pkv_version", "pkv_set_profile_events",
            "pkv_attn_varlen_kvcache_fwd_noalloc", "pkv_plan_decode_dynamic", "pkv_get_status_noalloc",
            "pkv_qk_norm_rope", "pkv_rope_kv_append", "pkv_rope_attn_varlen_kvcache_fwd",
            "pkv_plan_shared_prefix"]


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class PkvInputError(PkvError, ValueError):
    """Refused by the binding: tensors that do not serve the call (the library sees their addresses alone)."""

    def __init__(self, msg: str):
        super().__init__(1, msg)


class Problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_heads_q", ctypes.c_int32), ("num_heads_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("cache_capacity", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("cache_dtype", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float)]


class FwdArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_stride_tok", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("o_stride_tok", ctypes.c_int64), ("o_stride_head", ctypes.c_int64),
                ("lse", ctypes.c_void_p), ("cu_seqlens_q", ctypes.c_void_p), ("max_seqlen_q", ctypes.c_int32),
                ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p), ("knew_stride_tok", ctypes.c_int64),
                ("knew_stride_head", ctypes.c_int64), ("cu_seqlens_knew", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("kc_stride_page", ctypes.c_int64),
                ("kc_stride_tok", ctypes.c_int64), ("kc_stride_head", ctypes.c_int64),
                ("cache_seqlens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("block_table_stride", ctypes.c_int32), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_indptr", ctypes.c_void_p), ("q_scale", ctypes.c_void_p), ("q_rows", ctypes.c_int32)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("num_positions", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p)]


class QkArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "num_heads_q", "num_heads_kv", "head_dim")] + [
        (n, ctypes.c_int64 if "stride" in n else ctypes.c_void_p)
        for n in ("q", "q_stride_tok", "q_stride_head", "q_out", "qo_stride_tok", "qo_stride_head",
                  "k", "k_stride_tok", "k_stride_head", "k_out", "ko_stride_tok", "ko_stride_head", "positions")]


class RopeAppendArgs(ctypes.Structure):
    _fields_ = [("spec", RopeSpec), ("q_out", ctypes.c_void_p), ("qo_stride_tok", ctypes.c_int64),
                ("qo_stride_head", ctypes.c_int64)]


class WorkItemInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("seq", "kv_head", "q_row0", "q_index0", "n_q", "q_len", "kv_len",
                                               "kv_begin", "kv_end", "kind", "partial_slot", "cta",
                                               "head0", "num_heads")] + [
        ("cost", ctypes.c_double)]


class PlanStats(ctypes.Structure):
    _fields_ = [("num_items", ctypes.c_int32), ("num_decode_items", ctypes.c_int32),
                ("num_prefill_items", ctypes.c_int32), ("num_split_units", ctypes.c_int32),
                ("num_ctas", ctypes.c_int32), ("total_q", ctypes.c_int32), ("total_new", ctypes.c_int32),
                ("max_items_per_cta", ctypes.c_int32), ("max_cta_cost", ctypes.c_double),
                ("mean_cta_cost", ctypes.c_double), ("upload_bytes", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"pkv CUDA library not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        L.pkv_plan.argtypes = [ctypes.POINTER(Problem), vp, vp, vp, i32, ctypes.POINTER(vp), ctypes.POINTER(sz)]
        L.pkv_plan_decode_dynamic.argtypes = L.pkv_plan.argtypes
        L.pkv_plan_shared_prefix.argtypes = [ctypes.POINTER(Problem), vp, vp, vp, i32, vp, vp, i32, i32, i32,
                                             ctypes.POINTER(vp), ctypes.POINTER(sz)]
        L.pkv_plan_upload.argtypes = [vp, vp, sz, vp]
        L.pkv_plan_get_stats.argtypes = [vp, ctypes.POINTER(PlanStats)]
        L.pkv_plan_get_items.argtypes = [vp, ctypes.POINTER(WorkItemInfo), i32, ctypes.POINTER(i32)]
        L.pkv_attn_varlen_kvcache_fwd.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(FwdArgs), vp, vp, sz, vp]
        L.pkv_kv_append.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(FwdArgs), i32, vp, vp]
        L.pkv_get_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
        L.pkv_set_profile_events.argtypes = [vp, vp]
        L.pkv_attn_varlen_kvcache_fwd_noalloc.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(FwdArgs), vp, vp]
        L.pkv_get_status_noalloc.argtypes = [vp, ctypes.POINTER(i32)]
        L.pkv_qk_norm_rope.argtypes = [ctypes.POINTER(QkArgs), ctypes.POINTER(RopeSpec), vp, vp]
        L.pkv_rope_kv_append.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(FwdArgs),
                                         ctypes.POINTER(RopeAppendArgs), i32, i32, vp, vp]
        L.pkv_rope_attn_varlen_kvcache_fwd.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(FwdArgs),
                                                       ctypes.POINTER(RopeAppendArgs), vp, vp, sz, vp]
        L.pkv_plan_destroy.argtypes = [vp]
        L.pkv_plan_destroy.restype = None
        L.pkv_last_error.restype = ctypes.c_char_p
        L.pkv_version.restype = ctypes.c_char_p
        for name in ("pkv_plan", "pkv_plan_upload", "pkv_plan_get_stats", "pkv_plan_get_items", "pkv_attn_varlen_kvcache_fwd",
                     "pkv_kv_append", "pkv_get_status", "pkv_set_profile_events",
                     "pkv_attn_varlen_kvcache_fwd_noalloc", "pkv_get_status_noalloc", "pkv_qk_norm_rope",
                     "pkv_rope_kv_append", "pkv_rope_attn_varlen_kvcache_fwd"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != 0:
        raise PkvError(status, lib().pkv_last_error().decode())


def last_error() -> str:
    return lib().pkv_last_error().decode()


def version() -> str:
    return lib().pkv_version().decode()


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch
        # (torch's own raw query, where this torch has it: the current_stream() object costs 3 us a call on the host)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return torch.cuda.current_stream().cuda_stream if raw is None else raw(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_problem(*, batch, num_heads_q, num_heads_kv, head_dim, page_size, cache_capacity, num_pages,
                 cache_dtype, causal, softmax_scale) -> Problem:
    dt = {"bf16": PKV_BF16, "fp8": PKV_FP8_E4M3}.get(cache_dtype, cache_dtype)
    return Problem(batch, num_heads_q, num_heads_kv, head_dim, page_size, cache_capacity, num_pages, dt,
                   int(bool(causal)), softmax_scale)


def make_args(*, q, out, cu_seqlens_q, max_seqlen_q, k_cache, v_cache, cache_seqlens, lse=None, k_new=None,
              v_new=None, cu_seqlens_knew=None, block_table=None, k_scale=None, v_scale=None,
              page_indptr=None, q_scale=None, q_rows=0) -> FwdArgs:
    """Pointers and element strides of torch tensors laid out as in pkv.h (which the struct keeps alive)."""
    a = FwdArgs()
    a.keep = (q, out, cu_seqlens_q, k_cache, v_cache, cache_seqlens, lse, k_new, v_new, cu_seqlens_knew, block_table,
              k_scale, v_scale, page_indptr, q_scale)
    _same_layout(k_new, v_new, "k_new", "v_new")
    _same_layout(k_cache, v_cache, "k_cache", "v_cache")
    # what the calls compare with the problem and the counts of tokens, of each
    # tensor whose address the struct still holds by then
    a.given = {what: (t.data_ptr(), tuple(t.shape), str(getattr(t, "dtype", "bfloat16")).removeprefix("torch."))
               for what, t in (("q", q), ("out", out), ("lse", lse), ("k_new", k_new), ("v_new", v_new),
                               ("k_cache", k_cache), ("cu_seqlens_q", cu_seqlens_q), ("cache_seqlens", cache_seqlens),
                               ("cu_seqlens_knew", cu_seqlens_knew), ("block_table", block_table),
                               ("page_indptr", page_indptr))
               if t is not None}
    a.checked = None  # the last call that they were found to serve
    if q is not None:
        a.q, a.q_stride_tok, a.q_stride_head = q.data_ptr(), q.stride(0), q.stride(1)
    if out is not None:
        a.out, a.o_stride_tok, a.o_stride_head = out.data_ptr(), out.stride(0), out.stride(1)
    a.lse = _ptr(lse)
    a.cu_seqlens_q = _ptr(cu_seqlens_q)
    a.max_seqlen_q = int(max_seqlen_q)
    if k_new is not None:
        a.k_new, a.v_new = k_new.data_ptr(), _ptr(v_new)
        a.knew_stride_tok, a.knew_stride_head = k_new.stride(0), k_new.stride(1)
        a.cu_seqlens_knew = _ptr(cu_seqlens_knew)
    a.k_cache, a.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    a.kc_stride_page, a.kc_stride_tok, a.kc_stride_head = k_cache.stride(0), k_cache.stride(1), k_cache.stride(2)
    a.cache_seqlens = _ptr(cache_seqlens)
    if block_table is not None:
        a.block_table = block_table.data_ptr()
        a.block_table_stride = block_table.stride(0) if block_table.dim() > 1 else 0
    a.k_scale, a.v_scale = _ptr(k_scale), _ptr(v_scale)
    a.page_indptr = _ptr(page_indptr)
    a.q_scale = _ptr(q_scale)
    a.q_rows = int(q_rows)
    return a


def _same_layout(x, y, what_x: str, what_y: str) -> None:
    """Raises ValueError unless y has the shape of x and its strides, which serve both."""
    if x is None or y is None:
        return
    if tuple(x.shape) != tuple(y.shape) or any(n > 1 and x.stride(i) != y.stride(i) for i, n in enumerate(x.shape)):
        raise PkvInputError(f"{what_y} must have the shape and strides of {what_x}")


def _check_rows(problem: Problem, args: FwdArgs, total_q: int, total_new: int, bf16: bool = False) -> None:
    """The tensors of make_args against the rows that the call reads and writes:
    q and out (rows, Hq, D), k_new and v_new (rows, Hkv, D), lse (Hq, rows), with
    at least so many rows and heads, and the caches, offsets and page tables with the
    problem.  Structs that were not made by make_args, and addresses put in since,
    are taken as they are."""
    given = getattr(args, "given", None)
    if given is None:
        return
    call = (total_q, total_new, bf16, bytes(problem))
    if call == args.checked:
        return
    d, batch = problem.head_dim, problem.batch
    for what, rows, heads in (("q", total_q, problem.num_heads_q), ("out", total_q, problem.num_heads_q),
                              ("k_new", total_new, problem.num_heads_kv), ("v_new", total_new, problem.num_heads_kv)):
        if rows > 0 and what in given:
            ptr, shape, dtype = given[what]
            if ((len(shape) != 3 or shape[0] < rows or shape[1] < heads or shape[2] != d)
                    and getattr(args, what) == ptr):
                raise PkvInputError(f"{what} {shape}: ({rows}, {heads}, {d}) expected")
            if bf16 and dtype != "bfloat16" and getattr(args, what) == ptr:
                raise PkvInputError(f"{what}: bfloat16 expected, got {dtype}")
    if total_q > 0 and "lse" in given:
        ptr, shape, _ = given["lse"]
        if math.prod(shape) < problem.num_heads_q * total_q and args.lse == ptr:
            raise PkvInputError(f"lse {shape}: ({problem.num_heads_q}, {total_q}) expected")
    for what, least in (("cu_seqlens_q", batch + 1 if total_q > 0 else 0), ("cache_seqlens", batch),
                        ("cu_seqlens_knew", batch + 1 if total_new > 0 else 0), ("page_indptr", batch + 1)):
        if what in given:
            ptr, shape, _ = given[what]
            if math.prod(shape) < least and getattr(args, what) == ptr:
                raise PkvInputError(f"{what} {shape}: {least} values expected")
    tokens = problem.page_size or problem.cache_capacity
    ptr, shape, _ = given["k_cache"]
    if (len(shape) != 4 or shape[0] < problem.num_pages or shape[1] < tokens or shape[2] < problem.num_heads_kv
            or shape[3] != d) and args.k_cache == ptr:
        raise PkvInputError(f"k_cache {shape}: ({problem.num_pages}, {tokens}, {problem.num_heads_kv}, {d}) expected")
    if "block_table" in given and "page_indptr" not in given:  # (the library looks at the stride of its rows)
        ptr, shape, _ = given["block_table"]
        if shape[0] < batch and args.block_table == ptr:
            raise PkvInputError(f"block_table {shape}: {batch} rows expected")
    args.checked = call


def _check_status_words(device_status) -> None:
    if device_status is not None and device_status.numel() * device_status.element_size() < 12:
        raise PkvInputError("device_status: three int32 expected")


def _need(t, what: str, dtypes: tuple, ndim: int) -> None:
    """Raises ValueError unless t has one of the dtypes (by name), ndim dims and a unit innermost stride."""
    if str(t.dtype).removeprefix("torch.") not in dtypes or t.dim() != ndim:
        raise ValueError(f"{what}: {ndim}-d tensor of {' or '.join(dtypes)} expected, got {tuple(t.shape)} {t.dtype}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: innermost stride must be 1")


def make_rope_spec(*, cos_sin=None, interleaved=False, eps=1e-6, q_weight=None, k_weight=None) -> RopeSpec:
    """How rows are normed and rotated.  cos_sin: (positions, rot_dim) fp32, the
    rot_dim/2 cosines and then sines of each position (None: no rotation);
    q_weight / k_weight: (head_dim,) bf16 RMS norm weights (None: no norm).  The
    spec keeps the tensors alive."""
    r = RopeSpec(interleaved=int(bool(interleaved)), eps=eps, q_weight=_ptr(q_weight), k_weight=_ptr(k_weight))
    r.keep = (cos_sin, q_weight, k_weight)
    r.weight_dim = None  # head_dim that the weights are made for
    for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _need(w, what, ("bfloat16",), 1)
            if r.weight_dim not in (None, w.shape[0]):
                raise ValueError(f"q_weight and k_weight differ in length ({r.weight_dim}, {w.shape[0]})")
            r.weight_dim = w.shape[0]
    if cos_sin is not None:
        _need(cos_sin, "cos_sin", ("float32",), 2)
        if cos_sin.shape[0] > 1 and cos_sin.stride(0) != cos_sin.shape[1]:
            raise ValueError("cos_sin must be contiguous")
        r.cos_sin, (r.num_positions, r.rot_dim) = cos_sin.data_ptr(), cos_sin.shape
    return r


def make_qk_args(*, q=None, k=None, positions=None, q_out=None, k_out=None) -> QkArgs:
    """Tensors of ``qk_norm_rope``: q (T, Hq, D) and / or k (T, Hkv, D) bf16, int32
    positions (T,), and where the results go (None: in place).  The struct keeps the tensors alive."""
    if q is None and k is None:
        raise ValueError("q or k must be given")
    a = QkArgs()
    a.keep = (q, k, positions, q_out, k_out)
    t = q if q is not None else k
    a.num_tokens, a.head_dim = t.shape[0], t.shape[-1]
    if positions is not None:
        _need(positions, "positions", ("int32",), 1)
        if positions.shape[0] != a.num_tokens:
            raise ValueError(f"positions: {a.num_tokens} tokens expected, got {positions.shape[0]}")
        a.positions = positions.data_ptr()
    for what, x, y in (("q", q, q_out), ("k", k, k_out)):
        if x is None:
            if y is not None:
                raise ValueError(f"{what}_out given without {what}")
            continue
        y = x if y is None else y
        _need(x, what, ("bfloat16",), 3)
        _need(y, what + "_out", ("bfloat16",), 3)
        if x.shape != y.shape or x.shape[0] != a.num_tokens or x.shape[2] != a.head_dim:
            raise ValueError(f"{what} {tuple(x.shape)} and {what}_out {tuple(y.shape)} must agree in shape, and q and k "
                             "in tokens and head_dim")
        setattr(a, "num_heads_q" if what == "q" else "num_heads_kv", x.shape[1])
        setattr(a, what, x.data_ptr())
        setattr(a, what + "_stride_tok", x.stride(0))
        setattr(a, what + "_stride_head", x.stride(1))
        setattr(a, what + "_out", y.data_ptr())
        setattr(a, what + "o_stride_tok", y.stride(0))
        setattr(a, what + "o_stride_head", y.stride(1))
    return a


def make_rope_append_args(*, spec: RopeSpec, q_out=None) -> RopeAppendArgs:
    """The transform of ``rope_kv_append`` and where its queries go (None: the
    queries are left alone).  The struct keeps q_out and the spec's tensors alive."""
    r = RopeAppendArgs(spec=spec)
    r.keep = (getattr(spec, "keep", None), q_out)
    r.weight_dim, r.q_shape = getattr(spec, "weight_dim", None), None
    if q_out is not None:
        _need(q_out, "q_out", ("bfloat16",), 3)
        r.q_shape = tuple(q_out.shape)
        r.q_out, r.qo_stride_tok, r.qo_stride_head = q_out.data_ptr(), q_out.stride(0), q_out.stride(1)
    return r


def _check_weights(weight_dim, head_dim: int) -> None:
    if weight_dim is not None and weight_dim != head_dim:
        raise ValueError(f"norm weights of {weight_dim} values for head_dim {head_dim}")


def _check_rope(problem: Problem, rope: RopeAppendArgs, total_q: int) -> None:
    """The transform's tensors against the problem: what the pointers alone do not tell the library."""
    _check_weights(getattr(rope, "weight_dim", None), problem.head_dim)
    shape = getattr(rope, "q_shape", None)
    if shape is not None and (shape[0] < total_q or shape[1:] != (problem.num_heads_q, problem.head_dim)):
        raise ValueError(f"q_out {shape}: ({total_q}, {problem.num_heads_q}, {problem.head_dim}) expected")


class Plan:
    """Host work list made by ``pkv_plan`` (owned until ``close``)."""

    def __init__(self, problem: Problem, q_lens, cache_lens, new_lens, num_sms: int, dynamic: bool = False,
                 shared=None):
        import numpy as np
        for what, lens in (("q_lens", q_lens), ("cache_lens", cache_lens), ("new_lens", new_lens)):
            if lens is not None and (len(lens) < problem.batch or shared is not None and len(lens) != problem.batch):
                raise ValueError(f"{what}: {problem.batch} sequences expected, got {len(lens)}")
        self.problem = problem
        self._q = np.ascontiguousarray(q_lens, dtype=np.int32)
        self._c = np.ascontiguousarray(cache_lens, dtype=np.int32)
        self._n = None if new_lens is None else np.ascontiguousarray(new_lens, dtype=np.int32)
        h = ctypes.c_void_p()
        ws = ctypes.c_size_t()
        lens = (ctypes.byref(problem), self._q.ctypes.data, self._c.ctypes.data,
                None if self._n is None else self._n.ctypes.data)
        if shared is not None:  # (group_starts, prefix_lens, always)
            starts, prefixes = (np.ascontiguousarray(x, dtype=np.int32) for x in shared[:2])
            if len(starts) != len(prefixes) + 1:
                raise ValueError(f"{len(prefixes)} prefix_lens need {len(prefixes) + 1} group_starts, got {len(starts)}")
            _check(lib().pkv_plan_shared_prefix(*lens, len(prefixes), starts.ctypes.data, prefixes.ctypes.data,
                                                int(bool(shared[2])), int(dynamic), int(num_sms), ctypes.byref(h), ctypes.byref(ws)))
        else:
            fn = lib().pkv_plan_decode_dynamic if dynamic else lib().pkv_plan
            _check(fn(*lens, int(num_sms), ctypes.byref(h), ctypes.byref(ws)))
        self.handle = h
        self._shares = None if shared is not None else False  # tiles over a shared prefix (None: not looked at)
        self.workspace_bytes = int(ws.value)
        self.total_q = int(self._q[:problem.batch].sum())
        self.total_new = 0 if self._n is None else int(self._n[:problem.batch].sum())

    def rows(self, args: FwdArgs) -> int:
        """Rows of q, out and lse in a call of this plan (q_rows where the caller places them, which the library
        refuses if the plan shares a prefix)."""
        if args.q_rows <= 0:
            return self.total_q
        if self._shares is None:
            import numpy as np
            seq = np.repeat(np.arange(self.problem.batch), self._q[:self.problem.batch])
            self._shares = any(seq[it["q_row0"]] != seq[it["q_row0"] + it["n_q"] - 1] for it in self.items())
        return self.total_q if self._shares else args.q_rows

    def stats(self) -> dict:
        s = PlanStats()
        _check(lib().pkv_plan_get_stats(self.handle, ctypes.byref(s)))
        return {k: getattr(s, k) for k, _ in PlanStats._fields_}

    def items(self) -> list[dict]:
        n = ctypes.c_int32()
        _check(lib().pkv_plan_get_items(self.handle, None, 0, ctypes.byref(n)))
        arr = (WorkItemInfo * max(1, n.value))()
        _check(lib().pkv_plan_get_items(self.handle, arr, n.value, ctypes.byref(n)))
        return [{k: getattr(arr[i], k) for k, _ in WorkItemInfo._fields_} for i in range(n.value)]

    def upload(self, workspace, stream=None) -> None:
        _check(lib().pkv_plan_upload(self.handle, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     _stream_handle(stream)))

    def close(self) -> None:
        if self.handle:
            lib().pkv_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def plan(problem: Problem, q_lens, cache_lens, new_lens=None, num_sms: Optional[int] = None) -> Plan:
    if num_sms is None:
        import torch
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return Plan(problem, q_lens, cache_lens, new_lens, num_sms)


def plan_decode_dynamic(problem: Problem, q_lens, max_cache_lens, new_lens=None,
                        num_sms: Optional[int] = None) -> Plan:
    """A decode plan whose cache lengths are read on the device at every call
    (bounded by max_cache_lens), for a call captured once in a CUDA graph."""
    if num_sms is None:
        import torch
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return Plan(problem, q_lens, max_cache_lens, new_lens, num_sms, dynamic=True)


def plan_shared_prefix(problem: Problem, q_lens, cache_lens, new_lens=None, *, group_starts, prefix_lens,
                       always: bool = False, dynamic: bool = False, num_sms: Optional[int] = None) -> Plan:
    """A plan for groups of consecutive sequences (group g: group_starts[g] ..
    group_starts[g+1] - 1) whose first prefix_lens[g] tokens lie in the same
    pages: the prefix is attended once for the whole group, where that is expected
    to be faster (always: in any case).  dynamic: as ``plan_decode_dynamic``
    (cache_lens are bounds)."""
    if num_sms is None:
        import torch
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return Plan(problem, q_lens, cache_lens, new_lens, num_sms, dynamic=dynamic,
                shared=(group_starts, prefix_lens, always))


def attn_varlen_kvcache_fwd(problem: Problem, args: FwdArgs, plan_: Plan, workspace, stream=None) -> None:
    _check_rows(problem, args, plan_.rows(args), plan_.total_new)
    _check(lib().pkv_attn_varlen_kvcache_fwd(ctypes.byref(problem), ctypes.byref(args), plan_.handle,
                                             workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                             _stream_handle(stream)))


def attn_varlen_kvcache_fwd_noalloc(problem: Problem, args: FwdArgs, plan_: Plan, stream=None) -> None:
    """The attention call without a caller workspace (for callers that cannot
    allocate device memory); uses the library's fixed 32 MiB device scratch."""
    _check_rows(problem, args, plan_.rows(args), plan_.total_new)
    _check(lib().pkv_attn_varlen_kvcache_fwd_noalloc(ctypes.byref(problem), ctypes.byref(args), plan_.handle,
                                                     _stream_handle(stream)))


def get_status_noalloc(stream=None) -> int:
    """Device status word left by the last no-workspace call on this device (then reset)."""
    st = ctypes.c_int32()
    _check(lib().pkv_get_status_noalloc(_stream_handle(stream), ctypes.byref(st)))
    return int(st.value)


def kv_append(problem: Problem, args: FwdArgs, total_new: int, device_status=None, stream=None) -> None:
    _check_rows(problem, args, 0, total_new)
    _check(lib().pkv_kv_append(ctypes.byref(problem), ctypes.byref(args), int(total_new), _ptr(device_status),
                               _stream_handle(stream)))


def qk_norm_rope(args: QkArgs, spec: RopeSpec, device_status=None, stream=None) -> None:
    """Norm of every head of q and k and the rotation by each token's position, in one pass."""
    _check_weights(getattr(spec, "weight_dim", None), args.head_dim)
    _check_status_words(device_status)
    _check(lib().pkv_qk_norm_rope(ctypes.byref(args), ctypes.byref(spec), _ptr(device_status),
                                  _stream_handle(stream)))


def rope_kv_append(problem: Problem, args: FwdArgs, rope: RopeAppendArgs, total_q: int, total_new: int,
                   device_status=None, stream=None) -> None:
    """``kv_append`` with the norm and rotation on the way into the cache, and of the queries into rope's q_out."""
    _check_rope(problem, rope, total_q)
    _check_rows(problem, args, total_q if rope.q_out else 0, total_new, bf16=True)
    _check_status_words(device_status)
    _check(lib().pkv_rope_kv_append(ctypes.byref(problem), ctypes.byref(args), ctypes.byref(rope), int(total_q),
                                    int(total_new), _ptr(device_status), _stream_handle(stream)))


def rope_attn_varlen_kvcache_fwd(problem: Problem, args: FwdArgs, rope: RopeAppendArgs, plan_: Plan, workspace,
                                 stream=None) -> None:
    """The attention call with ``rope_kv_append`` in place of its append."""
    _check_rope(problem, rope, plan_.total_q)
    _check_rows(problem, args, plan_.total_q, plan_.total_new, bf16=True)
    _check(lib().pkv_rope_attn_varlen_kvcache_fwd(ctypes.byref(problem), ctypes.byref(args), ctypes.byref(rope),
                                                  plan_.handle, workspace.data_ptr(),
                                                  workspace.numel() * workspace.element_size(),
                                                  _stream_handle(stream)))


def get_status(workspace, stream=None) -> int:
    st = ctypes.c_int32()
    _check(lib().pkv_get_status(workspace.data_ptr(), _stream_handle(stream), ctypes.byref(st)))
    return int(st.value)


def set_profile_events(start=None, stop=None) -> None:
    """Record torch.cuda.Event objects around the attention kernel of later calls.

    torch creates the CUDA event lazily, on its first record(); record both once
    here so that the handles passed to the library exist."""
    if start is not None:
        start.record()
        stop.record()
        assert start.cuda_event and stop.cuda_event
    _check(lib().pkv_set_profile_events(None if start is None else start.cuda_event,
                                        None if stop is None else stop.cuda_event))


def workspace_tensor(nbytes: int, device="cuda"):
    """A caller-owned, 256-byte aligned device workspace of at least nbytes."""
    import torch
    return torch.zeros(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device)
