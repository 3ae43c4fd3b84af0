"""Thin ctypes binding of libekv.so (the C ABI of include/ekv.h).

Argument marshalling only: PyTorch supplies device memory and the current
stream; every step of the decode path runs in the library's CUDA kernels.
There is no fallback — if the library is missing or fails to load, every call
raises ``EkvUnavailable``.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "EkvError", "EkvUnavailable", "Cache", "Seqs", "StepParams", "lib", "lib_path",
    "EKV_F32", "EKV_BF16", "EKV_POLICY_TOPK", "EKV_POLICY_GAUSS", "EKV_POLICY_FULL",
    "EKV_OP_SELECT_GAUSS", "EKV_OP_ENTMAX_DECODE", "EKV_OP_DECODE_STEP",
    "EKV_EFLAG_BAD_PAGE", "EKV_EFLAG_BAD_LEN", "EKV_EFLAG_SEL_OVERFLOW", "EKV_EFLAG_BAD_SEL",
    "make_cache", "make_seqs", "workspace", "ekv_build_page_meta", "ekv_append",
    "ekv_score_pages", "ekv_select_topk", "ekv_select_gauss", "ekv_entmax_decode",
    "ekv_decode_step", "ekv_workspace_bytes", "ekv_get_error", "ekv_status_string",
    "ekv_entmax_decode_static_ws", "ekv_step_kernel_count", "ekv_softmax_decode", "EKV_OP_SOFTMAX_DECODE",
    "ekv_exactness_certificate", "EKV_OP_SELECT_TOPK", "ekv_selftest_wait_timeout", "EKV_EFLAG_TIMEOUT",
    "ekv_decode_adaptive", "EKV_OP_DECODE_ADAPTIVE", "EKV_EFLAG_BAD_POS",
    "CacheQ4", "Rope", "NewTokens", "ScoreMod", "make_cache_q4", "make_rope", "make_new_tokens", "make_score_mod",
    "q4_record_bytes", "ekv_rope_append", "ekv_rope_append_q4", "ekv_q4_read", "ekv_softmax_decode_mod",
    "ekv_softmax_decode_q4", "ekv_softmax_mod_workspace_bytes",
]

EKV_F32, EKV_BF16 = 0, 1
EKV_POLICY_TOPK, EKV_POLICY_GAUSS, EKV_POLICY_FULL = 0, 1, 2
EKV_OP_SELECT_GAUSS, EKV_OP_ENTMAX_DECODE, EKV_OP_DECODE_STEP, EKV_OP_SOFTMAX_DECODE = 1, 2, 3, 4
EKV_OP_SELECT_TOPK = 5
EKV_OP_DECODE_ADAPTIVE = 6
EKV_EFLAG_BAD_PAGE, EKV_EFLAG_BAD_LEN, EKV_EFLAG_SEL_OVERFLOW, EKV_EFLAG_BAD_SEL = 1, 2, 4, 8
EKV_EFLAG_TIMEOUT = 16
EKV_EFLAG_BAD_POS = 32

lib_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libekv.so")


class EkvError(RuntimeError):
    def __init__(self, name, status):
        super().__init__(f"{name}: {ekv_status_string(status)} (status {status})")
        self.status = status


class EkvUnavailable(RuntimeError):
    pass


class Cache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("num_phys_pages", ctypes.c_int32), ("k_pool", ctypes.c_void_p),
                ("v_pool", ctypes.c_void_p), ("box", ctypes.c_void_p), ("mom", ctypes.c_void_p)]


class Seqs(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class StepParams(ctypes.Structure):
    _fields_ = [("policy", ctypes.c_int32), ("k", ctypes.c_int32), ("delta", ctypes.c_float),
                ("cap", ctypes.c_int32), ("alpha", ctypes.c_float), ("scale", ctypes.c_float),
                ("dense_v", ctypes.c_int32), ("append", ctypes.c_int32)]


class CacheQ4(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("num_phys_pages", ctypes.c_int32), ("pool", ctypes.c_void_p), ("box", ctypes.c_void_p),
                ("mom", ctypes.c_void_p)]


class Rope(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class NewTokens(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("indptr", ctypes.c_void_p), ("num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class ScoreMod(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32), ("slopes", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p), ("starts", ctypes.c_void_p)]


_LIB = None
_P = ctypes.c_void_p
_I = ctypes.c_int32
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_SIGS = {
    "ekv_build_page_meta": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _P],
    "ekv_append": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _P, _P, _P],
    "ekv_score_pages": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _P, _I, _F, _P, _P],
    "ekv_select_topk": [ctypes.POINTER(Seqs), _I, _I, _P, _I, _P, _P, _P, _SZ, _P],
    "ekv_select_gauss": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _P, _I, _F, _F, _F, _I,
                         _P, _P, _P, _P, _SZ, _P],
    "ekv_entmax_decode": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _P, _I, _F, _F, _P, _P,
                          _I, _I, _P, _P, _P, _P, _P, _SZ, _P],
    "ekv_decode_step": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), ctypes.POINTER(StepParams),
                        _P, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P],
    "ekv_workspace_bytes": [_I, ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _I, _I],
    "ekv_softmax_decode": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _P, _I, _F, _P, _P, _I, _P, _P,
                           _P, _SZ, _P],
    "ekv_exactness_certificate": [ctypes.POINTER(Seqs), _I, _I, _I, _F, _P, _P, _P, _I, _P, _P, _P],
    "ekv_decode_adaptive": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _P, _I, _F, _F, _I, _P, _P, _P, _P, _P,
                            ctypes.POINTER(ctypes.c_int32), _P, _SZ, _P],
    "ekv_rope_append": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), ctypes.POINTER(Rope), ctypes.POINTER(NewTokens),
                        _P],
    "ekv_rope_append_q4": [ctypes.POINTER(CacheQ4), ctypes.POINTER(Seqs), ctypes.POINTER(Rope),
                           ctypes.POINTER(NewTokens), _P],
    "ekv_q4_read": [ctypes.POINTER(CacheQ4), ctypes.POINTER(Seqs), _P, _I, _I, _P, _P, _P],
    "ekv_softmax_decode_mod": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _P, _I, _I, _F, ctypes.POINTER(ScoreMod),
                               _P, _P, _I, _P, _P, _P, _SZ, _P],
    "ekv_softmax_decode_q4": [ctypes.POINTER(CacheQ4), ctypes.POINTER(Seqs), _P, _I, _I, _F,
                              ctypes.POINTER(ScoreMod), _P, _P, _I, _P, _P, _P, _SZ, _P],
    "ekv_softmax_mod_workspace_bytes": [_I, _I, _I, _I],
    "ekv_selftest_wait_timeout": [ctypes.c_uint32, _P],
    "ekv_step_kernel_count": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), ctypes.POINTER(StepParams), _I],
    "ekv_entmax_decode_static_ws": [ctypes.POINTER(Cache), ctypes.POINTER(Seqs), _P, _I, _F, _F, _P,
                                    _P, _I, _I, _P, _P, _P, _P, _P],
    "ekv_get_error": [ctypes.POINTER(ctypes.c_uint32)],
    "ekv_status_string": [_I],
}


def lib():
    """The loaded libekv.so (raises EkvUnavailable when it is missing)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(lib_path):
            raise EkvUnavailable(f"{lib_path} is missing: build it with sparse_kv_cache_kmax_b200.build_lib.build()")
        try:
            h = ctypes.CDLL(lib_path)
        except OSError as e:
            raise EkvUnavailable(f"cannot load {lib_path}: {e}") from e
        for name, args in _SIGS.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int32
        h.ekv_workspace_bytes.restype = ctypes.c_size_t
        h.ekv_softmax_mod_workspace_bytes.restype = ctypes.c_size_t
        h.ekv_status_string.restype = ctypes.c_char_p
        _LIB = h
    return _LIB


def ekv_status_string(status: int) -> str:
    try:
        return lib().ekv_status_string(int(status)).decode()
    except EkvUnavailable:
        return f"status {status}"


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(name, status):
    if status != 0:
        raise EkvError(name, status)


_DTYPES = {torch.float32: EKV_F32, torch.bfloat16: EKV_BF16}


def make_cache(k_pool, v_pool, box=None, mom=None) -> Cache:
    """Describe a paged cache.  k_pool, v_pool: [num_phys, Hkv, S, d];
    box, mom: [Hkv, num_phys, 2, d] (head-major) of the same dtype (allocated
    here if None)."""
    if box is None:
        box = torch.empty(k_pool.shape[1], k_pool.shape[0], 2, k_pool.shape[3], dtype=k_pool.dtype,
                          device=k_pool.device)
    if mom is None:
        mom = torch.empty_like(box)
    for t in (k_pool, v_pool, box, mom):
        if not t.is_contiguous():
            raise ValueError("cache tensors must be contiguous")
    c = Cache(_DTYPES[k_pool.dtype], k_pool.shape[3], k_pool.shape[2], k_pool.shape[1],
              k_pool.shape[0], k_pool.data_ptr(), v_pool.data_ptr(), box.data_ptr(), mom.data_ptr())
    c._keep = (k_pool, v_pool, box, mom)
    c.box_t, c.mom_t = box, mom
    return c


def make_seqs(page_table, seq_lens) -> Seqs:
    """page_table: int32 [B, max_pages]; seq_lens: int32 [B] (device)."""
    if page_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("page_table and seq_lens must be int32")
    if not page_table.is_contiguous() or not seq_lens.is_contiguous():
        raise ValueError("page_table and seq_lens must be contiguous")
    _same_device(page_table, seq_lens)
    s = Seqs(page_table.data_ptr(), seq_lens.data_ptr(), page_table.shape[0], page_table.shape[1])
    s._keep, s.device_index = (page_table, seq_lens), page_table.get_device()
    return s


def q4_record_bytes(head_dim: int) -> int:
    """Bytes of a 4-bit cache's record: 16 tokens of one (page, KV head), K and V."""
    return 16 * head_dim + 128


def make_cache_q4(pool, head_dim, box=None, mom=None) -> CacheQ4:
    """Describe a 4-bit cache.  pool: uint8 [num_phys, Hkv, S/16, q4_record_bytes(head_dim)];
    box, mom: bf16 [Hkv, num_phys, 2, d] (both None: no metadata is kept).  With
    metadata, ``.meta`` is the bf16 cache description that ekv_score_pages and
    ekv_select_gauss take (they read no K)."""
    if pool.dtype != torch.uint8 or pool.dim() != 4 or pool.shape[3] != q4_record_bytes(head_dim):
        raise ValueError(f"pool must be uint8 [num_phys, Hkv, S/16, {q4_record_bytes(head_dim)}]")
    if (box is None) != (mom is None):
        raise ValueError("box and mom come together")
    for t in (box, mom):
        if t is not None and (t.dtype != torch.bfloat16
                              or tuple(t.shape) != (pool.shape[1], pool.shape[0], 2, head_dim)):
            raise ValueError("box and mom must be bf16 [Hkv, num_phys, 2, d]")
    keep = [t for t in (pool, box, mom) if t is not None]
    _same_device(*keep)
    if not all(t.is_contiguous() for t in keep):
        raise ValueError("cache tensors must be contiguous")
    ptrs = [0 if t is None else t.data_ptr() for t in (pool, box, mom)]
    c = CacheQ4(head_dim, 16 * pool.shape[2], pool.shape[1], pool.shape[0], *ptrs)
    c._keep, c.box_t, c.mom_t, c.device_index = keep, box, mom, pool.get_device()
    if box is not None:
        c.meta = Cache(EKV_BF16, head_dim, c.page_size, c.num_kv_heads, c.num_phys_pages, ptrs[0], ptrs[0], *ptrs[1:])
        c.meta._keep, c.meta.box_t, c.meta.mom_t = keep, box, mom
    return c


def make_rope(cos_sin, interleaved=False) -> Rope:
    """cos_sin: fp32 [positions, rot_dim], a row's cosines, then its sines."""
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be contiguous fp32 [positions, rot_dim]")
    r = Rope(cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], int(bool(interleaved)))
    r._keep, r.device_index = cos_sin, cos_sin.get_device()
    return r


def make_new_tokens(k, v, q=None, q_out=None, indptr=None) -> NewTokens:
    """k, v: [tokens, Hkv, d] and q: [tokens, Hq, d], rows strided as one likes,
    heads dense; q_out: dense [tokens, Hq, d]; indptr: int32 [B + 1] (None: one
    token per sequence)."""
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    if k.shape != v.shape or k.dim() != 3:
        raise ValueError("k and v must be [tokens, Hkv, d]")
    rows = [t for t in (k, v, q, q_out) if t is not None]
    for t in rows:
        if t.dtype != k.dtype or t.dtype not in _DTYPES or t.shape[0] != k.shape[0] or t.shape[2] != k.shape[2]:
            raise ValueError("q, k, v and q_out must share their type, tokens and head size")
        if t.stride(2) != 1 or (t.stride(1) != t.shape[2] and t.shape[1] > 1):
            raise ValueError("the heads of a token must be dense")
    if q is not None and (q.shape != q_out.shape or not q_out.is_contiguous()):
        raise ValueError("q_out must be dense, of q's shape")
    if indptr is not None and (indptr.dtype != torch.int32 or indptr.dim() != 1 or not indptr.is_contiguous()):
        raise ValueError("indptr must be int32 [batch + 1]")
    _same_device(*rows, *([] if indptr is None else [indptr]))
    pq = (lambda t: 0 if t is None else t.data_ptr())
    stride = (lambda t: 0 if t is None else t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2])
    n = NewTokens(pq(q), k.data_ptr(), v.data_ptr(), pq(q_out), stride(q), stride(k), stride(v), pq(indptr), k.shape[0],
                  0 if q is None else q.shape[1], _DTYPES[k.dtype])
    n._keep, n.device_index, n.heads = (rows, indptr), k.get_device(), (k.shape[1], k.shape[2])
    n.sequences = None if indptr is None else indptr.numel() - 1
    return n


def make_score_mod(softcap=0.0, slopes=None, window=0, prefix_lens=None, starts=None) -> ScoreMod:
    """How scores are capped, biased and masked (include/ekv.h, ekv_score_mod).
    slopes: fp32 [Hq]; prefix_lens, starts: int32 [B]."""
    for t, dt in ((slopes, torch.float32), (prefix_lens, torch.int32), (starts, torch.int32)):
        if t is not None and (t.dtype != dt or t.dim() != 1 or not t.is_contiguous()):
            raise ValueError("slopes must be fp32 [Hq], prefix_lens and starts int32 [batch]")
    if not 0 <= int(window or 0) < 2 ** 31:
        raise ValueError("window must be 0 (none) or a positive 32-bit number")
    keep = [t for t in (slopes, prefix_lens, starts) if t is not None]
    if keep:
        _same_device(*keep)
    ptr = (lambda t: 0 if t is None else t.data_ptr())
    m = ScoreMod(float(softcap or 0.0), int(window or 0), ptr(slopes), ptr(prefix_lens), ptr(starts))
    m._keep = (slopes, prefix_lens, starts)
    m.device_index = keep[0].get_device() if keep else None
    m.query_heads = None if slopes is None else slopes.numel()
    lens = {t.numel() for t in (prefix_lens, starts) if t is not None}
    if len(lens) > 1:
        raise ValueError("prefix_lens and starts must have one entry per sequence")
    m.sequences = lens.pop() if lens else None
    return m


def _same_device(*tensors):
    if any(t.device != tensors[0].device for t in tensors):
        raise ValueError("all tensors must be on one device")


def _on_current(device):
    """Kernels launch on the current device: another one's tensors (index −1: the
    host's) are refused."""
    if device < 0 or device != torch.cuda.current_device():
        raise ValueError(f"tensors on device {device}, which is not the current CUDA device")


def workspace(nbytes: int, device) -> torch.Tensor:
    """A 256-byte-aligned device scratch buffer of at least nbytes."""
    t = torch.empty(max(int(nbytes), 1) + 256, dtype=torch.uint8, device=device)
    off = (-t.data_ptr()) % 256
    return t[off: off + max(int(nbytes), 1)] if off else t


def ekv_workspace_bytes(op, cache, seqs, num_q_heads, cap) -> int:
    return int(lib().ekv_workspace_bytes(op, ctypes.byref(cache), ctypes.byref(seqs), num_q_heads, cap))


def ekv_build_page_meta(cache, seqs, stream=None):
    _check("ekv_build_page_meta", lib().ekv_build_page_meta(ctypes.byref(cache), ctypes.byref(seqs), _stream(stream)))


def ekv_append(cache, seqs, k_new, v_new, stream=None):
    _check("ekv_append", lib().ekv_append(ctypes.byref(cache), ctypes.byref(seqs), _ptr(k_new),
                                          _ptr(v_new), _stream(stream)))


def ekv_score_pages(cache, seqs, q, scale, ub, stream=None):
    _check("ekv_score_pages", lib().ekv_score_pages(ctypes.byref(cache), ctypes.byref(seqs), _ptr(q),
                                                    q.shape[1], scale, _ptr(ub), _stream(stream)))


def ekv_select_topk(seqs, num_kv_heads, page_size, ub, k, sel, n_sel, stream=None, *, ws=None):
    """ws: ekv_workspace_bytes(EKV_OP_SELECT_TOPK, ..., k) bytes (None when 0,
    or to select long sequences in one stage)."""
    _check("ekv_select_topk", lib().ekv_select_topk(ctypes.byref(seqs), num_kv_heads, page_size, _ptr(ub),
                                                    k, _ptr(sel), _ptr(n_sel), _ptr(ws),
                                                    0 if ws is None else ws.numel(), _stream(stream)))


def ekv_select_gauss(cache, seqs, q, scale, alpha, delta, cap, sel, n_sel, tau_hat, ws, stream=None):
    _check("ekv_select_gauss", lib().ekv_select_gauss(
        ctypes.byref(cache), ctypes.byref(seqs), _ptr(q), q.shape[1], scale, alpha, delta, cap,
        _ptr(sel), _ptr(n_sel), _ptr(tau_hat), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def ekv_entmax_decode(cache, seqs, q, scale, alpha, sel, n_sel, cap, out, ws, *, dense_v=False,
                      tau=None, support_count=None, support_bits=None, stream=None):
    _check("ekv_entmax_decode", lib().ekv_entmax_decode(
        ctypes.byref(cache), ctypes.byref(seqs), _ptr(q), q.shape[1], scale, alpha, _ptr(sel),
        _ptr(n_sel), cap, int(bool(dense_v)), _ptr(out), _ptr(tau), _ptr(support_count),
        _ptr(support_bits), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def ekv_decode_step(cache, seqs, params: StepParams, q, k_new, v_new, sel, n_sel, out, ws, *,
                    tau=None, stream=None):
    _check("ekv_decode_step", lib().ekv_decode_step(
        ctypes.byref(cache), ctypes.byref(seqs), ctypes.byref(params), _ptr(q), q.shape[1],
        _ptr(k_new), _ptr(v_new), _ptr(sel), _ptr(n_sel), _ptr(out), _ptr(tau), _ptr(ws),
        0 if ws is None else ws.numel(), _stream(stream)))


def ekv_softmax_decode(cache, seqs, q, scale, sel, n_sel, cap, out, ws, *, lse=None, stream=None):
    """Softmax decode over the selected pages (sel None: every page)."""
    _check("ekv_softmax_decode", lib().ekv_softmax_decode(
        ctypes.byref(cache), ctypes.byref(seqs), _ptr(q), q.shape[1], scale, _ptr(sel), _ptr(n_sel), cap,
        _ptr(out), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def ekv_exactness_certificate(seqs, num_kv_heads, page_size, alpha, ub, sel, n_sel, tau, certified, *,
                              stream=None):
    """certified[b, hq] = 1 when head hq's sparse output equals its full-cache one."""
    _check("ekv_exactness_certificate", lib().ekv_exactness_certificate(
        ctypes.byref(seqs), num_kv_heads, page_size, tau.shape[1], alpha, _ptr(ub), _ptr(sel), _ptr(n_sel),
        sel.shape[-1], _ptr(tau), _ptr(certified), _stream(stream)))


def ekv_decode_adaptive(cache, seqs, q, scale, alpha, k0, sel, n_sel, out, tau, certified, ws, stream=None) -> int:
    """Top-k decode whose budget doubles from k0 until every head is certified
    exact; returns the final k (sel then holds [batch, Hkv, k])."""
    k_used = ctypes.c_int32(0)
    _check("ekv_decode_adaptive", lib().ekv_decode_adaptive(
        ctypes.byref(cache), ctypes.byref(seqs), _ptr(q), q.shape[1], scale, alpha, int(k0), _ptr(sel), _ptr(n_sel),
        _ptr(out), _ptr(tau), _ptr(certified), ctypes.byref(k_used), _ptr(ws), 0 if ws is None else ws.numel(),
        _stream(stream)))
    return int(k_used.value)


def _raw_stream(stream, device):
    """The cudaStream_t of a stream, or of the current one, as an int."""
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(device)
    return torch.cuda.current_stream().cuda_stream


# the current stream's handle without a Stream object around it (1 us less)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# The serving calls run once per layer of a decode step, next to kernels of a few
# microseconds: what can be checked once is checked where the descriptions are
# made, and a call compares integers.
def _check_append(device, heads, seqs, rope, new):
    if new.device_index != device or seqs.device_index != device or (rope is not None and rope.device_index != device):
        raise ValueError("all tensors must be on one device")
    _on_current(device)
    if new.heads != heads:
        raise ValueError(f"new tokens have [Hkv, d] = {new.heads}, the cache {heads}")
    if new.sequences is not None and new.sequences != seqs.batch:
        raise ValueError("indptr must have batch + 1 entries")


def ekv_rope_append(cache, seqs, rope, new, stream=None):
    """Rotate and append new tokens (rope None: no rotation); see include/ekv.h."""
    device = cache.box_t.get_device()
    _check_append(device, (cache.num_kv_heads, cache.head_dim), seqs, rope, new)
    st = lib().ekv_rope_append(cache, seqs, rope, new, _raw_stream(stream, device))
    if st:
        raise EkvError("ekv_rope_append", st)


def ekv_rope_append_q4(cache, seqs, rope, new, stream=None):
    """ekv_rope_append into a 4-bit cache."""
    device = cache.device_index
    _check_append(device, (cache.num_kv_heads, cache.head_dim), seqs, rope, new)
    st = lib().ekv_rope_append_q4(cache, seqs, rope, new, _raw_stream(stream, device))
    if st:
        raise EkvError("ekv_rope_append_q4", st)


def ekv_q4_read(cache, seqs, indptr, k_out=None, v_out=None, stream=None):
    """Read tokens of a 4-bit cache back as values.  k_out, v_out: fp32 or bf16
    [tokens, Hkv, d], dense, either None; indptr: int32 [batch + 1], the rows of
    each sequence's last tokens."""
    out = k_out if k_out is not None else v_out
    if out is None:
        raise ValueError("k_out or v_out is needed")
    shape, dt = out.shape, _DTYPES.get(out.dtype)
    if dt is None or len(shape) != 3 or shape[1] != cache.num_kv_heads or shape[2] != cache.head_dim:
        raise ValueError("k_out and v_out must be fp32 or bf16 [tokens, Hkv, d]")
    if v_out is not None and (v_out.shape != shape or v_out.dtype != out.dtype):
        raise ValueError("k_out and v_out must be alike")
    if indptr.dtype != torch.int32 or indptr.numel() != seqs.batch + 1:
        raise ValueError("indptr must be int32 [batch + 1]")
    device = cache.device_index
    for t in (k_out, v_out, indptr):
        if t is not None and not (t.is_contiguous() and t.get_device() == device):
            raise ValueError("k_out, v_out and indptr must be dense, on the cache's device")
    if seqs.device_index != device:
        raise ValueError("all tensors must be on one device")
    _on_current(device)
    st = lib().ekv_q4_read(cache, seqs, indptr.data_ptr(), shape[0], dt, None if k_out is None else k_out.data_ptr(),
                           None if v_out is None else v_out.data_ptr(), _raw_stream(stream, device))
    if st:
        raise EkvError("ekv_q4_read", st)


def ekv_softmax_mod_workspace_bytes(head_dim, num_kv_heads, num_q_heads, num_q_tokens=1) -> int:
    return int(lib().ekv_softmax_mod_workspace_bytes(head_dim, num_kv_heads, num_q_heads, num_q_tokens))


def _softmax_mod(name, call, cache, device, seqs, q, scale, mod, sel, n_sel, cap, out, ws, lse, stream):
    shape = q.shape
    if len(shape) != 4 or q.dtype != torch.bfloat16:
        raise ValueError("q must be bf16 [batch, T, Hq, d]")
    batch, T, Hq, d = shape
    if batch != seqs.batch or d != cache.head_dim:
        raise ValueError("q does not fit the batch and the cache")
    if seqs.device_index != device:
        raise ValueError("all tensors must be on one device")
    if out.shape != shape or out.dtype != torch.float32:
        raise ValueError("out must be fp32 of q's shape")
    if lse is not None and (lse.shape != shape[:3] or lse.dtype != torch.float32):
        raise ValueError("lse must be fp32 [batch, T, Hq]")
    if sel is not None and (sel.dtype != torch.int32 or tuple(sel.shape) != (batch, cache.num_kv_heads, cap)):
        raise ValueError("sel must be int32 [batch, Hkv, cap]")
    if n_sel is not None and (n_sel.dtype != torch.int32 or n_sel.numel() != batch * cache.num_kv_heads):
        raise ValueError("n_sel must be int32 [batch, Hkv]")
    for t in (q, out, ws, lse, sel, n_sel):
        if t is not None and not (t.is_contiguous() and t.get_device() == device):
            raise ValueError("q, out, lse, sel, n_sel and ws must be dense, on the cache's device")
    if mod is not None:
        if mod.query_heads not in (None, Hq):
            raise ValueError("slopes must have one entry per query head")
        if mod.sequences not in (None, batch):
            raise ValueError("prefix_lens and starts must have one entry per sequence")
        if mod.device_index not in (None, device):
            raise ValueError("all tensors must be on one device")
    _on_current(device)
    st = call(cache, seqs, q.data_ptr(), Hq, T, scale, mod, None if sel is None else sel.data_ptr(),
              None if n_sel is None else n_sel.data_ptr(), cap, out.data_ptr(), None if lse is None else lse.data_ptr(),
              ws.data_ptr(), ws.numel(), _raw_stream(stream, device))
    if st:
        raise EkvError(name, st)


def ekv_softmax_decode_mod(cache, seqs, q, scale, mod, sel, n_sel, cap, out, ws, *, lse=None, stream=None):
    """Softmax decode with capped, biased and masked scores (mod: make_score_mod,
    or None) for the last T tokens of every sequence.  q: bf16 [B, T, Hq, d]."""
    _softmax_mod("ekv_softmax_decode_mod", lib().ekv_softmax_decode_mod, cache, cache.box_t.get_device(), seqs, q, scale,
                 mod, sel, n_sel, cap, out, ws, lse, stream)


def ekv_softmax_decode_q4(cache, seqs, q, scale, mod, sel, n_sel, cap, out, ws, *, lse=None, stream=None):
    """ekv_softmax_decode_mod over a 4-bit cache."""
    _softmax_mod("ekv_softmax_decode_q4", lib().ekv_softmax_decode_q4, cache, cache.device_index, seqs, q, scale, mod, sel,
                 n_sel, cap, out, ws, lse, stream)


def ekv_selftest_wait_timeout(polls=1024, stream=None):
    """One bounded wait that nothing satisfies: raises EKV_EFLAG_TIMEOUT."""
    _check("ekv_selftest_wait_timeout", lib().ekv_selftest_wait_timeout(polls, _stream(stream)))


def ekv_step_kernel_count(cache, seqs, params: StepParams, num_q_heads) -> int:
    """Kernels one ekv_decode_step call with these arguments enqueues."""
    return int(lib().ekv_step_kernel_count(ctypes.byref(cache), ctypes.byref(seqs), ctypes.byref(params),
                                           num_q_heads))


def ekv_entmax_decode_static_ws(cache, seqs, q, scale, alpha, sel, n_sel, cap, out, *, dense_v=False,
                                tau=None, support_count=None, support_bits=None, stream=None):
    """ekv_entmax_decode with the library's static scratch array (no workspace,
    no allocation); see include/ekv.h for its limits."""
    _check("ekv_entmax_decode_static_ws", lib().ekv_entmax_decode_static_ws(
        ctypes.byref(cache), ctypes.byref(seqs), _ptr(q), q.shape[1], scale, alpha, _ptr(sel), _ptr(n_sel),
        cap, int(bool(dense_v)), _ptr(out), _ptr(tau), _ptr(support_count), _ptr(support_bits),
        _stream(stream)))


def ekv_get_error() -> int:
    v = ctypes.c_uint32(0)
    _check("ekv_get_error", lib().ekv_get_error(ctypes.byref(v)))
    return int(v.value)
