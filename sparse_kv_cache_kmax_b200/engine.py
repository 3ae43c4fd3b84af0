"""Decode sessions over one paged cache.

``DecodeEngine`` owns the metadata pools, the selection / output buffers and the
device workspace, and runs whole decode steps through ``ekv_decode_step`` (one
C-ABI call per step; with a rotation table two, the rotated append first).
``Q4Engine`` is the same for a cache held in 4 bits, decoded by softmax over
every page or over the top-k ones.
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import binding as B


class DecodeEngine:
    def __init__(self, k_pool, v_pool, page_table, seq_lens, num_q_heads, *, policy="topk", k=None,
                 delta=None, alpha=1.5, scale=None, cap=None, dense_v=False, cos_sin=None, interleaved=False):
        """cos_sin: fp32 [positions, rot_dim] (a position's cosines, then its
        sines): keys and queries come unrotated and are rotated on the way into
        the cache.  None: they come as they are to be used."""
        self.cache = B.make_cache(k_pool, v_pool)
        self.rope = None if cos_sin is None else B.make_rope(cos_sin, interleaved)
        self.seqs = B.make_seqs(page_table, seq_lens)
        self.device = k_pool.device
        self.Hq = int(num_q_heads)
        self.Hkv = int(k_pool.shape[1])
        self.d = int(k_pool.shape[3])
        self.S = int(k_pool.shape[2])
        self.batch = int(page_table.shape[0])
        self.max_pages = int(page_table.shape[1])
        pol = {"topk": B.EKV_POLICY_TOPK, "gauss": B.EKV_POLICY_GAUSS, "full": B.EKV_POLICY_FULL}[policy]
        if cap is None:
            cap = int(k) if policy == "topk" else self.max_pages
        self.cap = self.max_pages if policy == "full" else int(cap)
        self.params = B.StepParams(pol, int(k or 0), float(delta if delta is not None else 0.0), self.cap,
                                   float(alpha), float(scale if scale is not None else 1.0 / math.sqrt(self.d)),
                                   int(bool(dense_v)), 1)
        dev = self.device
        self.sel = torch.zeros(self.batch, self.Hkv, self.cap, dtype=torch.int32, device=dev)
        self.n_sel = torch.zeros(self.batch, self.Hkv, dtype=torch.int32, device=dev)
        self.out = torch.zeros(self.batch, self.Hq, self.d, dtype=torch.float32, device=dev)
        self.tau = torch.zeros(self.batch, self.Hq, dtype=torch.float32, device=dev)
        nbytes = B.ekv_workspace_bytes(B.EKV_OP_DECODE_STEP, self.cache, self.seqs, self.Hq, self.cap)
        if nbytes == 0:
            raise ValueError("invalid decode configuration")
        self.ws = B.workspace(nbytes, dev)
        self.scale = self.params.scale
        self.mod_bytes = {}  # scratch bytes of the masked softmax decode, by query tokens

    @property
    def box(self):
        return self.cache.box_t

    @property
    def mom(self):
        return self.cache.mom_t

    def build_meta(self, stream=None):
        B.ekv_build_page_meta(self.cache, self.seqs, stream)

    def append(self, k, v, q=None, indptr=None, stream=None):
        """Append new tokens of every sequence (seq_lens already counts them):
        k, v [tokens, Hkv, d], a sequence's rows by indptr (int32 [B + 1]; None:
        one each), rotated when the engine has a table, with the metadata of the
        pages they touch.  Returns q [tokens, Hq, d] rotated alike (q without a
        table, None without q)."""
        turn = q is not None and self.rope is not None
        with torch.cuda.stream(stream):  # memory that other streams do not take back too early
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if turn else None
        B.ekv_rope_append(self.cache, self.seqs, self.rope,
                          B.make_new_tokens(k, v, q if turn else None, out, indptr), stream)
        return out if turn else q

    def step(self, q, k_new=None, v_new=None, stream=None):
        """One decode step; appends (k_new, v_new) first when given.  With a
        rotation table, q is rotated with its token's append (a step without
        k_new takes q as rotated)."""
        self.params.append = int(k_new is not None and self.rope is None)
        if k_new is not None and self.rope is not None:
            q = self.append(k_new, v_new, q, stream=stream)
        B.ekv_decode_step(self.cache, self.seqs, self.params, q, k_new, v_new, self.sel, self.n_sel,
                          self.out, self.ws, tau=self.tau, stream=stream)
        return self.out

    def softmax(self, q, *, selected=False, stream=None, **mod):
        """Softmax decode of the last T tokens of every sequence, q [B, T, Hq, d]
        (rotated), over every page or over the last step's selection, with
        make_score_mod's options (softcap, slopes, window, prefix_lens, starts).
        Returns (out [B, T, Hq, d], lse [B, T, Hq]).  Calls on different streams do
        not disturb one another; steps share the engine's buffers and want one
        stream at a time."""
        sel, n_sel, cap = (self.sel, self.n_sel, self.cap) if selected else (None, None, self.max_pages)
        return _softmax(B.ekv_softmax_decode_mod, self, q, sel, n_sel, cap, mod, stream)

    def decode_adaptive(self, q, k_new=None, v_new=None, k0=None, stream=None):
        """Top-k decode whose budget doubles until every query head is
        certified exact (one ekv_decode_adaptive call: no unselected page can
        hold support, so the output is the full-cache one).  Appends first
        when k_new is given.  Returns (out [B, Hq, d], k used)."""
        Bsz, Hkv, P = self.batch, self.Hkv, self.max_pages
        dev = self.device
        if not hasattr(self, "_ad"):
            nbytes = B.ekv_workspace_bytes(B.EKV_OP_DECODE_ADAPTIVE, self.cache, self.seqs, self.Hq, P)
            with _on(stream):  # the zeros come first on it, and no other stream's freed memory is written
                self._ad = dict(sel=torch.empty(Bsz * Hkv * P, dtype=torch.int32, device=dev),
                                n=torch.zeros(Bsz, Hkv, dtype=torch.int32, device=dev),
                                out=torch.zeros(Bsz, self.Hq, self.d, device=dev),
                                tau=torch.zeros(Bsz, self.Hq, device=dev),
                                cert=torch.zeros(Bsz, self.Hq, dtype=torch.int32, device=dev),
                                ws=B.workspace(nbytes, dev))
        a = self._ad
        if k_new is not None and self.rope is not None:
            q = self.append(k_new, v_new, q, stream=stream)
        elif k_new is not None:
            B.ekv_append(self.cache, self.seqs, k_new, v_new, stream)
        k = B.ekv_decode_adaptive(self.cache, self.seqs, q, self.params.scale, self.params.alpha,
                                  max(1, min(int(k0 or self.params.k or 1), P)), a["sel"], a["n"], a["out"],
                                  a["tau"], a["cert"], a["ws"], stream)
        return a["out"], k


_CURRENT = contextlib.nullcontext()


def _on(stream):
    """The stream as the current one; None: the current one as it is (torch.cuda.stream(None) takes 2 us for that)."""
    return _CURRENT if stream is None else torch.cuda.stream(stream)


def _softmax(call, eng, q, sel, n_sel, cap, mod, stream):
    """One masked softmax decode with an engine's cache and scale.  The scratch is the
    call's own, on its stream: calls on two streams, or captured into two graphs,
    share none, and the allocator orders its reuse."""
    T = q.shape[1]
    nbytes = eng.mod_bytes.get(T)
    if nbytes is None:
        nbytes = B.ekv_softmax_mod_workspace_bytes(eng.d, eng.Hkv, eng.Hq, T)
        if nbytes == 0:
            raise ValueError("unsupported heads or query tokens")
        eng.mod_bytes[T] = nbytes
    with _on(stream):
        ws = B.workspace(nbytes, eng.device)
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    call(eng.cache, eng.seqs, q, eng.scale, B.make_score_mod(**mod), sel, n_sel, cap, out, ws, lse=lse, stream=stream)
    return out, lse


class Q4Engine:
    """A decode session over a cache held in 4 bits.  pool: uint8 [num_phys, Hkv,
    S/16, B.q4_record_bytes(d)] (``Q4Engine.new_pool``); the engine owns the
    metadata of its pages, so a step can pick the k pages with the largest
    bounding-box scores first.  It has metadata of the pages that its own appends
    touched: with k, a pool starts empty."""

    def __init__(self, pool, head_dim, page_table, seq_lens, num_q_heads, *, k=None, scale=None, cos_sin=None,
                 interleaved=False):
        dev = pool.device
        self.d, self.Hkv, self.S = int(head_dim), int(pool.shape[1]), 16 * int(pool.shape[2])
        self.Hq, self.device = int(num_q_heads), dev
        meta = (self.Hkv, pool.shape[0], 2, self.d)
        self.cache = B.make_cache_q4(pool, self.d, torch.zeros(meta, dtype=torch.bfloat16, device=dev),
                                     torch.zeros(meta, dtype=torch.bfloat16, device=dev))
        self.seqs = B.make_seqs(page_table, seq_lens)
        self.batch, self.max_pages = int(page_table.shape[0]), int(page_table.shape[1])
        self.scale = float(scale if scale is not None else 1.0 / math.sqrt(self.d))
        self.rope = None if cos_sin is None else B.make_rope(cos_sin, interleaved)
        self.k = None if k is None else min(int(k), self.max_pages)
        self.mod_bytes = {}
        if self.k is not None:
            self.ub = torch.empty(self.batch, self.Hkv, self.max_pages, device=dev)
            self.sel = torch.zeros(self.batch, self.Hkv, self.k, dtype=torch.int32, device=dev)
            self.n_sel = torch.zeros(self.batch, self.Hkv, dtype=torch.int32, device=dev)
            nbytes = B.ekv_workspace_bytes(B.EKV_OP_SELECT_TOPK, self.cache.meta, self.seqs, self.Hq, self.k)
            self.topk_ws = B.workspace(nbytes, dev) if nbytes else None

    @staticmethod
    def new_pool(num_pages, num_kv_heads, page_size, head_dim, device):
        return torch.zeros(num_pages, num_kv_heads, page_size // 16, B.q4_record_bytes(head_dim), dtype=torch.uint8,
                           device=device)

    def append(self, k, v, q=None, indptr=None, stream=None):
        """As DecodeEngine.append, into the 4-bit cache."""
        turn = q is not None and self.rope is not None
        with torch.cuda.stream(stream):  # memory that other streams do not take back too early
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if turn else None
        B.ekv_rope_append_q4(self.cache, self.seqs, self.rope,
                             B.make_new_tokens(k, v, q if turn else None, out, indptr), stream)
        return out if turn else q

    def select(self, q, stream=None):
        """The k pages of every KV head with the largest bounding-box scores for
        q [B, Hq, d] (rotated)."""
        if self.k is None:
            raise ValueError("the engine was made without k")
        B.ekv_score_pages(self.cache.meta, self.seqs, q, self.scale, self.ub, stream)
        B.ekv_select_topk(self.seqs, self.Hkv, self.S, self.ub, self.k, self.sel, self.n_sel, stream, ws=self.topk_ws)
        return self.sel, self.n_sel

    def softmax(self, q, *, selected=False, stream=None, **mod):
        """As DecodeEngine.softmax."""
        if selected and self.k is None:
            raise ValueError("the engine was made without k")
        sel, n_sel, cap = (self.sel, self.n_sel, self.k) if selected else (None, None, self.max_pages)
        return _softmax(B.ekv_softmax_decode_q4, self, q, sel, n_sel, cap, mod, stream)

    def step(self, q, k_new, v_new, stream=None, **mod):
        """One decode step: append, the selection (with k), softmax.  q [B, Hq, d].
        Returns (out [B, Hq, d], lse [B, Hq])."""
        q = self.append(k_new, v_new, q, stream=stream)
        if self.k is not None:
            self.select(q, stream)
        out, lse = self.softmax(q[:, None], selected=self.k is not None, stream=stream, **mod)
        return out[:, 0], lse[:, 0]

    def read(self, indptr, tokens, dtype=torch.bfloat16, stream=None):
        """The last tokens of every sequence as values: (k, v) [tokens, Hkv, d],
        rows by indptr."""
        with torch.cuda.stream(stream):  # the zeros come first on it
            k = torch.zeros(tokens, self.Hkv, self.d, dtype=dtype, device=self.device)
            v = torch.zeros_like(k)
        B.ekv_q4_read(self.cache, self.seqs, indptr, k, v, stream)
        return k, v
