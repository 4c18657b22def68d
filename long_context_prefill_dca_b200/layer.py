"""Convenience wrappers over the q1m C ABI: device buffers from PyTorch, calls into libq1m.

``Layer`` runs the whole chunked-prefill layer (``q1m_dca_sparse_prefill``); ``Stages`` runs
the same kernels one stage at a time (RoPE/DCA views, estimator, selection, block masks,
block-sparse attention, LSE merge) so each can be checked on its own; ``PagedCache`` serves a
ragged batch of sequences from a paged cache (append, decode, decode over a shared prefix,
prefill). Nothing here computes: tensors are allocated and pointers passed.
"""
from __future__ import annotations

from contextlib import contextmanager

import torch

from . import q1m


def _r128(x: int) -> int:
    return (x + 127) // 128 * 128


class Layer:
    def __init__(self, w, out_dtype: str = "f32", device="cuda"):
        self.w = w
        self.p = q1m.params(w, out_dtype)
        self.out_dtype = torch.bfloat16 if out_dtype == "bf16" else torch.float32
        self.ws_bytes = q1m.workspace_bytes(w.seq_len, w.n_q_heads, w.n_kv_heads, w.head_dim, self.p)
        if self.ws_bytes == 0:
            raise q1m.Q1MError("q1m_workspace_bytes", -1, "invalid shape or parameters")
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)

    def __call__(self, q, k, v, out=None, lse=None, stream=None):
        w = self.w
        if out is None:
            out = torch.empty(w.seq_len, w.n_q_heads, w.head_dim, dtype=self.out_dtype, device=q.device)
        q1m.dca_sparse_prefill(q, k, v, out, lse, w.seq_len, w.n_q_heads, w.n_kv_heads,
                               w.head_dim, self.p, self.ws, self.ws_bytes, stream)
        return out

    def chunks(self, q, k, v, first, last, out, lse=None, stream=None):
        """Prefill chunks [first, last) only, on this layer's workspace: a prefill resumed at
        chunk granularity (chunks before `first` must have run on this layer already)."""
        w = self.w
        q1m.dca_sparse_prefill_chunks(q, k, v, out, lse, w.seq_len, w.n_q_heads, w.n_kv_heads,
                                      w.head_dim, self.p, first, last, self.ws, self.ws_bytes,
                                      stream)
        return out


class HostLayer:
    """The layer from host (pinned) buffers through q1m_dca_sparse_prefill_host."""

    def __init__(self, w, out_dtype: str = "f32", device="cuda"):
        self.w = w
        self.p = q1m.params(w, out_dtype)
        self.ws_bytes = q1m.host_workspace_bytes(w.seq_len, w.n_q_heads, w.n_kv_heads, w.head_dim, self.p)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)

    def __call__(self, q_h, k_h, v_h, out_h, lse_h=None, stream=None):
        w = self.w
        q1m.dca_sparse_prefill_host(q_h, k_h, v_h, out_h, lse_h, w.seq_len, w.n_q_heads,
                                    w.n_kv_heads, w.head_dim, self.p, self.ws, self.ws_bytes, stream)
        return out_h


class Stages:
    """Buffers for running the layer stage by stage (one prefill chunk at a time)."""

    def __init__(self, w, out_dtype: str = "f32", device="cuda"):
        self.w, self.dev = w, device
        self.p = q1m.params(w, out_dtype)
        n, hq, hkv, d = w.seq_len, w.n_q_heads, w.n_kv_heads, w.head_dim
        self.ld_tokens = _r128(n)
        self.ld_rows = _r128(max(e - s0 for s0, e in q1m.prefill_bounds(w)))
        self.table = torch.empty(w.dca_chunk * d, dtype=torch.float32, device=device)
        self.k_rot = torch.zeros(hkv, self.ld_tokens, d, dtype=torch.int16, device=device)
        self.v16 = torch.zeros(hkv, self.ld_tokens, d, dtype=torch.int16, device=device)
        self.qv = torch.empty(3, hq, self.ld_rows, d, dtype=torch.int16, device=device)
        self.o_part = torch.empty(3, hq, self.ld_rows, d, dtype=torch.float32, device=device)
        self.lse_part = torch.empty(3, hq, self.ld_rows, dtype=torch.float32, device=device)
        self.attn_scratch = torch.empty(q1m.attn_scratch_bytes(0, self.ld_rows, hq, d) + 64,
                                        dtype=torch.uint8, device=device)
        q1m.rope_table(self.table, w.dca_chunk, d, w.rope_base)

    # the views are fp16 bit patterns held in int16 tensors
    @staticmethod
    def as_f16(t):
        return t.view(torch.float16)

    def keys(self, k, v, s0, e):
        w = self.w
        q1m.rope_dca_keys(k, v, s0, e, w.n_kv_heads, w.head_dim, self.p, self.table, self.k_rot,
                          self.v16, self.ld_tokens)

    def queries(self, q, s0, e):
        w = self.w
        q1m.rope_dca_queries(q, s0, e, w.n_q_heads, w.head_dim, self.p, self.table, self.qv,
                             self.ld_rows)

    def estimate(self, q, s0, e):
        w = self.w
        vert = torch.empty(w.n_q_heads, e, dtype=torch.float32, device=self.dev)
        slash = torch.empty(w.n_q_heads, e, dtype=torch.float32, device=self.dev)
        nb = q1m.vs_estimate_scratch_bytes(e, w.n_q_heads, w.n_kv_heads, w.head_dim)
        scratch = torch.empty(nb, dtype=torch.uint8, device=self.dev)
        q1m.vs_estimate(q, self.k_rot, self.ld_tokens, s0, e, w.n_q_heads, w.n_kv_heads,
                        w.head_dim, self.p, self.table, vert, slash, e, scratch, nb)
        return vert, slash

    def select(self, vert, slash, e):
        w = self.w
        nv, ns = min(w.vs_vertical, e), min(w.vs_slash, e)
        V = torch.empty(w.n_q_heads, max(nv, 1), dtype=torch.int32, device=self.dev)
        S = torch.empty(w.n_q_heads, ns, dtype=torch.int32, device=self.dev)
        q1m.vs_select(vert, slash, vert.stride(0), e, w.n_q_heads, self.p, V, S)
        return V[:, :nv], S

    def masks(self, V, S, s0, e):
        w = self.w
        nqb = (e - s0 + 127) // 128
        nkw = ((e + 127) // 128 + 31) // 32
        nv = min(w.vs_vertical, e)
        mask = torch.empty(w.n_q_heads, nqb, nkw, dtype=torch.int32, device=self.dev)
        resid = torch.empty(w.n_q_heads, nqb, max(nv, 1), dtype=torch.int32, device=self.dev)
        cnt = torch.empty(w.n_q_heads, nqb, 8, dtype=torch.int32, device=self.dev)
        Vc = V.contiguous() if nv else torch.empty(w.n_q_heads, 1, dtype=torch.int32, device=self.dev)
        q1m.vs_build_masks(Vc, S.contiguous(), s0, e, w.n_q_heads, self.p, mask, resid, cnt)
        return mask, resid[:, :, :nv] if nv else resid[:, :, :0], cnt

    def attn(self, s0, e, mask=None, resid=None, cnt=None):
        w = self.w
        if mask is not None and (resid is None or resid.shape[-1] == 0):
            resid = torch.empty(w.n_q_heads, mask.shape[1], 1, dtype=torch.int32, device=self.dev)
        q1m.block_sparse_attn(self.qv, self.ld_rows, self.k_rot, self.v16, self.ld_tokens,
                              mask, resid.contiguous() if resid is not None else None, cnt, s0, e,
                              w.n_q_heads, w.n_kv_heads, w.head_dim, self.p, self.o_part,
                              self.lse_part, self.attn_scratch, self.attn_scratch.numel())

    def merge(self, s0, e, out, lse=None):
        w = self.w
        q1m.lse_merge(self.o_part, self.lse_part, 3, self.ld_rows, s0, e, w.seq_len,
                      w.n_q_heads, w.head_dim, self.p.out_dtype, self.p, out, lse)

    def decode(self, q_tok, k_tok, v_tok, pos, out, lse=None):
        """One decode step: the token at `pos` (q [Hq][D], k, v [Hkv][D]) is appended to the
        cache and attends keys [0, pos]; out [Hq][D], lse [Hq] (natural log)."""
        w = self.w
        nb = q1m.dca_decode_scratch_bytes(w.n_q_heads, w.head_dim)
        if getattr(self, "_dec_scratch", None) is None or self._dec_scratch.numel() < nb:
            self._dec_scratch = torch.empty(nb, dtype=torch.uint8, device=self.dev)
        q1m.dca_decode(q_tok, k_tok, v_tok, pos, self.k_rot, self.v16, self.ld_tokens,
                       w.n_q_heads, w.n_kv_heads, w.head_dim, self.p, self.table, out, lse,
                       self._dec_scratch, nb)


class PagedCache:
    """A paged fp16 cache of one layer's DCA keys and values and the calls that serve a ragged
    batch from it (include/q1m.h, "Paged cache").

    w: the layer (a Workload, or any object with its fields); w.seq_len is not used.
    k_pages, v_pages: float16 [n_pages, Hkv, page_size, D], page_size 16, 32, 64 or 128.
    page_table: int32 [batch, pages], a slice of a larger table if need be: position j of sequence
    b is row j % page_size of page page_table[b, j // page_size]. Only entries of pages a call
    needs are read.
    out_dtype: "f32" (results within about 1e-6 of 64 bits; the prefill and the shared prefix take
    twice the tensor work) or "bf16" (their queries and weights are rounded to fp16).
    table: the RoPE table [dca_chunk, D / 2, 2] when the caller has one already; otherwise the
    constructor computes it and waits until it is there.

    A call serves the first len(seq_len) rows of the page table. seq_len (int32, on the device)
    holds each sequence's length with the call's tokens, which are its last; cu_tokens (int32
    [batch + 1]) the rows of ragged batches. q, k and v may be slices of a fused projection
    (any token stride that is a multiple of 8). Calls queue their work on `stream` (a
    torch.cuda.Stream; default: the current stream of the cache's device) and can be captured;
    outputs and scratch come from PyTorch's allocator on that stream. A call with stream= marks its
    tensors as used there, and its result as used on the caller's current stream, so both may be
    dropped at once; ordering the streams is the caller's (wait_stream). Device-side faults (a
    missing page, fp16 overflow) are reported by q1m.check_status()."""

    def __init__(self, w, k_pages, v_pages, page_table, out_dtype: str = "f32", table=None):
        self.w = w
        self.p = q1m.params(w, out_dtype)
        self.in_dtype = torch.bfloat16 if self.p.in_dtype == q1m.BF16 else torch.float32
        self.out_dtype = torch.bfloat16 if self.p.out_dtype == q1m.BF16 else torch.float32
        self.hq, self.hkv, self.d = w.n_q_heads, w.n_kv_heads, w.head_dim
        self.device, self.index = k_pages.device, k_pages.device.index
        if not k_pages.is_cuda:
            self._bad("__init__", "k_pages must be on a CUDA device")
        if k_pages.dim() != 4 or k_pages.shape[1] != self.hkv or k_pages.shape[3] != self.d:
            self._bad("__init__", "k_pages must be [n_pages, n_kv_heads, page_size, head_dim]")
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t.dtype != torch.float16 or t.shape != k_pages.shape or not t.is_contiguous() or t.device != self.device:
                self._bad("__init__", f"{name} must be contiguous float16 of k_pages' shape, on its device")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.desc = q1m.PagedCacheDesc(k_pages.data_ptr(), v_pages.data_ptr(), None, k_pages.shape[0], 0,
                                       k_pages.shape[2], self.hkv, self.d)
        self.set_page_table(page_table)
        if table is None:
            with self._on("__init__", None):
                table = torch.empty(w.dca_chunk, self.d // 2, 2, dtype=torch.float32, device=self.device)
                q1m.rope_table(table, w.dca_chunk, self.d, w.rope_base)
                if not torch.cuda.is_current_stream_capturing():
                    torch.cuda.current_stream().synchronize()   # the first call may come on any stream
        elif (table.dtype != torch.float32 or table.numel() < w.dca_chunk * self.d or not table.is_contiguous()
              or table.device != self.device):
            self._bad("__init__", "table must be contiguous float32 [dca_chunk, head_dim / 2, 2], on the cache's device")
        self.table = table

    def set_page_table(self, page_table):
        """Takes another page table. (A table changed in place needs no call.)"""
        t = page_table
        if t.dtype != torch.int32 or t.dim() != 2 or t.device != self.device or (t.shape[1] > 1 and t.stride(1) != 1):
            self._bad("set_page_table", "page_table must be int32 [batch, pages] with contiguous rows, on the cache's device")
        if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
            self._bad("set_page_table", "page_table rows must not overlap")
        if t.shape[1] >= 1 << 31:
            self._bad("set_page_table", "page_table is too wide")
        self.page_table, self.places = t, t.shape[0]
        self.desc.page_table = t.data_ptr()
        self.desc.table_stride = t.stride(0) if t.shape[0] > 1 else t.shape[1]
        self.desc.table_width = t.shape[1]

    def append(self, k, v, seq_len, cu_tokens=None, stream=None):
        """Writes the new tokens' keys (rotated) and values [tokens, Hkv, D] into their pages:
        one token per sequence, or the ragged batch of cu_tokens."""
        if stream is not None or torch.cuda.current_device() != self.index:
            return self._elsewhere("append", stream, lambda: self.append(k, v, seq_len, cu_tokens),
                                   k, v, seq_len, cu_tokens)
        n, batch = k.shape[0], self._batch("append", seq_len, cu_tokens)
        if v.shape[0] != n:
            self._bad("append", "k and v must have the same number of tokens")
        ks, vs = self._rows("append", "k", k, self.hkv), self._rows("append", "v", v, self.hkv)
        q1m.paged_append(k, v, ks, vs, n, cu_tokens, seq_len, batch, self.desc, self.p, self.table, self._stream())

    def decode(self, q, seq_len, window: int = 0, sinks: int = 0, out=None, lse=None, stream=None):
        """Attention of one query token per sequence, q [batch, Hq, D] at position seq_len - 1,
        over all its keys or, with a window, the last `window` and the first `sinks`.
        Returns out [batch, Hq, D]; lse (optional) is [Hq, batch]."""
        if stream is not None or torch.cuda.current_device() != self.index:
            return self._elsewhere("decode", stream, lambda: self.decode(q, seq_len, window, sinks, out, lse),
                                   q, seq_len, out, lse)
        batch = self._batch("decode", seq_len, None)
        qs = self._rows("decode", "q", q, self.hq, batch)
        out = self._outputs("decode", q, out, lse)
        nb = q1m.paged_decode_scratch_bytes(batch, self.hq, self.hkv, self.d)
        q1m.paged_decode(q, qs, seq_len, batch, window, sinks, self.desc, self.hq, self.p, self.table, out, lse,
                         self._scratch(nb), nb, self._stream())
        return out

    def decode_shared(self, q, seq_len, prefix_table, prefix_len: int, out=None, lse=None, stream=None):
        """decode() over all keys when the first prefix_len positions of every sequence are the
        pages prefix_table (int32): they are read once for the whole batch."""
        if stream is not None or torch.cuda.current_device() != self.index:
            return self._elsewhere("decode_shared", stream, lambda: self.decode_shared(q, seq_len, prefix_table, prefix_len, out, lse),
                                   q, seq_len, prefix_table, out, lse)
        batch = self._batch("decode_shared", seq_len, None)
        qs = self._rows("decode_shared", "q", q, self.hq, batch)
        self._ints("decode_shared", "prefix_table", prefix_table)
        if prefix_table.shape[0] * self.desc.page_size < prefix_len:
            self._bad("decode_shared", "prefix_table must have prefix_len / page_size entries")
        out = self._outputs("decode_shared", q, out, lse)
        nb = q1m.shared_prefix_decode_scratch_bytes(batch, prefix_len, self.hq, self.hkv, self.d, self.p)
        q1m.shared_prefix_decode(q, qs, seq_len, batch, prefix_table, prefix_len, self.desc, self.hq, self.p,
                                 self.table, out, lse, self._scratch(nb), nb, self._stream())
        return out

    def prefill(self, q, seq_len, cu_tokens, window: int = 0, sinks: int = 0, out=None, lse=None, stream=None):
        """Causal attention of a ragged batch of prompts (or prompt chunks) q [tokens, Hq, D] over
        the cache, which holds their keys already. Rows behind cu_tokens[batch] are not written."""
        if stream is not None or torch.cuda.current_device() != self.index:
            return self._elsewhere("prefill", stream, lambda: self.prefill(q, seq_len, cu_tokens, window, sinks, out, lse),
                                   q, seq_len, cu_tokens, out, lse)
        batch = self._batch("prefill", seq_len, cu_tokens)
        qs, n = self._rows("prefill", "q", q, self.hq), q.shape[0]
        out = self._outputs("prefill", q, out, lse)
        nb = q1m.paged_prefill_scratch_bytes(n, batch, self.hq, self.hkv, self.d, self.p)
        q1m.paged_prefill(q, qs, n, cu_tokens, seq_len, batch, window, sinks, self.desc, self.hq, self.p, self.table,
                          out, lse, self._scratch(nb), nb, self._stream())
        return out

    # ---- argument checks and buffers ---------------------------------------------------------
    @staticmethod
    def _bad(call, msg):
        raise q1m.Q1MError(f"PagedCache.{call}", -1, msg)

    def _ints(self, call, name, t, n=None):
        if (t.dtype is not torch.int32 or t.get_device() != self.index or t.dim() != 1 or not t.is_contiguous()
                or (n is not None and t.shape[0] != n)):
            self._bad(call, f"{name} must be contiguous int32{'' if n is None else f' [{n}]'} on the cache's device")

    def _batch(self, call, seq_len, cu_tokens):
        self._ints(call, "seq_len", seq_len)
        batch = seq_len.shape[0]
        if batch > self.places:
            self._bad(call, f"{batch} sequences, but the page table has {self.places} rows")
        if cu_tokens is not None:
            self._ints(call, "cu_tokens", cu_tokens, batch + 1)
        return batch

    def _rows(self, call, name, t, heads, rows=None):
        """Checks a [rows, heads, D] input and returns its token stride."""
        if t.dtype is not self.in_dtype or t.get_device() != self.index:
            self._bad(call, f"{name} must be {self.in_dtype} on {self.device}")
        shape, stride, d = t.shape, t.stride(), self.d
        if len(shape) != 3 or shape[1] != heads or shape[2] != d or (rows is not None and shape[0] != rows):
            self._bad(call, f"{name} must be [{'tokens' if rows is None else rows}, {heads}, {d}], not {list(shape)}")
        if stride[2] != 1 or (heads > 1 and stride[1] != d):
            self._bad(call, f"{name}'s heads must be contiguous")
        return stride[0] if shape[0] > 1 else heads * d

    def _outputs(self, call, q, out, lse):
        if out is None:
            out = torch.empty_like(q, dtype=self.out_dtype, memory_format=torch.contiguous_format)
        elif out.dtype != self.out_dtype or out.shape != q.shape or not out.is_contiguous() or out.device != self.device:
            self._bad(call, f"out must be contiguous {self.out_dtype} {list(q.shape)}")
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != (self.hq, q.shape[0])
                                or not lse.is_contiguous() or lse.device != self.device):
            self._bad(call, f"lse must be contiguous float32 [{self.hq}, {q.shape[0]}]")
        return out

    def _scratch(self, nb):
        # of the call's own: overlapping calls and captured graphs never share one
        return torch.empty(nb, dtype=torch.uint8, device=self.device)

    def _stream(self):
        return torch._C._cuda_getCurrentRawStream(self.index)

    def _elsewhere(self, call, stream, run, *tensors):
        """run() with the cache's device, and the stream a call is given, current. The memory of what
        that stream reads and writes is kept until it is done, the result's until the caller's is."""
        caller = torch.cuda.current_stream(self.device)
        with self._on(call, stream):
            out = run()
            if stream is None or stream == caller or torch.cuda.is_current_stream_capturing():
                return out
            for t in (*tensors, self.k_pages, self.v_pages, self.page_table, self.table):
                if t is not None:
                    t.record_stream(stream)
        if out is not None:
            out.record_stream(caller)
        return out

    @contextmanager
    def _on(self, call, stream):
        """Makes the cache's device, and the stream a call is given, current."""
        if stream is not None and stream.device != self.device:
            self._bad(call, f"stream is on {stream.device}, the cache on {self.device}")
        with torch.cuda.device(self.device), torch.cuda.stream(stream):
            yield
