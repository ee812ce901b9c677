"""Operators over a paged KV cache that the caller owns (include/rtp_paged.h), for torch tensors.

Argument marshalling only: every step runs in the CUDA kernels of librtp.so.  A ``PagedKV`` holds
the page tensors and the block table; lengths, weights and lists are arguments of each call.
"""
from __future__ import annotations

import contextlib
import ctypes as C
from typing import Optional

from . import RTP_EINVAL, RTP_ERANGE, RTP_ETIMEOUT, RTPError, _check, lib, rtp_paged_kv

_ERANGE, _ETIMEOUT = 2, 4  # bits of the device error word


def _dtypes():
    import torch

    return {torch.float16: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2}


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


class PagedKV:
    """A paged cache of one layer.

    k, v: [n_pages][Hkv][page_size][D] tensors (fp16, bf16 or float8_e4m3fn) with D contiguous and
    any other strides that are multiples of 16 bytes; pages laid out token by token are passed as
    ``x.transpose(1, 2)``.  block_table: int32 [n_seqs][max_pages], its rows contiguous.
    k_scale, v_scale: a key is stored * k_scale.  bounds: [n_pages][Hkv][2][D] of the pages' dtype,
    contiguous, or None: the least and greatest stored key of each page, kept by ``append`` and read
    by ``select_pages``.

    Methods are asynchronous on ``stream`` (default: the current stream of the cache's device) and
    can be captured into a CUDA graph.  Workspaces come from torch's allocator for each call.
    What only the device can see wrong (a page number outside the pool, a length outside the table)
    is left out of the result and reported by ``check()``.
    """

    def __init__(self, k, v, block_table, *, k_scale: float = 1.0, v_scale: float = 1.0, bounds=None):
        import torch

        for t, name in ((k, "k"), (v, "v"), (block_table, "block_table")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if k.dim() != 4 or tuple(v.shape) != tuple(k.shape):
            raise ValueError("k and v: expected [n_pages][Hkv][page_size][D] tensors of one shape")
        if k.dtype not in _dtypes() or v.dtype != k.dtype:
            raise ValueError("k and v: expected one of float16, bfloat16, float8_e4m3fn for both")
        if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.stride(1) != 1 and block_table.shape[1] > 1:
            raise ValueError("block_table: expected int32 [n_seqs][max_pages] with contiguous rows")
        if v.device != k.device or block_table.device != k.device:
            raise ValueError("k, v and block_table must be on one device")
        if k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("k and v: the last dimension must be contiguous")
        n_pages, hkv, ps, d = k.shape
        self.k, self.v, self.block_table, self.bounds = k, v, block_table, bounds
        self.device, self.dtype = k.device, k.dtype
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = n_pages, hkv, ps, d
        self.n_seqs, self.max_pages = block_table.shape
        self.capacity = self.max_pages * ps  # slots of a sequence
        if bounds is not None:
            self._exact(bounds, "bounds", (n_pages, hkv, 2, d), k.dtype)
        self.err = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._h = rtp_paged_kv(
            k=k.data_ptr(), v=v.data_ptr(), k_stride=(C.c_int64 * 3)(*self._strides(k)),
            v_stride=(C.c_int64 * 3)(*self._strides(v)), n_pages=n_pages, page_size=ps, n_kv_heads=hkv, head_dim=d,
            dtype=_dtypes()[k.dtype], k_scale=k_scale, v_scale=v_scale, block_table=block_table.data_ptr(),
            table_stride=block_table.stride(0) if self.n_seqs > 1 else max(1, self.max_pages),
            max_pages=self.max_pages, n_seqs=self.n_seqs, bounds=_ptr(bounds), err=self.err.data_ptr())
        self._ref = C.byref(self._h)
        self._io = (k.dtype,) if k.dtype != torch.float8_e4m3fn else (torch.float16, torch.bfloat16)
        self._codes = _dtypes()
        self._sizes = {}

    @staticmethod
    def _strides(t):
        # a dimension of one entry may carry any stride: give it that of a packed tensor
        packed = (t.shape[1] * t.shape[2] * t.shape[3], t.shape[2] * t.shape[3], t.shape[3])
        return [packed[i] if t.shape[i] == 1 else t.stride(i) for i in range(3)]

    # ------------------------------------------------------------ checks of arguments

    def _exact(self, t, name, shape, dtype):
        """A contiguous tensor of exactly this shape and dtype on the cache's device."""
        self._is(t, name, dtype)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")

    def _is(self, t, name, *dtypes):
        import torch

        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.device != self.device:
            raise ValueError(f"{name}: expected a tensor on {self.device}, got {t.device}")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: expected dtype {' or '.join(map(str, dtypes))}, got {t.dtype}")

    def _heads(self, t, name, rows=None, heads=None, dtype=None) -> int:
        """[rows][heads][D] activations with contiguous heads; returns the row stride."""
        self._is(t, name, *(self._io if dtype is None else (dtype,)))
        if t.dim() != 3 or t.shape[2] != self.head_dim or (rows is not None and t.shape[0] != rows) or (
                heads is not None and t.shape[1] != heads):
            want = [rows if rows is not None else "rows", heads if heads is not None else "heads", self.head_dim]
            raise ValueError(f"{name}: expected shape {tuple(want)}, got {tuple(t.shape)}")
        if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != self.head_dim):
            raise ValueError(f"{name}: the heads of a row must be contiguous")
        return t.stride(0) if t.shape[0] > 1 else t.shape[1] * self.head_dim

    def _queries(self, q):
        stride = self._heads(q, "q")
        if q.shape[1] < 1 or q.shape[1] % self.n_kv_heads:
            raise ValueError(f"q: {q.shape[1]} heads are no multiple of the {self.n_kv_heads} KV heads")
        return stride

    def _rows(self, q, row_len, row_seq):
        import torch

        n = q.shape[0]
        self._exact(row_len, "lengths", (n,), torch.int32)
        if row_seq is not None:
            self._exact(row_seq, "row_seq", (n,), torch.int32)
        elif n > self.n_seqs:
            raise ValueError(f"q: {n} rows for {self.n_seqs} sequences need row_seq")

    @contextlib.contextmanager
    def _elsewhere(self, stream):
        import torch

        with torch.cuda.device(self.device), torch.cuda.stream(stream):
            yield

    def _on(self, stream):
        """Work (and what it allocates) goes to `stream`, on the cache's device."""
        import torch

        if self.device.type != "cuda":
            return contextlib.nullcontext()
        if stream is not None:
            return self._elsewhere(stream)
        if torch.cuda.current_device() != self.device.index:
            return torch.cuda.device(self.device)
        return contextlib.nullcontext()

    def _handle(self) -> int:
        import torch

        if self.device.type != "cuda":
            raise ValueError(f"the cache must be on a CUDA device, not {self.device}")
        return torch.cuda.current_stream(self.device).cuda_stream

    def _workspace(self, what, *sizes):
        import torch

        n = self._sizes.get((what,) + sizes)
        if n is None:
            n = self._sizes[(what,) + sizes] = getattr(lib(), what)(self._ref, *sizes)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=self.device), n

    # ------------------------------------------------------------ operators

    def append(self, q, k, v, seq_lens, *, cu_new=None, max_new: Optional[int] = None, positions=None, q_weight=None,
               k_weight=None, eps: float = 1e-6, rope_base: float = 1.0e6, q_out=None, slot_positions=None,
               stream=None):
        """Append new tokens: norm and rotate q and k per head, write k and v to their pages.

        q: [T][Hq][D] or None; k, v: [T][Hkv][D] (rows may be slices of one projection's output).
        seq_lens: int32 [n_seqs], the lengths before the call.  cu_new: int32 [n_seqs + 1], the rows
        of each sequence (None: one token for each); max_new bounds the tokens of one sequence
        (default T).  positions: int32 [T] (default: each token's slot).  q_weight, k_weight: [D]
        norm weights in the activations' dtype (None: no norm).  slot_positions: int32
        [n_seqs][Hkv][S], receives the position of each new slot.  Returns q_out ([T][Hq][D], which
        may be q itself), or None without q.  The caller advances its lengths.
        """
        import torch

        dt = getattr(k, "dtype", None)
        ks = self._heads(k, "k", None, self.n_kv_heads)
        T = k.shape[0]
        vs = self._heads(v, "v", T, self.n_kv_heads, dt)
        self._exact(seq_lens, "seq_lens", (self.n_seqs,), torch.int32)
        if cu_new is not None:
            self._exact(cu_new, "cu_new", (self.n_seqs + 1,), torch.int32)
        elif T != self.n_seqs:
            raise ValueError(f"k: {T} tokens for {self.n_seqs} sequences need cu_new")
        if positions is not None:
            self._exact(positions, "positions", (T,), torch.int32)
        for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None:
                self._exact(w, name, (self.head_dim,), dt)
        sps = 0
        if slot_positions is not None:
            self._is(slot_positions, "slot_positions", torch.int32)
            sps = self._slots(slot_positions, "slot_positions")
        if T == 0:
            return q
        with self._on(stream):
            qs = os_ = hq = 0
            if q is not None:
                qs = self._heads(q, "q", T, None, dt)
                hq = q.shape[1]
                if q_out is None:
                    q_out = torch.empty((T, hq, self.head_dim), dtype=dt, device=self.device)
                os_ = self._heads(q_out, "q_out", T, hq, dt)
            elif q_out is not None:
                raise ValueError("q_out needs q")
            _check(lib().rtp_paged_append(
                self._ref, _ptr(q), k.data_ptr(), v.data_ptr(), self._codes[dt], qs, ks, vs, T, hq, _ptr(cu_new),
                T if max_new is None else max_new, seq_lens.data_ptr(), _ptr(positions), _ptr(q_weight),
                _ptr(k_weight), eps, rope_base, _ptr(q_out), os_, _ptr(slot_positions), sps, self._handle()))
        return q_out

    def _slots(self, t, name) -> int:
        if t.dim() != 3 or t.shape[0] != self.n_seqs or t.shape[1] != self.n_kv_heads or t.shape[2] < self.capacity:
            raise ValueError(f"{name}: expected ({self.n_seqs}, {self.n_kv_heads}, at least {self.capacity}), "
                             f"got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
        return t.shape[2]

    def update_bounds(self, seq_lens, *, stream=None) -> None:
        """Recompute the page bounds of every sequence's first seq_lens[b] slots from the stored keys."""
        import torch

        if self.bounds is None:
            raise ValueError("the cache keeps no page bounds")
        self._exact(seq_lens, "seq_lens", (self.n_seqs,), torch.int32)
        with self._on(stream):
            _check(lib().rtp_paged_bounds(self._ref, seq_lens.data_ptr(), self._handle()))

    def decode(self, q, seq_lens, *, row_seq=None, window: int = 0, n_sink: int = 0, sm_scale: float = 0.0, pages=None,
               scores=None, out=None, return_lse: bool = False, stream=None):
        """Attention of query rows over their sequences' pages.

        q: [rows][Hq][D]; row r attends to the first seq_lens[r] slots of sequence row_seq[r]
        (default: sequence r).  window > 0 keeps the last `window` slots and the first n_sink.
        pages: (indexes, counts) from ``select_pages`` keeps those pages alone.  scores: fp32
        [n_seqs][Hkv][S], to which each slot's weight, summed over the KV head's queries, is added.
        sm_scale 0: 1/sqrt(D).  Returns out ([rows][Hq][D], q's dtype) and, with return_lse, also
        the fp32 [rows][Hq] natural log-sum-exp.  A row without slots gives zeros and -inf.
        """
        import torch

        qs = self._queries(q)
        self._rows(q, seq_lens, row_seq)
        n, hq = q.shape[0], q.shape[1]
        sel = cnt = None
        ss = st = 0
        if pages is not None:
            sel, cnt = pages
            self._is(sel, "pages", torch.int32)
            if sel.dim() != 3 or sel.shape[0] != n or sel.shape[1] != self.n_kv_heads or not sel.is_contiguous():
                raise ValueError(f"pages: expected contiguous indexes [{n}][{self.n_kv_heads}][...], "
                                 f"got {tuple(sel.shape)}")
            self._exact(cnt, "page counts", (n, self.n_kv_heads), torch.int32)
            ss = sel.shape[2]
        if scores is not None:
            self._is(scores, "scores", torch.float32)
            st = self._slots(scores, "scores")
        with self._on(stream):
            if out is None:
                out = torch.empty((n, hq, self.head_dim), dtype=q.dtype, device=self.device)
            os_ = self._heads(out, "out", n, hq, q.dtype)
            lse = torch.empty((n, hq), dtype=torch.float32, device=self.device) if return_lse else None
            if n:
                ws, nb = self._workspace("rtp_paged_decode_workspace", n, hq, 0 if scores is None else 1)
                _check(lib().rtp_paged_decode(
                    self._ref, q.data_ptr(), self._codes[q.dtype], qs, n, hq, _ptr(row_seq), seq_lens.data_ptr(),
                    window, n_sink, sm_scale, _ptr(sel), _ptr(cnt), ss, out.data_ptr(), os_, _ptr(lse), _ptr(scores),
                    st, ws.data_ptr(), nb, self._handle()))
        return (out, lse) if return_lse else out

    def select_pages(self, q, seq_lens, top_pages: int, *, row_seq=None, n_first: int = 0, n_recent: int = 1,
                     stream=None):
        """The pages each row attends to: the first n_first, the last n_recent and, up to top_pages
        in all, those whose bounds allow the greatest score to any query head of a KV head.
        Returns int32 (indexes [rows][Hkv][top_pages] ascending, padded by -1; counts [rows][Hkv])."""
        import torch

        qs = self._queries(q)
        self._rows(q, seq_lens, row_seq)
        if self.bounds is None:
            raise ValueError("the cache keeps no page bounds")
        if top_pages < 1:
            raise ValueError("top_pages must be at least 1")
        n, hq = q.shape[0], q.shape[1]
        with self._on(stream):
            sel = torch.empty((n, self.n_kv_heads, top_pages), dtype=torch.int32, device=self.device)
            cnt = torch.empty((n, self.n_kv_heads), dtype=torch.int32, device=self.device)
            if n:
                ws, nb = self._workspace("rtp_paged_select_workspace", n, hq)
                _check(lib().rtp_paged_select(
                    self._ref, q.data_ptr(), self._codes[q.dtype], qs, n, hq, _ptr(row_seq), seq_lens.data_ptr(),
                    top_pages, n_first, n_recent, sel.data_ptr(), top_pages, cnt.data_ptr(), ws.data_ptr(), nb,
                    self._handle()))
        return sel, cnt

    def evict(self, seq_lens, budget: int, scores, positions, *, n_recent: int = 0, n_sink: int = 0,
              out_scores=None, out_positions=None, stream=None):
        """Bring every sequence of more than `budget` slots back to it, for each KV head by itself.

        scores: fp32, positions: int32, both [n_seqs][Hkv][S].  The first n_sink positions, the
        last n_recent and then the slots of greatest score stay (ties: the lower position); rows
        behind the budget move into the freed slots below it.  Returns (new lengths, scores,
        positions), the latter two updated in place unless out_scores / out_positions are given.
        Page bounds, where kept, are recomputed.
        """
        import torch

        self._exact(seq_lens, "seq_lens", (self.n_seqs,), torch.int32)
        self._is(scores, "scores", torch.float32)
        self._is(positions, "positions", torch.int32)
        out_scores = scores if out_scores is None else out_scores
        out_positions = positions if out_positions is None else out_positions
        self._is(out_scores, "out_scores", torch.float32)
        self._is(out_positions, "out_positions", torch.int32)
        st = self._slots(scores, "scores")
        for t, name in ((positions, "positions"), (out_scores, "out_scores"), (out_positions, "out_positions")):
            if self._slots(t, name) != st:
                raise ValueError(f"{name}: expected {st} slots, as scores have")
        with self._on(stream):
            out_len = torch.empty(self.n_seqs, dtype=torch.int32, device=self.device)
            ws, nb = self._workspace("rtp_paged_evict_workspace", st)
            _check(lib().rtp_paged_evict(
                self._ref, seq_lens.data_ptr(), budget, n_recent, n_sink, scores.data_ptr(), positions.data_ptr(), st,
                out_scores.data_ptr(), out_positions.data_ptr(), out_len.data_ptr(), ws.data_ptr(), nb,
                self._handle()))
            if self.bounds is not None:
                _check(lib().rtp_paged_bounds(self._ref, out_len.data_ptr(), self._handle()))
        return out_len, out_scores, out_positions

    def check(self, stream=None) -> None:
        """Wait for the stream; raise RTPError if a kernel met an entry out of range or gave up a wait."""
        with self._on(stream):
            w = int(self.err.item())  # ordered on the current stream, and waits for it
            if w:
                self.err.zero_()
        if w & _ETIMEOUT:
            raise RTPError(RTP_ETIMEOUT, "a bounded in-kernel wait gave up")
        if w & _ERANGE:
            raise RTPError(RTP_ERANGE, "a page, length or sequence number out of range was left out")
        if w:
            raise RTPError(RTP_EINVAL, f"unknown device error {w}")
