"""Operators over a paged KV cache that the caller owns (include/rtp_paged.h), for torch tensors.

Argument marshalling only (csrc/paged_torch.cpp): every step runs in the CUDA kernels of librtp.so.
A ``PagedKV`` holds the page tensors and the block table; lengths, weights and lists are arguments
of each call.
"""
from __future__ import annotations

import torch  # noqa: F401  (the compiled module links to it)

from . import RTP_EINVAL, RTP_ERANGE, RTP_ETIMEOUT, RTPError

try:
    from . import _paged
except ImportError as e:
    raise ImportError("the torch binding _paged.so is missing or does not load; build it with "
                      f"`python -m long_context_sparse_idx16_b200.build` ({e})") from e

_ERANGE, _ETIMEOUT = 2, 4  # bits of the device error word


class PagedKV(_paged.PagedKV):
    """A paged cache of one layer: ``PagedKV(k, v, block_table, *, k_scale=1, v_scale=1, bounds=None)``.

    k, v: [n_pages][Hkv][page_size][D] tensors (fp16, bf16 or float8_e4m3fn) with D contiguous and
    any other strides that are multiples of 16 bytes; pages laid out token by token are passed as
    ``x.transpose(1, 2)``.  block_table: int32 [n_seqs][max_pages], its rows contiguous.
    k_scale, v_scale: a key is stored * k_scale.  bounds: [n_pages][Hkv][2][D] of the pages' dtype,
    contiguous, or None: the least and greatest stored key of each page, kept by ``append`` and read
    by ``select_pages``.

    Methods are asynchronous on ``stream`` (default: the current stream of the cache's device) and
    can be captured into a CUDA graph.  Outputs and workspaces come from torch's allocator, on that
    stream, for each call.  With a stream other than the current one, the caller makes it wait for the
    work that the inputs come from, and the current one for the results; tensors may be dropped on either
    side as soon as the call has returned.  What only the device can see wrong (a page number outside the pool, a
    length outside the table) is left out of the result and reported by ``check()``.

    append(q, k, v, seq_lens, *, cu_new=None, max_new=None, positions=None, q_weight=None,
           k_weight=None, eps=1e-6, rope_base=1e6, q_out=None, slot_positions=None, stream=None)
        Append new tokens: norm and rotate q and k per head, write k and v to their pages.
        q: [T][Hq][D] or None; k, v: [T][Hkv][D] (rows may be slices of one projection's output).
        seq_lens: int32 [n_seqs], the lengths before the call.  cu_new: int32 [n_seqs + 1], ascending
        from 0, the rows of each sequence (None: one token for each; rows behind the last are left
        alone); max_new: about the most tokens of one sequence (default T, sizes a launch).
        positions: int32 [T] (default: each token's slot).  q_weight, k_weight: [D] norm weights in
        the activations' dtype (None: no norm).  slot_positions: int32 [n_seqs][Hkv][S], receives the
        position of each new slot.  Returns q_out ([T][Hq][D], which may be q itself), or None
        without q.  The caller advances its lengths.

    decode(q, seq_lens, *, row_seq=None, window=0, n_sink=0, sm_scale=0, pages=None, scores=None,
           out=None, return_lse=False, stream=None)
        Attention of query rows over their sequences' pages.  q: [rows][Hq][D]; row r attends to the
        first seq_lens[r] slots of sequence row_seq[r] (default: sequence r).  window > 0 keeps the
        last `window` slots and the first n_sink (slots, not positions: after ``evict`` they are not
        the last tokens).  pages: (indexes, counts) from ``select_pages``
        keeps those pages alone.  scores: fp32 [n_seqs][Hkv][S], to which each slot's weight, summed
        over the KV head's queries, is added.  sm_scale 0: 1/sqrt(D).  Returns out ([rows][Hq][D],
        q's dtype) and, with return_lse, also the fp32 [rows][Hq] natural log-sum-exp.  A row
        without slots gives zeros and -inf.

    select_pages(q, seq_lens, top_pages, *, row_seq=None, n_first=0, n_recent=1, stream=None)
        The pages each row attends to: the first n_first, the last n_recent and, up to top_pages in
        all, those whose bounds allow the greatest score to any query head of a KV head.  Returns
        int32 (indexes [rows][Hkv][top_pages] ascending, padded by -1; counts [rows][Hkv]).

    evict(seq_lens, budget, scores, positions, *, n_recent=0, n_sink=0, out_scores=None,
          out_positions=None, stream=None)
        Bring every sequence of more than `budget` slots back to it, for each KV head by itself.
        scores: fp32, positions: int32, both [n_seqs][Hkv][S].  The first n_sink positions, the last
        n_recent and then the slots of greatest score stay (ties: the lower position); rows behind
        the budget move into the freed slots below it.  Returns (new lengths, scores, positions),
        the latter two updated in place unless out_scores / out_positions are given.  Page bounds,
        where kept, are recomputed.

    update_bounds(seq_lens, *, stream=None)
        Recompute the page bounds of every sequence's first seq_lens[b] slots from the stored keys.
        Sequences that share a page must use it to the same slot.
    """

    def check(self, stream=None) -> None:
        """Wait for the stream; raise RTPError if a kernel met an entry out of range or gave up a wait."""
        w = self._errors(stream)
        if w & _ETIMEOUT:
            raise RTPError(RTP_ETIMEOUT, "a bounded in-kernel wait gave up")
        if w & _ERANGE:
            raise RTPError(RTP_ERANGE, "a page, length, sequence or row number out of range was left out")
        if w:
            raise RTPError(RTP_EINVAL, f"unknown device error {w}")
