"""Plain fp64 forms of the paged-cache operators, and cases built for them.

Everything is written from the operators' definitions (include/rtp_paged.h), on the CPU, with
loops over sequences and heads.  Tolerances are derived from the roundings that the definitions
allow: half a step of the stored type, fp32 sums, 16-bit weights in the product with the values.
"""
from __future__ import annotations

import math

import numpy as np
import torch

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
#: half a step, relative
U = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8, torch.float8_e4m3fn: 2.0**-4}
#: half the step of the smallest values
TINY = {torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134, torch.float8_e4m3fn: 2.0**-10}


def f64(t) -> np.ndarray:
    t = t.detach().cpu()
    return (t.to(torch.float32) if t.dtype in DT.values() else t).double().numpy()


class Case:
    """A paged cache with shuffled pages.  Slots that no sequence uses hold NaN, unused table
    entries a number outside the pool."""

    def __init__(self, lens, *, hq, hkv, d, page, kv="fp16", q=None, nhd=False, extra=0, seed=0, k_scale=1.0,
                 v_scale=1.0, device="cuda", room=0):
        self.lens = list(lens)
        self.hq, self.hkv, self.d, self.page, self.device = hq, hkv, d, page, device
        self.kt, self.qt = DT[kv], DT[q or kv]
        self.k_scale, self.v_scale = k_scale, v_scale
        self.g = torch.Generator().manual_seed(seed)
        n = len(self.lens)
        need = [-(-(x + room) // page) for x in self.lens]
        self.width = max(1, max(need) + extra)
        pool = sum(need) + 2
        ids = torch.randperm(pool, generator=self.g).tolist()
        table = torch.full((n, self.width), -7, dtype=torch.int32)
        for b, m in enumerate(need):
            table[b, :m] = torch.tensor([ids.pop() for _ in range(m)], dtype=torch.int32)
        self.table = table
        self.pool = pool
        kk, vv = (torch.full((pool, hkv, page, d), math.nan) for _ in "kv")
        for b, m in enumerate(self.lens):
            for i in range(-(-m // page)):
                rows = min(page, m - i * page)
                p = int(table[b, i])
                kk[p, :, :rows] = self.randn(hkv, rows, d) / k_scale
                vv[p, :, :rows] = self.randn(hkv, rows, d) / v_scale
        self.k, self.v = (self.put(x, nhd) for x in (kk, vv))

    def randn(self, *shape, std=1.0):
        return torch.randn(shape, generator=self.g) * std

    def put(self, x, nhd=False):
        x = x.to(self.kt)
        if nhd:
            return x.transpose(1, 2).contiguous().to(self.device).transpose(1, 2)
        return x.to(self.device)

    def dev(self, x, dtype=None):
        x = torch.as_tensor(x)
        return x.to(self.device, dtype) if dtype is not None else x.to(self.device)

    def ints(self, x):
        return torch.tensor(list(x), dtype=torch.int32, device=self.device)

    def cache(self, **kw):
        from long_context_sparse_idx16_b200 import PagedKV

        return PagedKV(self.k, self.v, self.table.to(self.device), k_scale=self.k_scale, v_scale=self.v_scale, **kw)

    def rows64(self, b, g, slots):
        k, v = f64(self.k), f64(self.v)
        p = self.table[b].numpy()[np.asarray(slots, dtype=np.int64) // self.page]
        o = np.asarray(slots, dtype=np.int64) % self.page
        return k[p, g, o] * self.k_scale, v[p, g, o] * self.v_scale


def attend(q, k, v, scale):
    """fp64 attention of q [d] over k, v [n][d]: output, lse, weights, and sum p |v| per element."""
    z = (k @ q) * scale
    m = z.max()
    e = np.exp(z - m)
    p = e / e.sum()
    return p @ v, m + math.log(e.sum()), p, p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * scale)


def slots_seen(n, window=0, sinks=0):
    j = np.arange(n)
    return j[(j >= n - window) | (j < sinks)] if window else j


def check_decode(case: Case, q, out, lse, rows, scale=None, scores=None, before=None):
    """out (and lse, accumulated scores) against fp64.  rows: per query row, (sequence, slots per
    KV head).

    Bound per element.  Scores: products of stored values are exact in fp32, their sum of d terms is
    off by at most d 2^-23 sum |q k| (d steps of 2^-23 cover sums that truncate), so
    ds = d 2^-23 max_j scale sum |q k| + 2^-22 |s| for the scaling; a weight is then off by
    exp(2 ds) - 1 ~ 2 ds, by 2^-20 for the exponential and the joining of partial sums, and by half a
    step u_p of its 16-bit form.  A sum of n positive fp32 terms added one after another is off by at
    most n 2^-24 of itself; the terms are spread over at least 8 partial sums: sm = n / 8 * 2^-24.
    |d out| <= (u_p + 2 ds + 2^-20 + sm) (sum p |v| + |out|) + half a step of the output.  u_p is
    fp16's for fp16 and e4m3 pages and bf16's for bf16 pages."""
    scale = scale or 1.0 / math.sqrt(case.d)
    G = case.hq // case.hkv
    o, Q = f64(out), f64(q)
    up = U[torch.bfloat16] if case.kt == torch.bfloat16 else U[torch.float16]
    L = None if lse is None else f64(lse)
    for r, (b, per_head) in enumerate(rows):
        for g in range(case.hkv):
            slots = per_head[g] if isinstance(per_head, (list, tuple)) else per_head
            weights = np.zeros(0)
            ds_all = 0.0
            if len(slots):
                k, v = case.rows64(b, g, slots)
                weights = np.zeros(len(slots))
            for h in range(g * G, g * G + G):
                if not len(slots):
                    assert np.all(o[r, h] == 0.0), (r, h)
                    assert L is None or L[r, h] == -math.inf
                    continue
                want, wl, p, mag, top = attend(Q[r, h], k, v, scale)
                ds = case.d * 2.0**-23 * top + 2.0**-22 * top
                sm = len(slots) / 8 * 2.0**-24
                ds_all = max(ds_all, ds + sm)
                tol = (up + 2 * ds + 2.0**-20 + sm) * (mag + np.abs(want)) + U[out.dtype] * np.abs(want) * 1.01 + TINY[out.dtype]
                err = np.abs(o[r, h] - want)
                assert np.all(err <= tol), (r, h, float((err / tol).max()), len(slots))
                if L is not None:
                    assert abs(L[r, h] - wl) <= ds + sm + 2.0**-20 * (1 + abs(wl)), (r, h)
                weights += p
            if scores is not None:
                s, s0 = f64(scores)[r, g], f64(before)[r, g]
                want = s0.copy()
                want[slots] += weights
                tol = 2.0**-23 * np.abs(want) + 1e-30
                tol[slots] += (2 * ds_all + 2.0**-19) * weights
                assert np.all(np.abs(s - want) <= tol), (r, g, float(np.abs(s - want).max()))
                rest = np.ones(len(s), bool)
                rest[slots] = False
                assert np.array_equal(s[rest], s0[rest])


def page_choice(case: Case, bounds, q, b, n, g, top, first, recent):
    """Pages of row q ([Hq][d] fp64) for KV head g by the definition."""
    G = case.hq // case.hkv
    pages = -(-n // case.page)
    if not pages:
        return []
    lim = bounds[case.table[b, :pages].numpy(), g]
    qq = q[g * G:g * G + G]
    score = np.maximum(qq[:, None] * lim[None, :, 0], qq[:, None] * lim[None, :, 1]).sum(-1).max(0)
    must = [j < first or j >= pages - recent for j in range(pages)]
    order = sorted(range(pages), key=lambda j: (not must[j], 0.0 if must[j] else -score[j], j))
    return sorted(order[:top])


def evict_choice(scores, pos, n, budget, recent, sinks):
    """(kept slots' mask, source slot of each of the budget slots) of one sequence and KV head."""
    x, p = scores[:n], pos[:n]
    newest = p.max() if n else 0
    must = [pp < sinks or pp > newest - recent for pp in p]
    rank = [(not must[i], 0.0 if must[i] else (1, 0) if math.isnan(x[i]) else (0, -x[i]), int(p[i]), i) for i in range(n)]
    rank = [(a, (0, 0) if m else b, c, d) for (a, b, c, d), m in zip(rank, must)]
    keep = np.zeros(n, bool)
    keep[[t[3] for t in sorted(rank)[:budget]]] = True
    src = np.arange(min(n, budget))
    if n > budget:
        src[np.flatnonzero(~keep[:budget])] = budget + np.flatnonzero(keep[budget:])
    return keep, src
