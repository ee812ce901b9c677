"""Cases of the paged-cache operators: append with head norms and rotation, decode attention,
page selection with attention over the pages selected, and eviction by accumulated weight.

Each case runs in two forms on the same state: elementary torch operations in 32 bits (64 where an
angle or a comparison needs them), or the calls a user makes of the package's ``PagedKV``.
"""
import math

import numpy as np
import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"fp16": 2, "bf16": 2, "e4m3": 1}
EPS = 1e-6
ROPE_BASE = 1.0e6
K_SCALE, V_SCALE = 0.0625, 0.03125  # e4m3 pages: key = stored * K_SCALE


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one decode step of a serving batch: 64 new tokens, each behind its own cache
        dict(name="append_decode", op="append", dtype="bf16", kv="bf16", hq=32, hkv=4, d=128, page=64, seqs=64,
             tokens=64, max_len=32768, nhd=False),
        # a 16K chunk of several prompts at once, the layer's largest prefill chunk
        dict(name="append_chunk", op="append", dtype="bf16", kv="bf16", hq=32, hkv=4, d=128, page=64, seqs=5,
             tokens=16384, max_len=131072, nhd=False),
        # odd sizes into 8-bit pages laid out token by token
        dict(name="append_e4m3", op="append", dtype="fp16", kv="e4m3", hq=16, hkv=8, d=64, page=16, seqs=3,
             tokens=2999, max_len=5000, nhd=True),
        # a single short conversation: latency
        dict(name="decode_short", op="decode", dtype="fp16", kv="fp16", hq=8, hkv=2, d=128, page=64, seqs=1,
             max_len=777, ragged=False, window=0, sinks=0, nhd=False),
        # a serving batch of mixed lengths, an empty sequence among them
        dict(name="decode_ragged", op="decode", dtype="bf16", kv="bf16", hq=32, hkv=4, d=128, page=64, seqs=48,
             max_len=32768, ragged=True, window=0, sinks=0, nhd=True),
        # the repository's 128K decode workload with every head dense
        dict(name="decode_128k", op="decode", dtype="fp16", kv="fp16", hq=32, hkv=4, d=128, page=64, seqs=8,
             max_len=131072, ragged=False, window=0, sinks=0, nhd=False),
        # one sequence of 1M tokens in 8-bit pages
        dict(name="decode_1m_e4m3", op="decode", dtype="bf16", kv="e4m3", hq=32, hkv=4, d=128, page=128, seqs=1,
             max_len=1048576, ragged=False, window=0, sinks=0, nhd=False),
        # the 128K batch, attending to 64 pages a query
        dict(name="sparse_128k", op="sparse", dtype="bf16", kv="bf16", hq=32, hkv=4, d=128, page=64, seqs=8, rows=1,
             max_len=131072, ragged=False, top=64, first=1, recent=2, nhd=False),
        # one sequence of 1M tokens, ragged end
        dict(name="sparse_1m", op="sparse", dtype="bf16", kv="bf16", hq=32, hkv=4, d=128, page=64, seqs=1, rows=1,
             max_len=1048573, ragged=False, top=128, first=1, recent=2, nhd=False),
        # chunk rows of two prompts, each row with its own pages
        dict(name="sparse_rows", op="sparse", dtype="fp16", kv="fp16", hq=32, hkv=4, d=128, page=32, seqs=2, rows=500,
             max_len=32701, ragged=False, top=32, first=1, recent=4, nhd=False),
        # a decode step of a bounded cache that keeps the weights each slot has drawn
        dict(name="decode_weights", op="weights", dtype="fp16", kv="fp16", hq=32, hkv=8, d=128, page=64, seqs=16,
             max_len=8192, ragged=True, nhd=False),
        # bringing bounded caches back to their budget
        dict(name="evict", op="evict", dtype="fp16", kv="fp16", hkv=8, d=128, page=64, seqs=16, max_len=16384,
             budget=8192, recent=256, sinks=4, nhd=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "sparse", "weights", "evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8, 16])
    dtype = rng.choice(["fp16", "bf16"])
    kv = rng.choice([dtype, dtype, "e4m3"])
    c = dict(op=op, dtype=dtype, kv=kv, hq=hkv * group, hkv=hkv, d=d, page=rng.choice([16, 32, 64, 128]),
             nhd=rng.random() < 0.3)
    if op == "append":
        c["seqs"] = _log(rng, 1, 64)
        c["tokens"] = c["seqs"] if rng.random() < 0.4 else max(c["seqs"], _log(rng, 1, 12000))
        c["max_len"] = _log(rng, 16, 30000)
    elif op in ("decode", "weights"):
        c["max_len"] = _log(rng, 1, 200000 if op == "decode" else 30000)
        c["seqs"] = _log(rng, 1, max(1.0, min(128.0, 400000 / c["max_len"])))
        c["ragged"] = rng.random() < 0.7
        if op == "decode":
            c["window"] = rng.choice([0, 0, _log(rng, 1, 8192)])
            c["sinks"] = rng.choice([0, 4]) if c["window"] else 0
    elif op == "sparse":
        c["max_len"] = _log(rng, 1, 200000)
        c["seqs"] = _log(rng, 1, max(1.0, min(32.0, 400000 / c["max_len"])))
        c["rows"] = rng.choice([1, 1, 1, _log(rng, 2, 6)])
        c["ragged"] = rng.random() < 0.5
        c["first"], c["recent"] = rng.choice([0, 1]), rng.choice([1, 2])
        c["top"] = max(4, _log(rng, 4, 4096 / c["page"]))
    else:
        del c["hq"], c["dtype"]
        c["max_len"] = _log(rng, 32, 16384)
        c["seqs"] = _log(rng, 1, max(1.0, min(32.0, 131072 / c["max_len"])))
        c["recent"], c["sinks"] = _log(rng, 1, max(1.0, c["max_len"] / 16)), rng.choice([0, 4])
        c["budget"] = min(c["max_len"], c["recent"] + c["sinks"] + _log(rng, 1, c["max_len"]))
    return c


def _lens(c, r):
    """Length of each sequence's cache."""
    n, top = c["seqs"], c["max_len"]
    if c["op"] == "append":
        return r.randint(0, top + 1, n)
    if c["op"] == "evict":  # from just past the budget to the full cache; a short one now and then
        lens = r.randint(min(c["budget"], top - 1) + 1, top + 1, n)
        if n > 3:
            lens[r.randint(n)] = max(1, c["budget"] // 2)
        return lens
    if c.get("ragged"):
        lens = np.exp(r.uniform(0, math.log(top + 0.5), n)).astype(np.int64).clip(1, top)
        lens[0] = top
        if n > 4:
            lens[r.randint(1, n)] = 0
        return lens
    return np.full(n, top, dtype=np.int64)


def _new_tokens(c, r):
    """New tokens of each sequence: one each in a decode step, else a random split of the chunk."""
    n, t = c["seqs"], c["tokens"]
    if t == n:
        return np.ones(n, dtype=np.int64)
    cuts = np.sort(r.randint(0, t + 1, n - 1))
    return np.diff(np.concatenate([[0], cuts, [t]])).astype(np.int64)


def prepare(case, seed):
    c = dict(case)
    r = np.random.RandomState(1)  # the lengths are the case's, as in work(); all else is the seed's
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    lens = _lens(c, r)
    new = _new_tokens(c, r) if c["op"] == "append" else np.zeros_like(lens)
    ps, hkv, d = c["page"], c["hkv"], c["d"]
    need = -(-(lens + new) // ps)
    old = lens // ps if c["op"] == "append" else np.zeros_like(lens)  # full pages, which an append leaves alone
    width = max(1, int(need.max()))
    pool = int((need - old).sum()) + 3
    ids = np.random.RandomState(seed % (1 << 31)).permutation(pool)
    table = np.full((c["seqs"], width), -1, dtype=np.int32)
    at = 0
    for b in range(c["seqs"]):
        n = need[b] - old[b]
        table[b, :old[b]] = ids[-1]  # one page stands for all of these
        table[b, old[b]:need[b]] = ids[at:at + n]
        at += n
    scale = {"k": K_SCALE, "v": V_SCALE} if c["kv"] == "e4m3" else {"k": 1.0, "v": 1.0}

    def rows(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std)

    def pages(std, s):
        shape = (pool, ps, hkv, d) if c["nhd"] else (pool, hkv, ps, d)
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.float16).mul_(std / s).to(DT[c["kv"]])
        return x.transpose(1, 2) if c["nhd"] else x  # [pool][hkv][page][d], any strides

    s = {"case": c, "k": pages(1.0, scale["k"]), "v": pages(1.0, scale["v"]),
         "table": torch.from_numpy(table).to(dev), "scale": scale, "bounds": None,
         "lens": torch.from_numpy(lens.astype(np.int32)).to(dev)}
    if c["op"] != "evict":
        n_rows = {"append": int(new.sum()), "sparse": c["seqs"] * c.get("rows", 1)}.get(c["op"], c["seqs"])
        dt = DT[c["dtype"]]
    if c["op"] == "append":
        # q, k and v as one projection leaves them: slices of one row per token
        qkv = rows(n_rows, c["hq"] + 2 * hkv, d, std=1.5).to(dt)
        s["q"], s["kn"], s["vn"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:c["hq"] + hkv], qkv[:, c["hq"] + hkv:]
        s["qw"], s["kw"] = (1 + 0.2 * rows(d)).to(dt), (1 + 0.2 * rows(d)).to(dt)
        s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev)
        s["one_each"] = bool((new == 1).all())
        s["max_new"] = int(new.max())
        b = rows(pool, hkv, 2, d).abs().div_(scale["k"])
        b[:, :, 0].neg_()
        s["bounds"] = b.to(DT[c["kv"]])
    elif c["op"] in ("decode", "sparse", "weights"):
        s["q"] = rows(n_rows, c["hq"], d, std=2.0).to(dt)
        if c["op"] == "sparse":
            R = c["rows"]
            s["row_seq"] = torch.arange(c["seqs"], device=dev, dtype=torch.int32).repeat_interleave(R)
            # row i of a chunk sees the keys up to its own
            s["row_len"] = (s["lens"].repeat_interleave(R) - torch.arange(R - 1, -1, -1, device=dev, dtype=torch.int32)
                            .repeat(c["seqs"])).clamp(min=0).to(torch.int32)
            f = s["k"].to(torch.float16) if c["kv"] == "e4m3" else s["k"]
            s["bounds"] = torch.stack([f.amin(2), f.amax(2)], 2).to(DT[c["kv"]]).contiguous()
        if c["op"] == "weights":
            s["scores"] = rows(c["seqs"], hkv, width * ps).abs_()
    else:
        cap = width * ps
        slot = torch.arange(cap, device=dev)
        live = slot < s["lens"][:, None, None]
        # weights drawn so far: heavy-tailed, with zeros (ties) among them
        w = torch.exp(rows(c["seqs"], hkv, cap)) * (torch.rand((c["seqs"], hkv, cap), generator=g, device=dev) > 0.1)
        s["scores"] = torch.where(live, w, 0.0)
        # positions: earlier evictions left the slots out of order, some positions gone
        key = torch.rand((c["seqs"], hkv, cap), generator=g, device=dev)
        order = torch.where(live, key, 2.0).argsort(-1).argsort(-1)
        near = slot >= s["lens"][:, None, None] - c["recent"] // 2  # the newest, appended since, are in order
        pos = torch.where(near, slot.expand_as(order), 0)
        rank = torch.where(live & ~near, order.double(), 1e9).argsort(-1).argsort(-1)
        s["pos"] = torch.where(live, torch.where(near, pos, rank), -1).to(torch.int32).contiguous()
    if own:
        from long_context_sparse_idx16_b200 import PagedKV

        s["cache"] = PagedKV(s["k"], s["v"], s["table"], k_scale=scale["k"], v_scale=scale["v"], bounds=s["bounds"])
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_append(s):
    q = s["cache"].append(s["q"], s["kn"], s["vn"], s["lens"], cu_new=None if s["one_each"] else s["cu"],
                          max_new=s["max_new"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, rope_base=ROPE_BASE)
    return _appended(s, q)


def _own_decode(s):
    c = s["case"]
    out, lse = s["cache"].decode(s["q"], s["lens"], window=c["window"], n_sink=c["sinks"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_sparse(s):
    c = s["case"]
    rows = dict(row_seq=s["row_seq"]) if c["rows"] > 1 else {}
    pages, count = s["cache"].select_pages(s["q"], s["row_len"], c["top"], n_first=c["first"], n_recent=c["recent"], **rows)
    out = s["cache"].decode(s["q"], s["row_len"], pages=(pages, count), **rows)
    return {"out": out, "pages": pages, "count": count}


def _own_weights(s):
    out = s["cache"].decode(s["q"], s["lens"], scores=s["scores"])
    return {"out": out, "scores": s["scores"]}


def _own_evict(s):
    c = s["case"]
    n, scores, pos = s["cache"].evict(s["lens"], c["budget"], s["scores"], s["pos"], n_recent=c["recent"],
                                      n_sink=c["sinks"], out_scores=torch.empty_like(s["scores"]),
                                      out_positions=torch.empty_like(s["pos"]))
    return _evicted(s, n, scores, pos)


_own = {"append": _own_append, "decode": _own_decode, "sparse": _own_sparse, "weights": _own_weights, "evict": _own_evict}


def _values(x):
    """8-bit pages as the numbers they hold."""
    return x.to(torch.float16) if x.dtype == torch.float8_e4m3fn else x


def _raw(x):
    """8-bit pages as bytes, which torch can index."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _appended(s, q):
    return {"q": q, "k": _values(s["k"]), "v": _values(s["v"]), "bounds": _values(s["bounds"])}


def _evicted(s, n, scores, pos):
    return {"k": _values(s["k"]), "v": _values(s["v"]), "len": n, "scores": scores, "pos": pos}


def _round(x, dtype):
    if dtype == torch.float8_e4m3fn:
        x = x.clamp(-448.0, 448.0)
    return x.to(dtype)


def _norm_rotate(x, w, pos):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    h = x.shape[-1] // 2
    theta = ROPE_BASE ** (-torch.arange(h, device=x.device, dtype=torch.float64) / h)
    a = pos.double()[:, None] * theta
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    return torch.cat([y[..., :h] * cos - y[..., h:] * sin, y[..., h:] * cos + y[..., :h] * sin], -1)


def _plain_append(s):
    c, ps = s["case"], s["case"]["page"]
    dt = s["k"].dtype
    t = torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:], t, right=True)
    slot = s["lens"][seq].long() + (t - s["cu"][seq]).long()
    page, off = s["table"][seq, slot // ps].long(), slot % ps
    q = _norm_rotate(s["q"], s["qw"], slot).to(s["q"].dtype)
    k = _round(_norm_rotate(s["kn"], s["kw"], slot) / s["scale"]["k"], dt)
    _raw(s["k"])[page, :, off] = _raw(k)
    _raw(s["v"])[page, :, off] = _raw(_round(s["vn"].float() / s["scale"]["v"], dt))
    # bounds: a page begun in this call starts from its new rows alone
    lo, hi = s["bounds"][:, :, 0].float(), s["bounds"][:, :, 1].float()
    touched = torch.zeros(lo.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)[:, None, None]
    begun = torch.zeros(lo.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page[off == 0], True)[:, None, None]
    at = page[:, None, None].expand(-1, c["hkv"], c["d"])
    nlo = torch.where(begun, math.inf, lo).scatter_reduce(0, at, k.float(), "amin")
    nhi = torch.where(begun, -math.inf, hi).scatter_reduce(0, at, k.float(), "amax")
    s["bounds"][:, :, 0] = torch.where(touched, nlo, lo).to(dt)
    s["bounds"][:, :, 1] = torch.where(touched, nhi, hi).to(dt)
    return _appended(s, q)


def _gathered(x, table, scale):
    """Pages of each table row as [row][hkv][slot][d] in 32 bits."""
    y = _raw(x)[table.clamp(min=0).long()].view(x.dtype).float() * scale  # [..., pages, hkv, page, d]
    return y.transpose(1, 2).flatten(2, 3)


def _attend(q, k, v, seen):
    """Attention weights, outputs and log-sum-exp; q [..., g, d], k, v [..., n, d], seen [..., 1, n]."""
    z = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(z - torch.where(m.isinf(), 0.0, m)), 0.0)
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    return p, p @ v, (m + torch.log(total)).squeeze(-1)


def _dense(s, window=0, sinks=0):
    c = s["case"]
    q = s["q"].float().view(c["seqs"], c["hkv"], -1, c["d"])
    k, v = _gathered(s["k"], s["table"], s["scale"]["k"]), _gathered(s["v"], s["table"], s["scale"]["v"])
    j = torch.arange(k.shape[2], device="cuda")
    n = s["lens"].long()[:, None, None, None]
    seen = j < n
    if window:
        seen = seen & ((j >= n - window) | (j < sinks))
    return _attend(q, k, v, seen) + (seen,)


def _plain_decode(s):
    p, o, lse, _ = _dense(s, s["case"]["window"], s["case"]["sinks"])
    return {"out": o.reshape(s["q"].shape).to(s["q"].dtype), "lse": lse.reshape(s["q"].shape[:2])}


def _plain_weights(s):
    p, o, lse, seen = _dense(s)
    s["scores"] += p.sum(2)
    return {"out": o.reshape(s["q"].shape).to(s["q"].dtype), "scores": s["scores"]}


def _plain_sparse(s):
    c, ps = s["case"], s["case"]["page"]
    S, R, H, D = c["seqs"], c["rows"], c["hkv"], c["d"]
    q = s["q"].view(S, R, H, -1, D)
    b = _values(s["bounds"])[s["table"].clamp(min=0).long()].double()
    b = b.permute(0, 2, 3, 4, 1)  # [S][H][2][D][pages]
    qd = q.double().permute(0, 2, 1, 3, 4).flatten(2, 3)  # [S][H][R*G][D]
    score = qd.clamp(max=0) @ b[:, :, 0] + qd.clamp(min=0) @ b[:, :, 1]
    score = score.view(S, H, R, -1, score.shape[-1]).amax(3).transpose(1, 2)  # [S][R][H][pages]
    j = torch.arange(score.shape[-1], device="cuda")
    n = s["row_len"].long().view(S, R, 1, 1)
    np_ = (n + ps - 1) // ps
    score = torch.where((j < c["first"]) | (j >= np_ - c["recent"]), math.inf, score)
    score = torch.where(j < np_, score, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :c["top"]]
    taken = torch.arange(order.shape[-1], device="cuda") < np_
    pages = torch.where(taken, order, 1 << 30).sort(-1).values
    pages = torch.where(pages < (1 << 30), pages, -1)
    if pages.shape[-1] < c["top"]:
        pages = torch.nn.functional.pad(pages, (0, c["top"] - pages.shape[-1]), value=-1)
    count = np_.squeeze(-1).clamp(max=c["top"]).expand(S, R, H)
    phys = s["table"].long().clamp(min=0)[torch.arange(S, device="cuda").view(-1, 1, 1, 1), pages.clamp(min=0)]
    h = torch.arange(H, device="cuda").view(1, 1, -1, 1)
    k, v = (_raw(s[x])[phys, h].view(s[x].dtype).float().flatten(3, 4) * s["scale"][x] for x in "kv")  # [S][R][H][slots][D]
    at = pages.unsqueeze(-1) * ps + torch.arange(ps, device="cuda")
    seen = ((pages.unsqueeze(-1) >= 0) & (at < n.unsqueeze(-1))).flatten(3, 4).unsqueeze(3)
    _, o, _ = _attend(q.float(), k, v, seen)
    return {"out": o.reshape(s["q"].shape).to(s["q"].dtype), "pages": pages.reshape(S * R, H, -1).to(torch.int32),
            "count": count.reshape(S * R, H).to(torch.int32)}


def _plain_evict(s):
    c, ps = s["case"], s["case"]["page"]
    scores, pos = s["scores"], s["pos"]
    cap = scores.shape[-1]
    slot = torch.arange(cap, device="cuda").expand_as(scores)
    n = s["lens"].long()[:, None, None]
    keep_n = n.clamp(max=c["budget"])
    live = slot < n
    newest = torch.where(live, pos, -1).amax(-1, keepdim=True)
    kept_first = live & ((pos > newest - c["recent"]) | (pos < c["sinks"]))
    key = torch.where(kept_first, math.inf, torch.where(live, scores, -math.inf))
    by_pos = torch.where(live, pos, 1 << 30).sort(dim=-1, stable=True).indices
    order = by_pos.gather(-1, key.gather(-1, by_pos).sort(dim=-1, descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(-1, order, slot)
    kept = live & (rank < keep_n)
    hole, mover = ~kept & (slot < keep_n), kept & (slot >= keep_n)
    movers = torch.where(mover, slot, 1 << 30).sort(-1).values
    src = torch.where(hole, movers.gather(-1, (hole.long().cumsum(-1) - 1).clamp(min=0)), slot)
    b, h, dst = hole.nonzero(as_tuple=True)
    frm = src[b, h, dst]
    to_page, from_page = s["table"][b, dst // ps].long(), s["table"][b, frm // ps].long()
    for x in (_raw(s["k"]), _raw(s["v"])):
        x[to_page, h, dst % ps] = x[from_page, h, frm % ps]
    rest = slot >= keep_n
    src = src.clamp(max=cap - 1)
    return _evicted(s, keep_n.flatten().to(torch.int32), torch.where(rest, 0.0, scores.gather(-1, src)),
                    torch.where(rest, -1, pos.gather(-1, src)))


_plain = {"append": _plain_append, "decode": _plain_decode, "sparse": _plain_sparse, "weights": _plain_weights, "evict": _plain_evict}


# ---------------------------------------------------------------- work


def work(case):
    c, es = dict(case), SIZE[case["kv"]]
    r = np.random.RandomState(1)
    lens, d, hkv, ps = _lens(c, r), c["d"], c["hkv"], c["page"]
    if c["op"] == "append":
        t = c["tokens"]
        touched = min(t, t // ps + c["seqs"])
        return {"bytes": t * d * (2 * 2 * c["hq"] + (2 + es) * 2 * hkv) + touched * hkv * 2 * d * es,
                "flops": t * d * (8 * c["hq"] + 8 * hkv)}
    if c["op"] == "evict":
        over = np.maximum(lens - c["budget"], 0)
        # of the slots past the budget, the newest stay and of the others as many as the budget's share
        stay = np.where(over > 0, np.minimum(over, c["recent"] // 2 + over * c["budget"] / np.maximum(lens, 1)), 0)
        cap = -(-int(lens.max()) // ps) * ps
        return {"bytes": hkv * (float(stay.sum()) * d * 4 * es + float(lens.sum()) * 8 + c["seqs"] * cap * 8),
                "flops": hkv * float(lens.sum())}
    hq = c["hq"]
    if c["op"] == "sparse":
        n = np.repeat(lens, c["rows"])
        pages = -(-n // ps)
        keys = np.minimum(pages, c["top"]) * ps
        # rows of one sequence share its bounds and, at most, all its pages
        b = float((-(-lens // ps)).sum()) * hkv * 2 * d * es
        kv = float(np.minimum(keys.reshape(len(lens), -1).sum(1), lens).sum()) * hkv * 2 * d * es
        return {"bytes": b + kv + len(n) * hq * d * 4 + len(n) * hkv * c["top"] * 4,
                "flops": 4.0 * hq * d * float(np.minimum(keys, n).sum()) + 4.0 * hq * d * float(pages.sum())}
    if c.get("window"):
        lens = np.minimum(lens, c["window"] + c["sinks"])
    keys = float(lens.sum())
    w = {"bytes": keys * hkv * 2 * d * es + c["seqs"] * hq * (d * 4 + 4), "flops": 4.0 * hq * d * keys}
    if c["op"] == "weights":
        w["bytes"] += keys * hkv * 8
    return w


# ---------------------------------------------------------------- in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "decode": _exact_decode, "weights": _exact_decode, "sparse": _exact_sparse,
            "evict": _exact_evict}[case["op"]](s)


def _wide(x):
    return _values(x).double()


def _exact_append(s):
    c, ps, d = s["case"], s["case"]["page"], s["case"]["d"]
    k, v, bounds = _wide(s["k"]), _wide(s["v"]), _wide(s["bounds"])
    q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens, cu, table = s["lens"].tolist(), s["cu"].tolist(), s["table"].tolist()
    freq = torch.tensor([ROPE_BASE ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device="cuda")

    def turn(x, w, pos):
        x = x.double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * w.double()
        z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * torch.polar(torch.ones_like(freq), pos[:, None] * freq)[:, None]
        return torch.cat([z.real, z.imag], -1)

    top = 448.0 if c["kv"] == "e4m3" else math.inf
    for b in range(c["seqs"]):
        first, n = lens[b], cu[b + 1] - cu[b]
        pos = torch.arange(first, first + n, device="cuda", dtype=torch.float64)
        rows = slice(cu[b], cu[b + 1])
        q_out[rows] = turn(s["q"][rows], s["qw"], pos)
        kn = (turn(s["kn"][rows], s["kw"], pos) / s["scale"]["k"]).clamp(-top, top)
        vn = (s["vn"][rows].double() / s["scale"]["v"]).clamp(-top, top)
        if c["kv"] == "e4m3":  # the definition stores the nearest 8-bit value
            kn, vn = _wide(kn.to(torch.float8_e4m3fn)), _wide(vn.to(torch.float8_e4m3fn))
        at = first
        while at < first + n:
            stop = min(first + n, (at // ps + 1) * ps)
            page = table[b][at // ps]
            part = kn[at - first:stop - first].transpose(0, 1)  # [hkv][slots][d]
            k[page, :, at % ps:at % ps + stop - at] = part
            v[page, :, at % ps:at % ps + stop - at] = vn[at - first:stop - first].transpose(0, 1)
            lo, hi = part.amin(1), part.amax(1)
            if at % ps:
                lo, hi = torch.minimum(lo, bounds[page, :, 0]), torch.maximum(hi, bounds[page, :, 1])
            bounds[page, :, 0], bounds[page, :, 1] = lo, hi
            at = stop
    return {"q": q_out, "k": k, "v": v, "bounds": bounds}


def _rows64(s, b, h, slots):
    ps = s["case"]["page"]
    page = s["table"][b].long()[slots // ps]
    return tuple(_wide(_raw(s[x])[page, h, slots % ps].view(s[x].dtype)) * s["scale"][x] for x in "kv")


def _softmax64(q, k, v):
    z = q.double() @ k.T * (q.shape[-1] ** -0.5)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[:, None])
    return p, p @ v, lse


def _exact_decode(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    scores = s["scores"].double() if c["op"] == "weights" else None
    for b, n in enumerate(s["lens"].tolist()):
        slots = torch.arange(n, device="cuda")
        if c.get("window"):
            slots = slots[(slots >= n - c["window"]) | (slots < c["sinks"])]
        if not len(slots):
            continue
        for h in range(c["hkv"]):
            p, out[b, h * g:h * g + g], lse[b, h * g:h * g + g] = _softmax64(s["q"][b, h * g:h * g + g], *_rows64(s, b, h, slots))
            if scores is not None:
                scores[b, h, :n] += p.sum(0)
    return {"out": out, "lse": lse} if scores is None else {"out": out, "scores": scores}


def _exact_sparse(s):
    c, ps = s["case"], s["case"]["page"]
    n_rows, g = s["q"].shape[0], c["hq"] // c["hkv"]
    if n_rows * c["hkv"] > 5000:  # a larger chunk would take too long row by row
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    seqs, lens = s["row_seq"].tolist(), s["row_len"].tolist()
    pages_out = torch.full((n_rows, c["hkv"], c["top"]), -1, dtype=torch.int32)
    count = torch.zeros((n_rows, c["hkv"]), dtype=torch.int32)
    for r in range(n_rows):
        b, n = seqs[r], lens[r]
        pages = -(-n // ps)
        if not pages:
            continue
        phys = s["table"][b, :pages].long()
        for h in range(c["hkv"]):
            lim = _wide(_raw(s["bounds"])[phys, h].view(s["bounds"].dtype))  # [pages][2][d]
            q = s["q"][r, h * g:h * g + g].double()
            score = torch.maximum(q[:, None] * lim[None, :, 0], q[:, None] * lim[None, :, 1]).sum(-1).amax(0)
            must = set(range(min(c["first"], pages))) | set(range(max(0, pages - c["recent"]), pages))
            val = score.tolist()
            take = sorted(range(pages), key=lambda j: (j not in must, 0 if j in must else -val[j], j))[:c["top"]]
            take.sort()
            pages_out[r, h, :len(take)] = torch.tensor(take, dtype=torch.int32)
            count[r, h] = len(take)
            slots = (torch.tensor(take, device="cuda")[:, None] * ps + torch.arange(ps, device="cuda")).flatten()
            _, out[r, h * g:h * g + g], _ = _softmax64(s["q"][r, h * g:h * g + g], *_rows64(s, b, h, slots[slots < n]))
    return {"out": out, "pages": pages_out, "count": count}


def _exact_evict(s):
    # nothing is computed here but comparisons: the wanted rows are the given ones, moved
    c, ps = s["case"], s["case"]["page"]
    k, v = _wide(s["k"]), _wide(s["v"])
    sc, ps_all = s["scores"].cpu().numpy().astype(np.float64), s["pos"].cpu().numpy()
    table, lens = s["table"].cpu().numpy(), s["lens"].tolist()
    new_sc, new_pos = np.zeros_like(sc), np.full_like(ps_all, -1)
    for b, n in enumerate(lens):
        for h in range(c["hkv"]):
            x, p = sc[b, h, :n], ps_all[b, h, :n]
            if n <= c["budget"]:
                new_sc[b, h, :n], new_pos[b, h, :n] = x, p
                continue
            first = (p > p.max() - c["recent"]) | (p < c["sinks"])
            order = np.lexsort((p, np.where(first, 0, -x), ~first))
            kept = np.zeros(n, bool)
            kept[order[:c["budget"]]] = True
            dst = np.flatnonzero(~kept[:c["budget"]])
            src = c["budget"] + np.flatnonzero(kept[c["budget"]:])
            frm = np.arange(c["budget"])
            frm[dst] = src
            new_sc[b, h, :c["budget"]], new_pos[b, h, :c["budget"]] = x[frm], p[frm]
            if len(dst):
                tp, fp = (torch.from_numpy(table[b][i // ps].astype(np.int64)).cuda() for i in (dst, src))
                to, fo = torch.from_numpy(dst % ps).cuda(), torch.from_numpy(src % ps).cuda()
                k[tp, h, to] = k[fp, h, fo]
                v[tp, h, to] = v[fp, h, fo]
    return {"k": k, "v": v, "len": None, "scores": torch.from_numpy(new_sc), "pos": None}
