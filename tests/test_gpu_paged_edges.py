"""Paged-cache operators on the GPU at the edges of what their arguments allow, against the
definitions in fp64 (tests/paged_ref.py)."""
import math

import numpy as np
import pytest
import torch

from paged_ref import TINY, U, Case, check_decode, f64

pytestmark = pytest.mark.gpu

TYPES = [("fp16", "fp16"), ("bf16", "bf16"), ("e4m3", "fp16"), ("e4m3", "bf16")]


# ---------------------------------------------------------------- scores far from zero


def far_scores(kv, q, z, other, n, where, seed):
    """One sequence of n keys and one KV head of two query heads whose base-2 scores are known to the
    last bit: `z` at the slots `where[0]`, `other` at where[1], far below both everywhere else.  Every
    product and sum behind them is a small multiple of a power of two, exact in fp32 (terms further than
    2^-22 from one another do not meet).  Values are random.  Returns the case, the queries and sm_scale."""
    c = Case([n], hq=2, hkv=1, d=64, page=64, kv=kv, q=q, seed=seed, k_scale=2.0**6 if kv == "e4m3" else 1.0)
    # scores: q0 k0 + 2 k1, times k_scale.  e4m3 keys are at most 448, and multiples of 2^-9
    q0 = 2.0**13 if abs(z) > 2**20 else 8.0
    queries = torch.zeros(1, 2, 64)
    queries[..., 0], queries[..., 1] = q0, 2.0
    top = math.copysign(2.0 ** math.floor(math.log2(abs(z))), z)  # the part of the score that dim 0 makes
    k = torch.zeros(n, 64)
    k[:, 0], k[:, 1] = top / q0 / c.k_scale, -192.0  # far below the others in base 2
    for slots, s in zip(where, (z, other)):
        k[slots, 1] = (s - top) / 2.0 / c.k_scale
    assert torch.equal(k.to(c.kt).float(), k)
    pages = torch.zeros(c.pool, 1, 64, 64)
    for i in range(-(-n // 64)):
        rows = k[i * 64:(i + 1) * 64]
        pages[int(c.table[0, i]), 0, :len(rows)] = rows
    c.k = c.put(pages)
    # sm_scale * log2(e) = 1 to fp32's last bit
    sm = float(np.float32(math.log(2.0)))
    assert np.float32(sm * float(np.float32(c.k_scale)) * 1.4426950408889634) == np.float32(c.k_scale)
    return c, queries.to(c.qt).to(c.device), sm


FAR = [(2**24 + 20, 2**24 + 16), (2**25 + 8, 2**25), (2**26 + 16, 2**26 + 16), (2**27 + 32, 2**27 + 32),
       (-(2**24) - 4, -(2**24) - 8), (-(2**25) - 8, -(2**25) - 16), (-(2**27) - 32, -(2**27) - 32), (100, 96)]


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("z,other", FAR)
@pytest.mark.parametrize("n", [200, 20000])
def test_decode_of_far_scores(kv, q, z, other, n):
    """Finite scores, however large, give the weights that their differences say: here 1 and
    2^(other - z), exactly, so that only the exponential (2^-21 with the sums) and the output round."""
    where = [[7], [n - 3]]
    c, x, sm = far_scores(kv, q, z, other, n, where, 1)
    out, lse = c.cache().decode(x, c.ints([n]), sm_scale=sm, return_lse=True)
    _, v = c.rows64(0, 0, np.arange(n))
    p = np.zeros(n)
    p[where[0]], p[where[1]] = 1.0, 2.0 ** (other - z)
    want = p @ v / p.sum()
    # (weights below 2^-24 of the largest are 0 in bf16 as in exact sums rounded to the output)
    tol = U[c.qt] * np.abs(want) * 1.01 + 2.0**-20 * (p @ np.abs(v)) + TINY[c.qt]
    for h in range(2):
        assert np.all(np.abs(f64(out)[0, h] - want) <= tol), (h, f64(out)[0, h, :4], want[:4])
        natural = (z + math.log2(p.sum())) * math.log(2.0)
        assert abs(float(lse[0, h]) - natural) <= 2.0**-22 * abs(natural) + 2.0**-20


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("z,other", FAR)
@pytest.mark.parametrize("n", [200, 20000])
def test_accumulated_weights_of_far_scores(kv, q, z, other, n):
    """The weights added up are those of the softmax: they sum to the number of query heads, at scores
    beside which the logarithm of their sum is below fp32's last bit."""
    where = [[7, 100], [n - 3]]
    c, x, sm = far_scores(kv, q, z, other, n, where, 2)
    kvc = c.cache()
    scores = torch.zeros((1, 1, kvc.capacity), device=c.device)
    kvc.decode(x, c.ints([n]), sm_scale=sm, scores=scores)
    p = np.zeros(kvc.capacity)
    p[where[0]], p[where[1]] = 1.0, 2.0 ** (other - z)
    want = 2 * p / p.sum()
    # the exponential, the logarithm of the sum (at most 2) and the sum of two heads; the exponent's rounding
    tol = (2.0**-20 + 2.0**-24 * (z - other + 2)) * want
    assert np.all(np.abs(f64(scores)[0, 0] - want) <= tol), (f64(scores)[0, 0][[7, 100, n - 3]], want[[7, 100, n - 3]])


@pytest.mark.parametrize("kv,q", [("fp16", "fp16"), ("e4m3", "fp16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("gap", [18.0, 20.0])
def test_small_weights_make_the_output(kv, q, gap):
    """The one key that carries nearly all the weight has a value of zero: what is left are 39999 keys
    of weights e^-18 and e^-20, which fp16 would round to 0 or to one step without their factor 2^15."""
    n = 40000
    c = Case([n], hq=4, hkv=1, d=64, page=64, kv=kv, q=q, seed=9)
    x = torch.zeros(1, 4, 64, dtype=c.qt, device=c.device)
    x[..., 0] = 8.0
    k, v = torch.zeros(c.pool, 1, 64, 64), torch.ones(c.pool, 1, 64, 64)
    v += torch.arange(64) / 64 * (kv == "fp16")
    at = int(c.table[0, 300])
    k[at, 0, 11, 0], v[at, 0, 11] = gap, 0.0
    c.k, c.v = c.put(k), c.put(v)
    out, lse = c.cache().decode(x, c.ints([n]), sm_scale=0.125, return_lse=True)
    check_decode(c, x, out, lse, [(0, np.arange(n))], scale=0.125)
    assert float(out.float().min()) > 0.5 * (n - 1) * math.exp(-gap)


# ---------------------------------------------------------------- e4m3 pages under queries of any size


@pytest.mark.parametrize("top", [2.0**127, 2.0**126, 2.0**-113, 2.0**-125])
def test_e4m3_queries_at_the_ends_of_bf16(top):
    """bf16 queries whose largest value has the greatest exponents there are, or the least: their
    products with the keys are in fp32's range, so the scores are finite and count."""
    c = Case([300], hq=2, hkv=1, d=64, page=64, kv="e4m3", q="bf16", seed=5, k_scale=2.0**-60 if top > 1 else 2.0**60)
    r = c.randn(c.pool, 1, 64, 64).sign()
    at = -9 if top > 1 else 4  # stored keys: the least there are, or large ones
    k = torch.where(torch.arange(64) < 2, r * 2.0 ** torch.randint(at, at + 4, r.shape, generator=c.g), 0.0)
    c.k, c.v = c.put(k), c.put(c.randn(c.pool, 1, 64, 64))
    x = torch.zeros(1, 2, 64)
    x[..., 0], x[..., 1] = top, top / 2
    x = x.to(c.qt).to(c.device)
    sm = 1.0 / (float(x.max()) * c.k_scale * 2.0 ** (at + 2))  # scores of up to a few units
    out, lse = c.cache().decode(x, c.ints([300]), sm_scale=sm, return_lse=True)
    check_decode(c, x, out, lse, [(0, np.arange(300))], scale=float(np.float32(sm)))


# ---------------------------------------------------------------- append


def rotated(x, w, pos, eps, base):
    """fp64 norm and rotation of [T][H][d], and the magnitude that its rounding errors scale with."""
    d = x.shape[-1]
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    a = np.asarray(pos, dtype=np.float64)[:, None, None] * base ** (-2.0 * np.arange(d // 2) / d)
    y0, y1 = y[..., :d // 2], y[..., d // 2:]
    mag = np.abs(y0) + np.abs(y1)
    return np.concatenate([y0 * np.cos(a) - y1 * np.sin(a), y1 * np.cos(a) + y0 * np.sin(a)], -1), np.concatenate([mag, mag], -1)


def close(got, want, mag, dtype, what):
    """Half a step of the stored type, and 2^-19 of |y0| + |y1| for the fp32 arithmetic before it: the
    norm's sum of d squares, root and products (2^-20), sine and cosine (reduced angle to 2^-24 pi,
    two steps of sincosf)."""
    tol = U[dtype] * np.abs(want) * 1.01 + 2.0**-19 * mag + TINY[dtype]
    err = np.abs(got - want)
    assert np.all(err <= tol), (what, float((err / tol).max()))


def check_append(kv, q, d, page, new, hq, hkv, lens, norm="qk", give_q=True, in_place=False, seed=0):
    """A chunk of new[b] tokens for each sequence, all that it writes against the definition, and the
    rest of the pages left as they were."""
    c = Case(lens, hq=hq, hkv=hkv, d=d, page=page, kv=kv, q=q, room=max(new) + 1, seed=seed,
             **(dict(k_scale=0.0625, v_scale=0.03125) if kv == "e4m3" else {}))
    T, eps, base = sum(new), 1e-5, 1e4
    qkv = c.randn(T, hq + 2 * hkv, d, std=1.5).to(c.qt).to(c.device)
    qn, kn, vn = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    q64, k64 = f64(qn), f64(kn)
    w = {x: (1 + 0.2 * c.randn(d)).to(c.qt).to(c.device) if x in norm else None for x in "qk"}
    bounds = torch.zeros((c.pool, hkv, 2, d), device=c.device).to(c.kt)
    slots = torch.full((len(lens), hkv, c.width * page), -1, dtype=torch.int32, device=c.device)
    old = {x: f64(getattr(c, x)) for x in "kv"}
    cache = c.cache(bounds=bounds)
    cache.update_bounds(c.ints(lens))
    cu = np.concatenate([[0], np.cumsum(new)])
    out = cache.append(qn if give_q else None, kn, vn, c.ints(lens), cu_new=c.ints(cu), max_new=max(new), q_weight=w["q"],
                       k_weight=w["k"], eps=eps, rope_base=base, q_out=qn if in_place else None, slot_positions=slots)
    cache.check()
    seq = np.repeat(np.arange(len(new)), new)
    pos = np.asarray(lens)[seq] + np.arange(T) - cu[seq]
    if give_q:
        assert out is qn or not in_place
        want, mag = rotated(q64, None if w["q"] is None else f64(w["q"]), pos, eps, base)
        close(f64(out), want, mag, c.qt, "q")
    else:
        assert out is None
    want, mag = rotated(k64, None if w["k"] is None else f64(w["k"]), pos, eps, base)
    p, o = c.table.numpy()[seq, pos // page], pos % page
    got = {x: f64(getattr(c, x)) for x in "kv"}
    close(got["k"][p, :, o], want / c.k_scale, mag / c.k_scale, c.kt, "k")
    close(got["v"][p, :, o], f64(vn) / c.v_scale, 0.0, c.kt, "v")
    lim, ends = f64(bounds), np.asarray(lens) + np.asarray(new)
    for b in range(len(lens)):  # each page's bounds are those of what it holds now
        for i in range(-(-int(ends[b]) // page)):
            rows = got["k"][int(c.table[b, i]), :, :min(page, int(ends[b]) - i * page)]
            assert np.array_equal(lim[int(c.table[b, i]), :, 0], rows.min(1)), (b, i)
            assert np.array_equal(lim[int(c.table[b, i]), :, 1], rows.max(1)), (b, i)
    for x in "kv":
        old[x][p, :, o] = got[x][p, :, o]
        assert np.array_equal(got[x], old[x], equal_nan=True)
    sp = np.full(slots.shape, -1)
    sp[seq, :, pos] = pos[:, None]
    assert np.array_equal(slots.cpu().numpy(), sp)


# Row groups of a token (D / 16 lanes a row, 32 lanes a group) and the run of them that a warp takes:
# the fewer tokens, the shorter, while 2368 warps are not reached.
LARGE = [
    (128, 32, 4, [3000]),            # 10 groups, all in one run
    (128, 32, 4, [1, 0, 1499]),      # runs of 5: q alone, then q, k and v
    (128, 32, 4, [350, 350]),        # runs of 3, the last of 1
    (128, 32, 4, [480]),             # runs of 2
    (64, 6, 1, [3001]),              # 3 groups, all in one run
    (64, 6, 1, [700, 601, 0]),       # runs of 2 and 1
    (64, 24, 3, [2400]),             # 5 groups, partly filled ones among them
    (128, 6, 3, [1190, 3]),          # 4 groups, runs of 2
]


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("d,hq,hkv,new", LARGE)
def test_append_large_chunks(kv, q, d, hq, hkv, new):
    check_append(kv, q, d, 64 if d == 128 else 16, new, hq, hkv, [0, 63, 1000][:len(new)], seed=sum(new))


@pytest.mark.parametrize("new", [[5, 0, 40], [1500, 2, 1000]])
@pytest.mark.parametrize("norm,give_q,in_place", [("qk", True, True), ("q", True, False), ("k", True, True), ("k", False, False),
                                                  ("", True, True)])
def test_append_norms_in_place_and_without_queries(new, norm, give_q, in_place):
    check_append("bf16", "bf16", 128, 32, new, 32, 4, [10, 0, 77], norm, give_q, in_place, seed=len(norm))


def chunk(c, T):
    return [c.randn(T, h, c.d).to(c.qt).to(c.device) for h in (c.hq, c.hkv, c.hkv)]


def same_pages(c, k0, v0):
    return np.array_equal(f64(c.k), k0, equal_nan=True) and np.array_equal(f64(c.v), v0, equal_nan=True)


def test_append_leaves_out_a_sequence_of_negative_length():
    """All of its tokens, not only those whose slot is negative; the sequence beside it is written."""
    from long_context_sparse_idx16_b200 import RTPError

    c = Case([20, 33], hq=2, hkv=1, d=64, page=16, kv="fp16", room=8, seed=2)
    bounds = torch.zeros((c.pool, 1, 2, 64), dtype=c.kt, device=c.device)
    slots = torch.full((2, 1, c.width * 16), -1, dtype=torch.int32, device=c.device)
    cache = c.cache(bounds=bounds)
    cache.update_bounds(c.ints(c.lens))
    q, k, v = chunk(c, 6)
    k0, v0, b0 = f64(c.k), f64(c.v), f64(bounds)
    cache.append(q, k, v, c.ints([-1, 33]), cu_new=c.ints([0, 4, 6]), slot_positions=slots)
    with pytest.raises(RTPError):
        cache.check()
    page, rows = int(c.table[1, 2]), slice(1, 3)
    for x, y in ((f64(c.k), k0), (f64(c.v), v0)):
        assert not np.isnan(x[page, :, rows]).any()
        y[page, :, rows] = x[page, :, rows]
    assert same_pages(c, k0, v0)
    want = np.full(slots.shape, -1)
    want[1, 0, 33:35] = [33, 34]
    assert np.array_equal(slots.cpu().numpy(), want)
    got = f64(bounds)
    assert np.array_equal(got[page, 0, 0], f64(c.k)[page, 0, :3].min(0))
    b0[page] = got[page]
    assert np.array_equal(got, b0)


@pytest.mark.parametrize("cu,rows,written", [
    ([0, 3, 9], 6, {0: 3, 1: 3}),        # the last sequence names rows that were not given
    ([0, 3, 1 << 30], 6, {0: 3, 1: 3}),
    ([2, 5, 6], 6, {0: 3, 1: 1}),        # rows before the first sequence
    ([-(2**31), 3, 6], 6, {1: 3}),       # tokens numbered beyond 32 bits
    ([-2, 3, 6], 6, {0: 3, 1: 3})])      # the first sequence's tokens 2, 3, 4, behind two that were not given
def test_append_row_offsets_outside_the_rows(cu, rows, written):
    """Only rows that are there and named are written, to the slots of their tokens; the page bounds
    enclose what the pages hold and nothing else, and the caller hears of it."""
    from long_context_sparse_idx16_b200 import RTPError

    c = Case([18, 33], hq=2, hkv=1, d=64, page=16, kv="fp16", room=16, seed=3)
    bounds = torch.zeros((c.pool, 1, 2, 64), dtype=c.kt, device=c.device)
    cache = c.cache(bounds=bounds)
    cache.update_bounds(c.ints(c.lens))
    q, k, v = chunk(c, rows)
    # what no sequence has written would show in the bounds
    kk = torch.nan_to_num(c.k, nan=100.0)
    c.k.copy_(kk)
    k0, b0 = f64(c.k), f64(bounds)
    out = torch.full_like(q, 9.0)
    cache.append(q, k, v, c.ints(c.lens), cu_new=c.ints(cu), q_out=out, max_new=rows)
    with pytest.raises(RTPError):
        cache.check()
    got, lim = f64(c.k), f64(bounds)
    touched = {}
    for b, n in written.items():
        first = max(cu[b], 0)
        for t in range(first, first + n):
            s = c.lens[b] + t - cu[b]
            p, o = int(c.table[b, s // 16]), s % 16
            assert np.all(np.abs(got[p, 0, o]) < 50) and not np.array_equal(got[p, 0, o], k0[p, 0, o])
            k0[p, 0, o] = got[p, 0, o]
            touched.setdefault((p, s // 16 * 16 < c.lens[b]), []).append(o)
    assert np.array_equal(got, k0)
    for (p, widened), o in touched.items():
        lo, hi = got[p, 0, o].min(0), got[p, 0, o].max(0)
        if widened:
            lo, hi = np.minimum(lo, b0[p, 0, 0]), np.maximum(hi, b0[p, 0, 1])
        assert np.array_equal(lim[p, 0, 0], lo) and np.array_equal(lim[p, 0, 1], hi)
        b0[p] = lim[p]
    assert np.array_equal(lim, b0)
    assert bool((out[:max(cu[0], 0)] == 9.0).all())


# ---------------------------------------------------------------- streams and threads


def busy(stream, cycles=200_000_000):
    """About 0.1 s of a kernel that only counts, on `stream`."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(cycles)


def overwrite(*like):
    """What later work of the current stream does with memory that was freed to it: ones everywhere."""
    return [torch.empty_like(x).fill_(1) for x in like for _ in range(6)]


def test_temporaries_given_to_another_stream():
    """Inputs that nobody holds once the call has returned: the stream that reads them later still finds
    them, whatever the current stream allocates meanwhile."""
    from long_context_sparse_idx16_b200 import RTPError

    c = Case([3000, 900], hq=8, hkv=2, d=128, page=64, kv="fp16", seed=31, room=70)
    lens = c.ints(c.lens)
    q = c.randn(2, 8, 128).to(c.qt).to(c.device)
    kn, vn = (c.randn(2, 2, 128).to(c.qt).to(c.device) for _ in "kv")
    bounds = torch.zeros((c.pool, 2, 2, 128), dtype=c.kt, device=c.device)
    cache = c.cache(bounds=bounds)
    cache.update_bounds(lens)
    k0, v0, b0 = c.k.clone(), c.v.clone(), bounds.clone()
    drawn = torch.rand((2, 2, cache.capacity), device=c.device)
    pos = torch.arange(cache.capacity, dtype=torch.int32, device=c.device).expand(2, 2, -1).contiguous()
    cu, seq = c.ints([0, 1, 2]), c.ints([1, 0])
    side = torch.cuda.Stream()

    def reset():
        c.k.copy_(k0), c.v.copy_(v0), bounds.copy_(b0)

    def steps(kw, t):
        """Each call and its result; t makes the inputs it is given."""
        yield lambda: (cache.append(t(q), t(kn), t(vn), t(lens), cu_new=t(cu), positions=t(lens), **kw), c.k, c.v, bounds)
        yield lambda: (cache.update_bounds(t(lens + 1), **kw), bounds)[1:]
        yield lambda: (cache.decode(t(q), t(lens), **kw),)
        yield lambda: (cache.decode(t(q), t(lens), row_seq=t(seq), **kw),)
        yield lambda: cache.select_pages(t(q), t(lens), 5, row_seq=t(seq), **kw)
        yield lambda: (cache.decode(t(q), t(lens), pages=tuple(t(x) for x in sel), **kw),)
        yield lambda: (*cache.evict(t(lens), 500, t(drawn), t(pos), n_recent=9, **kw), c.k, c.v)

    sel = cache.select_pages(q, lens, 5)
    want = []
    for f in steps({}, lambda x: x):
        d0, p0 = drawn.clone(), pos.clone()
        reset()
        want.append([x.clone() for x in f()])
        drawn.copy_(d0), pos.copy_(p0)

    def temporary(x):
        y = x.clone()
        side.wait_stream(torch.cuda.current_stream())
        return y

    for i, f in enumerate(steps(dict(stream=side), temporary)):
        reset()
        torch.cuda.synchronize()
        busy(side)
        got = f()
        held = overwrite(q, kn, lens, cu, seq, drawn, pos, *sel)
        torch.cuda.synchronize()
        del held
        for a, b in zip(got, want[i]):
            a, b = (x.nan_to_num(7.0) if x.is_floating_point() else x for x in (a, b))
            assert torch.equal(a, b), i
    with pytest.raises(RTPError):  # row_seq names 3000 slots of the sequence that has pages for 970
        cache.check()


def test_a_cache_dropped_while_another_stream_reads_it():
    c = Case([3000], hq=8, hkv=2, d=128, page=64, kv="fp16", seed=32)
    lens, q = c.ints(c.lens), c.randn(1, 8, 128).to(c.qt).to(c.device)
    want = c.cache().decode(q, lens)
    side = torch.cuda.Stream()
    k, v, table = c.k.clone(), c.v.clone(), c.table.to(c.device)
    torch.cuda.synchronize()
    busy(side)
    side.wait_stream(torch.cuda.current_stream())
    from long_context_sparse_idx16_b200 import PagedKV

    cache = PagedKV(k, v, table)
    del k, v, table
    out = cache.decode(q, lens, stream=side)
    del cache
    held = overwrite(c.k, c.table.to(c.device))
    torch.cuda.synchronize()
    del held
    assert torch.equal(out, want)


def test_results_dropped_while_the_current_stream_reads_them():
    """A result of another stream, dropped when its reader is enqueued, is not given to that stream's next
    call before the reader is done."""
    c = Case([300], hq=8, hkv=2, d=128, page=64, kv="fp16", seed=33)
    lens = c.ints(c.lens)
    q = [c.randn(1, 8, 128).to(c.qt).to(c.device) for _ in range(2)]
    bounds = torch.zeros((c.pool, 2, 2, 128), dtype=c.kt, device=c.device)
    cache = c.cache(bounds=bounds)
    cache.update_bounds(lens)
    calls = [lambda q, **kw: cache.decode(q, lens, return_lse=True, **kw), lambda q, **kw: cache.select_pages(q, lens, 3, **kw),
             lambda q, **kw: (cache.append(q, q[:, :2], q[:, 2:4], lens - 1, **kw),)]
    side, now = torch.cuda.Stream(), torch.cuda.current_stream()
    for f in calls:
        want = [x.clone() for x in f(q[0])]
        torch.cuda.synchronize()
        got = f(q[0], stream=side)
        now.wait_stream(side)
        busy(now)
        copies = [x.clone() for x in got]
        del got
        f(q[1], stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))


def test_errors_of_another_stream_are_kept():
    """The error word is ready when the constructor returns, whatever the current stream still has to do."""
    from long_context_sparse_idx16_b200 import RTPError

    c = Case([300], hq=4, hkv=2, d=128, page=64, kv="fp16", seed=12)
    q = c.randn(1, 4, 128).to(c.qt).to(c.device)
    c.table[0, 1] = -5
    lens, table = c.ints([300]), c.table.to(c.device)
    side = torch.cuda.Stream()
    from long_context_sparse_idx16_b200 import PagedKV

    torch.cuda.synchronize()
    busy(torch.cuda.current_stream())
    cache = PagedKV(c.k, c.v, table)
    cache.decode(q, lens, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    with pytest.raises(RTPError):
        cache.check()
    cache.check()


def test_check_lets_other_threads_run():
    """While check() waits for the GPU, another Python thread goes on."""
    import threading
    import time

    c = Case([10], hq=2, hkv=1, d=64, page=16, kv="fp16", seed=1)
    cache = c.cache()
    cache.check()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.002)

    t = threading.Thread(target=tick)
    t.start()
    time.sleep(0.02)
    busy(torch.cuda.current_stream(), 1_000_000_000)  # half a second
    began = time.monotonic()
    cache.check()
    ended = time.monotonic()
    stop.set()
    t.join()
    assert ended - began > 0.2
    inside = [x for x in ticks if began < x < ended - 0.05]
    assert len(inside) > 10, len(inside)


def test_errors_are_taken_once_and_none_is_lost():
    """Two streams that report errors while a third takes them: every report is followed by an answer."""
    from long_context_sparse_idx16_b200 import RTPError

    c = Case([300], hq=4, hkv=2, d=128, page=64, kv="fp16", seed=12)
    q = c.randn(1, 4, 128).to(c.qt).to(c.device)
    c.table[0, 1] = -5
    cache, lens = c.cache(), c.ints([300])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(50):
        for s in streams[:2]:
            cache.decode(q, lens, stream=s)
        heard = 0
        for last in (False, True):
            if last:
                torch.cuda.synchronize()
            try:
                cache.check(stream=streams[2])
            except RTPError:
                heard += 1
        assert heard >= 1, i
        cache.check()


def test_calls_from_two_threads():
    """Two threads with a stream each on one cache: every result is the one that a single thread gets."""
    import threading

    c = Case([4000, 900, 17], hq=8, hkv=2, d=128, page=64, kv="fp16", seed=71)
    lens = c.ints(c.lens)
    cache = c.cache(bounds=torch.zeros((c.pool, 2, 2, 128), dtype=c.kt, device=c.device))
    cache.update_bounds(lens)
    qs = [c.randn(3, 8, 128).to(c.qt).to(c.device) for _ in range(2)]

    def step(q, **kw):
        pages = cache.select_pages(q, lens, 9, n_first=1, **kw)
        return cache.decode(q, lens, **kw), cache.decode(q, lens, pages=pages, **kw), pages[0]

    want = [step(q) for q in qs]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream() for _ in range(2)]

    def work(i):
        for _ in range(40):
            got[i].append(step(qs[i], stream=streams[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert len(g) == 40
        assert all(torch.equal(a, b) for r in g for a, b in zip(w, r))
    cache.check()


@pytest.mark.parametrize("kv,q,d,group", [("fp16", "fp16", 128, 12), ("bf16", "bf16", 128, 17), ("e4m3", "bf16", 128, 16),
                                          ("e4m3", "fp16", 64, 8), ("e4m3", "bf16", 64, 3), ("bf16", "bf16", 64, 5),
                                          ("fp16", "fp16", 64, 16)])
def test_decode_long_rows_of_wide_groups_and_short_heads(kv, q, d, group):
    """Long sequences split over many CTAs, in the builds for more than eight heads and for head dim 64."""
    c = Case([12345, 0, 30001], hq=group, hkv=1, d=d, page=64, kv=kv, q=q, seed=group,
             **(dict(k_scale=0.0625, v_scale=0.03125) if kv == "e4m3" else {}))
    x = c.randn(3, group, d, std=2.0).to(c.qt).to(c.device)
    out, lse = c.cache().decode(x, c.ints(c.lens), return_lse=True)
    check_decode(c, x, out, lse, [(b, np.arange(n)) for b, n in enumerate(c.lens)])


def test_check_of_a_cache_that_calls_refuse():
    """A cache of a page size that no call takes has met no error."""
    from long_context_sparse_idx16_b200 import PagedKV, RTPError

    k = torch.zeros((3, 1, 24, 64), dtype=torch.float16, device="cuda")
    cache = PagedKV(k, k, torch.zeros((1, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(RTPError, match="page_size"):
        cache.decode(torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    cache.check()
