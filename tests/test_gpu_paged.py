"""The paged-cache operators on the GPU against their fp64 definitions (tests/paged_ref.py)."""
import math

import numpy as np
import pytest
import torch

from paged_ref import DT, TINY, U, Case, check_decode, evict_choice, f64, page_choice, slots_seen

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- decode


def run_decode(c: Case, window=0, sinks=0, scores=False, **kw):
    q = c.randn(len(c.lens), c.hq, c.d, std=2.0).to(c.qt).to(c.device)
    kv = c.cache()
    lens = c.ints(c.lens)
    acc = c.randn(len(c.lens), c.hkv, kv.capacity).abs().to(c.device) if scores else None
    before = acc.clone() if scores else None
    out, lse = kv.decode(q, lens, window=window, n_sink=sinks, scores=acc, return_lse=True, **kw)
    kv.check()
    rows = [(b, slots_seen(n, window, sinks)) for b, n in enumerate(c.lens)]
    check_decode(c, q, out, lse, rows, scores=acc, before=before)
    return kv, q, lens, out


TYPES = [("fp16", "fp16"), ("bf16", "bf16"), ("e4m3", "fp16"), ("e4m3", "bf16")]
SCALES = {"e4m3": dict(k_scale=0.0625, v_scale=0.03125)}


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_types_and_pages(kv, q, d, page):
    lens = [0, 1, page - 1, page, page + 1, 300, 0, 1111]
    run_decode(Case(lens, hq=8, hkv=2, d=d, page=page, kv=kv, q=q, extra=2, seed=page + d, **SCALES.get(kv, {})))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 12, 16, 17, 32, 64])
def test_decode_groups(group):
    run_decode(Case([77, 0, 513], hq=2 * group, hkv=2, d=128, page=32, kv="bf16", seed=group))


@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("nhd", [False, True])
def test_decode_heads_and_layouts(hkv, nhd):
    run_decode(Case([5, 260, 64, 1], hq=4 * hkv, hkv=hkv, d=128, page=64, kv="fp16", nhd=nhd, seed=hkv))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (63, 1), (64, 64), (100, 4), (5000, 4), (130, 70), (16, 300)])
def test_decode_window_and_sinks(window, sinks):
    run_decode(Case([0, 1, 64, 99, 100, 129, 640, 1000], hq=8, hkv=2, d=128, page=32, kv="bf16", seed=window), window, sinks)


@pytest.mark.parametrize("kv,q", TYPES)
def test_decode_long(kv, q):
    """One long sequence beside short ones: split over many CTAs and joined."""
    run_decode(Case([3, 20011, 0, 64], hq=8, hkv=1, d=128, page=64, kv=kv, q=q, seed=3, **SCALES.get(kv, {})))


def test_decode_many_short_sequences():
    r = np.random.default_rng(5)
    run_decode(Case(r.integers(0, 200, 300).tolist(), hq=4, hkv=2, d=64, page=16, kv="fp16", seed=5))


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("group", [1, 4, 20])
def test_decode_scores(kv, q, group):
    c = Case([0, 1, 64, 777, 2500], hq=2 * group, hkv=2, d=128, page=64, kv=kv, q=q, seed=group, extra=1, **SCALES.get(kv, {}))
    run_decode(c, scores=True)


def test_decode_scores_of_a_window():
    run_decode(Case([0, 40, 700], hq=8, hkv=2, d=128, page=32, kv="fp16", seed=8), 100, 4, scores=True)


def test_decode_rows_of_one_sequence():
    """Several rows of a sequence, each with its own length, rows out of order."""
    c = Case([400, 33], hq=8, hkv=2, d=128, page=32, kv="bf16", seed=4)
    q = c.randn(6, c.hq, c.d).to(c.qt).to(c.device)
    seq, n = [1, 0, 0, 1, 0, 0], [33, 400, 399, 0, 1, 32]
    out, lse = c.cache().decode(q, c.ints(n), row_seq=c.ints(seq), return_lse=True)
    check_decode(c, q, out, lse, [(b, np.arange(m)) for b, m in zip(seq, n)])


def test_decode_strided_queries_and_output():
    c = Case([100, 65], hq=8, hkv=2, d=128, page=64, kv="fp16", seed=6)
    q = c.randn(2, 12, 128).to(c.qt).to(c.device)[:, 2:10]
    wide = torch.full((2, 11, 128), 7.0, dtype=c.qt, device=c.device)
    out = wide[:, 3:11]
    c.cache().decode(q, c.ints([100, 65]), out=out, sm_scale=0.05)
    check_decode(c, q, out, None, [(b, np.arange(n)) for b, n in enumerate(c.lens)], scale=float(np.float32(0.05)))
    assert bool((wide[:, :3] == 7.0).all())


def test_decode_extreme_scores():
    """Weights far apart: one key carries nearly all the weight, a million others a percent or two."""
    c = Case([40000], hq=4, hkv=1, d=64, page=64, kv="fp16", seed=9)
    q = torch.zeros(1, 4, 64, dtype=c.qt, device=c.device)
    q[..., 0] = 8.0
    k = f64(c.k)
    k[:, :, :, 0] = 0.0
    p, o = int(c.table[0, 300]), 11
    k[p, 0, o, 0] = 12.0  # score 12 above every other
    c.k = c.put(torch.from_numpy(np.nan_to_num(k)).float())
    kv = c.cache()
    out, lse = kv.decode(q, c.ints([40000]), return_lse=True)
    check_decode(c, q, out, lse, [(0, np.arange(40000))])
    # the weights of all but that key lie below fp16's least value, yet count
    q[..., 0] = 13.0
    out, lse = kv.decode(q, c.ints([40000]), return_lse=True)
    check_decode(c, q, out, lse, [(0, np.arange(40000))])


def test_decode_inf_and_nan_stay_with_their_rows():
    c = Case([70, 70], hq=2, hkv=1, d=64, page=64, kv="bf16", seed=10)
    p = int(c.table[1, 0])
    c.v[p, 0, 3, 5] = math.inf
    q = c.randn(2, 2, 64).to(c.qt).to(c.device)
    out = f64(c.cache().decode(q, c.ints([70, 70])))
    assert np.isfinite(out[0]).all() and np.isinf(out[1, :, 5]).all() and np.isfinite(np.delete(out[1], 5, 1)).all()


def test_decode_bad_pages_and_lengths_are_left_out():
    """A page number outside the pool takes its slots out; lengths are brought into the table."""
    from long_context_sparse_idx16_b200 import RTP_ERANGE, RTPError

    c = Case([300, 200, 64], hq=4, hkv=2, d=128, page=64, kv="fp16", seed=12)
    q = c.randn(3, 4, 128).to(c.qt).to(c.device)
    good = c.table.clone()
    c.table[0, 1], c.table[0, 3] = -5, 1 << 30
    c.table[2, 0] = c.pool
    kv = c.cache()
    out, lse = kv.decode(q, c.ints([300, -3, 64]), return_lse=True)
    with pytest.raises(RTPError) as e:
        kv.check()
    assert e.value.status == RTP_ERANGE
    kv.check()  # reported once
    c.table = good
    j = np.arange(300)
    check_decode(c, q, out, lse, [(0, j[(j // 64 != 1) & (j // 64 != 3)]), (1, np.arange(0)), (2, np.arange(0))])
    # a sequence number outside the batch, and a length beyond the table
    kv = c.cache()
    out, lse = kv.decode(q, c.ints([10, 10, 1 << 30]), row_seq=c.ints([3, -1, 0]), return_lse=True)
    with pytest.raises(RTPError):
        kv.check()
    check_decode(c, q[:2], out[:2], lse[:2], [(0, np.arange(0)), (0, np.arange(0))])


def test_decode_page_lists():
    c = Case([1000, 500, 64, 0], hq=8, hkv=2, d=128, page=32, kv="fp16", seed=13, extra=3)
    q = c.randn(4, 8, 128).to(c.qt).to(c.device)
    lists = [[[0, 5, 31], [7]], [[15, 3, 9], [-1, 2, 40, 15]], [[1], []], [[0], [0]]]
    sel = torch.full((4, 2, 6), 77, dtype=torch.int32)
    cnt = torch.zeros((4, 2), dtype=torch.int32)
    for r in range(4):
        for g in range(2):
            sel[r, g, :len(lists[r][g])] = torch.tensor(lists[r][g], dtype=torch.int32)
            cnt[r, g] = len(lists[r][g])
    kv = c.cache()
    out, lse = kv.decode(q, c.ints(c.lens), pages=(sel.to(c.device), cnt.to(c.device)), return_lse=True)
    rows = [(r, [np.array([j for i in lists[r][g] if 0 <= i for j in range(i * 32, i * 32 + 32) if j < c.lens[r]], dtype=int)
                 for g in range(2)]) for r in range(4)]
    check_decode(c, q, out, lse, rows)
    kv.check()
    # counts beyond the list are cut to it
    out2, _ = kv.decode(q, c.ints(c.lens), pages=(sel[..., :1].contiguous().to(c.device), (cnt * 0 + 9).to(c.device)), return_lse=True)
    check_decode(c, q, out2, None, [(r, [np.array([j for j in range(max(0, int(sel[r, g, 0])) * 32, int(sel[r, g, 0]) * 32 + 32)
                                                   if j < c.lens[r]], dtype=int) for g in range(2)]) for r in range(4)])


# ---------------------------------------------------------------- append


def rotated(x, w, pos, eps, base):
    """fp64 norm and rotation of [T][H][d], and the magnitude its rounding errors scale with."""
    d = x.shape[-1]
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    a = np.asarray(pos, dtype=np.float64)[:, None, None] * base ** (-2.0 * np.arange(d // 2) / d)
    y0, y1 = y[..., :d // 2], y[..., d // 2:]
    mag = np.abs(y0) + np.abs(y1)
    return np.concatenate([y0 * np.cos(a) - y1 * np.sin(a), y1 * np.cos(a) + y0 * np.sin(a)], -1), np.concatenate([mag, mag], -1)


def close(got, want, mag, dtype, what):
    """Half a step of the stored type, plus the fp32 arithmetic before it: the norm's sum of d
    squares, root and products (2^-20 covers d / 2 of their roundings in a tree) and the angle's
    sine and cosine (reduced angle to 2^-24 pi, sincosf within 2 steps): 2^-19 of |y0| + |y1|."""
    tol = U[dtype] * np.abs(want) * 1.01 + 2.0**-19 * mag + TINY[dtype]
    err = np.abs(got - want)
    assert np.all(err <= tol), (what, float((err / tol).max()))


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,new", [(16, [1, 1, 1]), (64, [1, 1, 1]), (16, [0, 37, 5]), (64, [200, 0, 1]), (128, [3, 129, 300]), (32, [0, 0, 700])])
def test_append(kv, q, d, page, new):
    lens = [0, 63, 1000]
    c = Case(lens, hq=6, hkv=2, d=d, page=page, kv=kv, q=q, room=max(new) + 1, seed=sum(new) + d, nhd=page == 32,
             **SCALES.get(kv, {}))
    T, eps, base = sum(new), 1e-5, 1e4
    qkv = c.randn(T, 10, d, std=1.5).to(c.qt).to(c.device)
    qn, kn, vn = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    qw, kw = ((1 + 0.2 * c.randn(d)).to(c.qt).to(c.device) for _ in "qk")
    bounds = c.randn(c.pool, 2, 2, d).abs()
    bounds[:, :, 0] *= -1
    bounds = bounds.to(c.kt).to(c.device)
    b0 = f64(bounds)
    slots = torch.full((3, 2, c.width * page), -1, dtype=torch.int32, device=c.device)
    k0, v0 = f64(c.k), f64(c.v)
    cache = c.cache(bounds=bounds)
    cu = np.concatenate([[0], np.cumsum(new)])
    one = all(n == 1 for n in new)
    out = cache.append(qn, kn, vn, c.ints(lens), cu_new=None if one else c.ints(cu), max_new=max(new), q_weight=qw,
                       k_weight=kw, eps=eps, rope_base=base, slot_positions=slots)
    cache.check()
    pos = np.concatenate([lens[b] + np.arange(n) for b, n in enumerate(new)])
    want, mag = rotated(f64(qn), f64(qw), pos, eps, base)
    close(f64(out), want, mag, c.qt, "q")
    wk, mk = rotated(f64(kn), f64(kw), pos, eps, base)
    wk, mk, wv = wk / c.k_scale, mk / c.k_scale, f64(vn) / c.v_scale
    got_k, got_v = f64(c.k), f64(c.v)
    want_sp = np.full(slots.shape, -1)
    touched = {}
    for b in range(3):
        for i in range(new[b]):
            s, t = lens[b] + i, cu[b] + i
            p, o = int(c.table[b, s // page]), s % page
            close(got_k[p, :, o], wk[t], mk[t], c.kt, "k")
            close(got_v[p, :, o], wv[t], 0.0, c.kt, "v")
            k0[p, :, o], v0[p, :, o] = got_k[p, :, o], got_v[p, :, o]
            want_sp[b, :, s] = s
            touched.setdefault((p, s // page * page >= lens[b]), []).append(o)
    assert np.array_equal(got_k, k0, equal_nan=True) and np.array_equal(got_v, v0, equal_nan=True)  # all else untouched
    assert np.array_equal(slots.cpu().numpy(), want_sp)
    for (p, begun), os_ in touched.items():
        rows = got_k[p][:, os_]
        lo, hi = rows.min(1), rows.max(1)
        if not begun:
            lo, hi = np.minimum(lo, b0[p, :, 0]), np.maximum(hi, b0[p, :, 1])
        b0[p, :, 0], b0[p, :, 1] = lo, hi
    assert np.array_equal(f64(bounds), b0)


def test_append_positions_no_norm_in_place():
    """Far positions of the caller's choice, no norm weights, q rotated in place, no bounds."""
    c = Case([10, 0], hq=4, hkv=1, d=128, page=16, kv="bf16", room=4, seed=2)
    x = c.randn(5, 4, 128).to(c.qt).to(c.device)
    k, v = (c.randn(5, 1, 128).to(c.qt).to(c.device) for _ in "kv")
    x0 = f64(x)
    pos = [1048575, 7, 0, 2147483647, 123456789]
    kv = c.cache()
    out = kv.append(x, k, v, c.ints([10, 0]), cu_new=c.ints([0, 2, 5]), positions=c.ints(pos), q_out=x)
    assert out is x
    want, mag = rotated(x0, None, pos, 0.0, 1e6)
    # an fp64 angle is off by 2^-53 of itself: 2^-22 rad at 2^31
    close(f64(x), want, mag * 1.0, c.qt, "q")
    wk, mk = rotated(f64(k), None, pos, 0.0, 1e6)
    close(f64(c.k)[int(c.table[0, 0]), :, 10], wk[0], mk[0], c.kt, "k")


def test_append_padded_rows_and_full_table():
    """Rows behind the last sequence stay; tokens beyond the table are left out and reported."""
    from long_context_sparse_idx16_b200 import RTPError

    c = Case([4, 15], hq=2, hkv=1, d=64, page=16, kv="fp16", seed=2)
    q, k, v = (c.randn(6, h, 64).to(c.qt).to(c.device) for h in (2, 1, 1))
    out = torch.full_like(q, 9.0)
    kv = c.cache()
    kv.append(q, k, v, c.ints([4, 15]), cu_new=c.ints([0, 2, 3]), q_out=out)
    kv.check()
    assert bool((out[3:] == 9.0).all()) and not bool((out[:3] == 9.0).any())
    assert np.isnan(f64(c.k)[int(c.table[0, 0]), 0, 6:]).all()
    k0 = f64(c.k)
    kv.append(q, k, v, c.ints([16, 15]), cu_new=c.ints([0, 2, 4]), q_out=out)
    with pytest.raises(RTPError):
        kv.check()
    k1 = f64(c.k)
    k1[int(c.table[1, 0]), 0, 15] = k0[int(c.table[1, 0]), 0, 15]  # the one token that had a place
    assert np.array_equal(k0, k1, equal_nan=True)


def test_append_saturates_e4m3():
    c = Case([0], hq=1, hkv=1, d=64, page=16, kv="e4m3", q="bf16", room=2, seed=2, k_scale=0.5, v_scale=2.0)
    k = torch.full((1, 1, 64), 1000.0, dtype=c.qt, device=c.device)
    v = torch.full((1, 1, 64), -5000.0, dtype=c.qt, device=c.device)
    c.cache().append(None, k, v, c.ints([0]), positions=c.ints([0]))
    p = int(c.table[0, 0])
    assert np.all(f64(c.k)[p, 0, 0] == 448.0) and np.all(f64(c.v)[p, 0, 0] == -448.0)


# ---------------------------------------------------------------- bounds and selection


def stored_bounds(c: Case):
    b = np.zeros((c.pool, c.hkv, 2, c.d))
    k = f64(c.k)
    for s, n in enumerate(c.lens):
        for i in range(-(-n // c.page)):
            rows = k[int(c.table[s, i]), :, :min(c.page, n - i * c.page)]
            b[int(c.table[s, i]), :, 0], b[int(c.table[s, i]), :, 1] = rows.min(1), rows.max(1)
    return b


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (128, 128)])
def test_bounds(kv, q, d, page):
    c = Case([0, 1, 300, 64], hq=2, hkv=2, d=d, page=page, kv=kv, q=q, seed=d, nhd=page == 16, **SCALES.get(kv, {}))
    bounds = torch.zeros((c.pool, 2, 2, d), device=c.device).to(c.kt)
    kv_ = c.cache(bounds=bounds)
    kv_.update_bounds(c.ints(c.lens))
    kv_.check()
    assert np.array_equal(f64(bounds), stored_bounds(c))


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 8, 20])
def test_select_pages(kv, q, d, group):
    c = Case([0, 1, 15, 16, 700, 3333], hq=2 * group, hkv=2, d=d, page=16, kv=kv, q=q, seed=group, extra=3, **SCALES.get(kv, {}))
    bounds = torch.from_numpy(stored_bounds(c)).float().to(c.kt).to(c.device)
    cache = c.cache(bounds=bounds)
    x = c.randn(6, c.hq, d).to(c.qt).to(c.device)
    for top, first, recent in ((1, 0, 1), (1, 1, 0), (7, 1, 2), (40, 0, 0), (209, 1, 1), (300, 4, 4)):
        sel, cnt = cache.select_pages(x, c.ints(c.lens), top, n_first=first, n_recent=recent)
        cache.check()
        sel, cnt = sel.cpu().numpy(), cnt.cpu().numpy()
        for r, n in enumerate(c.lens):
            for g in range(2):
                want = page_choice(c, f64(bounds), f64(x)[r], r, n, g, top, first, recent)
                assert cnt[r, g] == len(want)
                assert sel[r, g].tolist() == want + [-1] * (top - len(want)), (top, r, g)


def test_select_ties_take_the_lower_page():
    c = Case([1600], hq=2, hkv=1, d=64, page=16, kv="fp16", seed=3)
    bounds = torch.zeros((c.pool, 1, 2, 64), dtype=c.kt, device=c.device)
    x = torch.ones((1, 2, 64), dtype=c.qt, device=c.device)
    cache = c.cache(bounds=bounds)
    for p in (10, 20, 77):
        bounds[int(c.table[0, p])] = 1.0
    sel, _ = cache.select_pages(x, c.ints([1600]), 9, n_first=0, n_recent=1)
    assert sel.flatten().tolist() == [0, 1, 2, 3, 4, 10, 20, 77, 99]
    bounds.fill_(-0.0)
    bounds[int(c.table[0, 4])] = 0.0  # the same score
    sel, _ = cache.select_pages(x, c.ints([1600]), 3, n_first=0, n_recent=0)
    assert sel.flatten().tolist() == [0, 1, 2]
    bounds[int(c.table[0, 0])] = math.nan  # ranks last
    bounds[int(c.table[0, 1])] = -math.inf
    sel, _ = cache.select_pages(x, c.ints([1600]), 99, n_first=0, n_recent=0)
    assert sel.flatten().tolist() == list(range(1, 100))


def test_select_and_attend_rows():
    """Chunk rows, each with its own pages, then attention over them."""
    c = Case([900, 411], hq=8, hkv=2, d=128, page=32, kv="bf16", seed=11)
    bounds = torch.from_numpy(stored_bounds(c)).float().to(c.kt).to(c.device)
    seq = [0] * 20 + [1] * 11
    n = [900 - i for i in range(19, -1, -1)] + [411 - 13 * i for i in range(11)]
    x = c.randn(31, 8, 128, std=2.0).to(c.qt).to(c.device)
    cache = c.cache(bounds=bounds)
    rows = dict(row_seq=c.ints(seq))
    pages = cache.select_pages(x, c.ints(n), 6, n_first=1, n_recent=2, **rows)
    out, lse = cache.decode(x, c.ints(n), pages=pages, return_lse=True, **rows)
    cache.check()
    want = []
    for r in range(31):
        per = [page_choice(c, f64(bounds), f64(x)[r], seq[r], n[r], g, 6, 1, 2) for g in range(2)]
        for g in range(2):
            assert pages[0][r, g].tolist() == per[g] + [-1] * (6 - len(per[g]))
        want.append((seq[r], [np.array([j for i in p for j in range(i * 32, i * 32 + 32) if j < n[r]]) for p in per]))
    check_decode(c, x, out, lse, want)


# ---------------------------------------------------------------- eviction


def run_evict(c: Case, budget, recent, sinks, seed, ties=False, in_place=True, scores=None):
    r = np.random.default_rng(seed)
    cap = c.width * c.page
    n_s = len(c.lens)
    if scores is None:
        scores = r.exponential(size=(n_s, c.hkv, cap)).astype(np.float32)
        if ties:
            scores = np.floor(scores * 2)
    pos = np.full((n_s, c.hkv, cap), -1, dtype=np.int32)
    for b, n in enumerate(c.lens):
        for g in range(c.hkv):
            pos[b, g, :n] = r.permutation(n + 50)[:n]
            scores[b, g, n:] = 0.0
    sc, ps = c.dev(scores), c.dev(pos)
    cache = c.cache()
    k0, v0 = f64(c.k), f64(c.v)
    kw = {} if in_place else dict(out_scores=torch.full_like(sc, 5.0), out_positions=torch.full_like(ps, 5))
    new, so, po = cache.evict(c.ints(c.lens), budget, sc, ps, n_recent=recent, n_sink=sinks, **kw)
    cache.check()
    if not in_place:
        assert np.array_equal(sc.cpu().numpy(), scores, equal_nan=True) and np.array_equal(ps.cpu().numpy(), pos)
    so, po = so.cpu().numpy(), po.cpu().numpy()
    for b, n in enumerate(c.lens):
        m = min(n, budget)
        assert int(new[b]) == m
        for g in range(c.hkv):
            _, src = evict_choice(scores[b, g], pos[b, g], n, budget, recent, sinks)
            assert np.array_equal(so[b, g], np.concatenate([scores[b, g][src], np.zeros(cap - m, np.float32)]), equal_nan=True)
            assert np.array_equal(po[b, g], np.concatenate([pos[b, g][src], np.full(cap - m, -1)]))
            for dst in np.flatnonzero(src != np.arange(m)):
                s = src[dst]
                fp, tp = int(c.table[b, s // c.page]), int(c.table[b, dst // c.page])
                for x in (k0, v0):  # the sources lie behind the budget: never written
                    x[tp, g, dst % c.page] = x[fp, g, s % c.page]
    assert np.array_equal(f64(c.k), k0, equal_nan=True) and np.array_equal(f64(c.v), v0, equal_nan=True)


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e4m3"])
@pytest.mark.parametrize("page,d", [(16, 64), (64, 128)])
@pytest.mark.parametrize("budget,recent,sinks", [(1, 0, 0), (1, 1, 0), (100, 0, 0), (100, 96, 4), (257, 32, 4), (999, 1, 1), (5000, 3, 3)])
def test_evict(kv, page, d, budget, recent, sinks):
    c = Case([0, 1, 100, 101, 640, 1000, 1777], hq=2, hkv=2, d=d, page=page, kv=kv, seed=budget, extra=1, nhd=page == 16)
    run_evict(c, budget, recent, sinks, budget, ties=recent == 32, in_place=budget % 2 == 0)


def test_evict_long():
    c = Case([30000, 9000], hq=2, hkv=1, d=64, page=128, kv="fp16", seed=1)
    run_evict(c, 8192, 256, 4, 3)


@pytest.mark.parametrize("kind", ["equal", "nan", "inf", "signed"])
def test_evict_odd_scores(kind):
    c = Case([600, 333], hq=2, hkv=2, d=64, page=16, kv="fp16", seed=1)
    r = np.random.default_rng(7)
    s = np.ones((2, 2, c.width * 16), dtype=np.float32)
    if kind == "nan":
        s[r.random(s.shape) < 0.6] = math.nan
    elif kind == "inf":
        s[r.random(s.shape) < 0.6] = math.inf
        s[r.random(s.shape) < 0.2] = -math.inf
    elif kind == "signed":
        s = r.standard_normal(s.shape).astype(np.float32)
        s[r.random(s.shape) < 0.3] = -0.0
        s[r.random(s.shape) < 0.3] = 0.0
    run_evict(c, 300, 20, 4, 5, scores=s)


# ---------------------------------------------------------------- together


def test_serving_loop_together():
    """Prefill, decode steps with accumulated weights, eviction, more steps, and the bounds that an
    eviction leaves: against the definitions applied to the cache as it stands."""
    c = Case([0, 0, 0], hq=8, hkv=2, d=64, page=16, kv="bf16", room=200, seed=21)
    bounds = torch.zeros((c.pool, 2, 2, 64), dtype=c.kt, device=c.device)
    kv = c.cache(bounds=bounds)
    cap = kv.capacity
    scores = torch.zeros((3, 2, cap), device=c.device)
    posns = torch.full((3, 2, cap), -1, dtype=torch.int32, device=c.device)
    w = torch.ones(64, dtype=c.qt, device=c.device)
    lens = c.ints([0, 0, 0])
    new = [100, 61, 1]
    q, k, v = (c.randn(sum(new), h, 64).to(c.qt).to(c.device) for h in (8, 2, 2))
    kv.append(q, k, v, lens, cu_new=c.ints([0, 100, 161, 162]), q_weight=w, k_weight=w, slot_positions=posns)
    lens = lens + c.ints(new)
    nxt = lens.clone()  # the next position, which evictions do not change
    for step in range(30):
        q, k, v = (c.randn(3, h, 64).to(c.qt).to(c.device) for h in (8, 2, 2))
        qr = kv.append(q, k, v, lens, positions=nxt, q_weight=w, k_weight=w, slot_positions=posns)
        lens, nxt = lens + 1, nxt + 1
        before = scores.clone()
        out, lse = kv.decode(qr, lens, scores=scores, return_lse=True)
        c.lens = lens.tolist()
        if step % 7 == 0:
            check_decode(c, qr, out, lse, [(b, np.arange(n)) for b, n in enumerate(c.lens)], scores=scores, before=before)
        if step % 10 == 9:
            s0, p0, k0 = f64(scores), posns.cpu().numpy().copy(), f64(c.k)
            lens, _, _ = kv.evict(lens, 64, scores, posns, n_recent=16, n_sink=2)
            for b in range(3):
                for g in range(2):
                    n = c.lens[b]
                    _, src = evict_choice(s0[b, g], p0[b, g], n, 64, 16, 2)
                    assert np.array_equal(posns[b, g].cpu().numpy()[:len(src)], p0[b, g][src])
                    assert int(posns[b, g].max()) == int(nxt[b]) - 1
                    got = f64(c.k)[c.table[b].numpy()[np.arange(len(src)) // 16], g, np.arange(len(src)) % 16]
                    assert np.array_equal(got, k0[c.table[b].numpy()[src // 16], g, src % 16])
            c.lens = lens.tolist()
            assert max(c.lens) <= 64
            b = stored_bounds(c)
            for s, n in enumerate(c.lens):
                for i in range(-(-n // 16)):
                    assert np.array_equal(f64(bounds)[int(c.table[s, i])], b[int(c.table[s, i])])
            pages = kv.select_pages(qr, lens, 3, n_first=1, n_recent=1)
            out, lse = kv.decode(qr, lens, pages=pages, return_lse=True)
            rows = [(s, [np.array([j for i in pages[0][s, g].tolist() if i >= 0 for j in range(16 * i, 16 * i + 16)
                                   if j < c.lens[s]]) for g in range(2)]) for s in range(3)]
            check_decode(c, qr, out, lse, rows)
    kv.check()


def test_graph_replay_and_streams():
    """A captured step follows lengths, queries and tables that change between replays; two streams
    at once keep their results; runs agree bit for bit."""
    c = Case([900, 3000, 17], hq=8, hkv=2, d=128, page=64, kv="fp16", seed=31, room=70)
    bounds = torch.from_numpy(stored_bounds(c)).float().to(c.kt).to(c.device)
    kv = c.cache(bounds=bounds)
    q = c.randn(3, 8, 128).to(c.qt).to(c.device)
    k, v = (c.randn(3, 2, 128).to(c.qt).to(c.device) for _ in "kv")
    lens = c.ints(c.lens)
    scores = torch.zeros((3, 2, kv.capacity), device=c.device)

    def step():
        qr = kv.append(q, k, v, lens)
        n = lens + 1
        out, lse = kv.decode(qr, n, scores=scores, return_lse=True)
        pages = kv.select_pages(qr, n, 8)
        return out, lse, kv.decode(qr, n, pages=pages), pages[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for n in ([900, 3000, 17], [5, 2999, 0], [899, 1024, 16]):
        lens.copy_(c.ints(n))
        q.copy_(c.randn(3, 8, 128))
        scores.zero_()
        g.replay()
        one = [x.clone() for x in got] + [scores.clone()]
        scores.zero_()
        two = list(step()) + [scores]
        assert all(torch.equal(x, y) for x, y in zip(one, two))
    kv.check()
    # the same calls on two streams at once, each with its own outputs
    want = kv.decode(q, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[kv.decode(q, lens, stream=s) for s in streams] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for pair in outs for o in pair)
    assert DT and TINY


def test_select_bad_pages_rank_last():
    from long_context_sparse_idx16_b200 import RTPError

    c = Case([1600], hq=4, hkv=2, d=64, page=16, kv="fp16", seed=3)
    bounds = torch.from_numpy(stored_bounds(c)).float().to(c.kt).to(c.device)
    x = c.randn(1, 4, 64).to(c.qt).to(c.device)
    good = c.table.clone()
    c.table[0, 7], c.table[0, 60] = 1 << 20, -1
    cache = c.cache(bounds=bounds)
    sel, cnt = cache.select_pages(x, c.ints([1600]), 97, n_first=0, n_recent=0)
    with pytest.raises(RTPError):
        cache.check()
    c.table = good
    for g in range(2):
        b = f64(bounds)
        b[[int(good[0, 7]), int(good[0, 60])]] = -np.inf
        got = sel[0, g].tolist()
        assert cnt[0, g] == 97 and len(set(got)) == 97 and not {7, 60} & set(got)


@pytest.mark.parametrize("n", [5000, 60000 * 16])
def test_select_long_lists(n):
    """More pages than one pass of threads; more than shared memory holds (60000 pages of 16)."""
    c = Case([1], hq=4, hkv=1, d=64, page=16, kv="bf16", seed=3)
    pages = -(-n // 16)
    c.table = torch.arange(pages, dtype=torch.int32).flip(0)[None]
    c.k = torch.zeros((pages, 1, 16, 64), dtype=c.kt, device=c.device)
    c.v = c.k
    g = torch.Generator(device="cuda").manual_seed(1)
    lim = torch.randn((pages, 1, 2, 64), generator=g, device=c.device).abs()
    lim[:, :, 0] *= -1
    bounds = lim.to(c.kt)
    x = c.randn(1, 4, 64).to(c.qt).to(c.device)
    sel, cnt = c.cache(bounds=bounds).select_pages(x, c.ints([n]), 100, n_first=1, n_recent=2)
    b = bounds[c.table[0].long().to(c.device), 0].double()
    q = x[0].double()
    score = torch.maximum(q[:, None] * b[None, :, 0], q[:, None] * b[None, :, 1]).sum(-1).amax(0)
    score[0] = score[pages - 2:] = math.inf
    want = score.sort(descending=True, stable=True).indices[:100].sort().values
    assert torch.equal(sel[0, 0].long(), want) and int(cnt) == 100
    # equal scores everywhere: the lowest pages
    bounds.fill_(0.5)
    sel, _ = c.cache(bounds=bounds).select_pages(x, c.ints([n]), 50, n_first=0, n_recent=1)
    assert sel.flatten().tolist() == list(range(49)) + [pages - 1]


def test_select_close_scores():
    """Scores nearer to one another than fp32 sums can tell: the exact order decides."""
    c = Case([16 * 500], hq=2, hkv=1, d=128, page=16, kv="fp16", seed=3)
    r = np.random.default_rng(2)
    base = np.abs(r.standard_normal(128)).astype(np.float16).astype(np.float64) * 30
    b = np.zeros((c.pool, 1, 2, 128))
    for p in range(500):
        # pages differ in one small term only, far below the size of the others
        t = base.copy()
        t[p % 128] = 0.0
        t[127 - p % 128] += 0.0
        b[int(c.table[0, p]), 0, 1] = base
        b[int(c.table[0, p]), 0, 1, 0] = 2.0**-14 * (1 + int(r.integers(0, 200)) / 1024)
    bounds = torch.from_numpy(b).to(c.kt).to(c.device)
    x = torch.ones((1, 2, 128), dtype=c.qt, device=c.device)
    sel, _ = c.cache(bounds=bounds).select_pages(x, c.ints([8000]), 40, n_first=0, n_recent=0)
    assert sel.flatten().tolist() == page_choice(c, f64(bounds), f64(x)[0], 0, 8000, 0, 40, 0, 0)


def test_evict_beyond_shared_memory():
    c = Case([50000, 70], hq=1, hkv=1, d=64, page=16, kv="e4m3", seed=1)
    run_evict(c, 20000, 100, 4, 3, ties=True)


def test_decode_e4m3_query_ranges():
    """bf16 queries far outside fp16's range over e4m3 pages: scaled per head, not rounded."""
    c = Case([130, 77], hq=4, hkv=2, d=128, page=32, kv="e4m3", q="bf16", seed=14, k_scale=2.0**-30)
    q = c.randn(2, 4, 128)
    q *= torch.tensor([2.0**30, 2.0**25, 2.0**-60, 2.0**33])[None, :, None]
    q = q.to(c.qt).to(c.device)
    c.k = c.put(torch.nan_to_num(c.randn(c.pool, 2, 32, 128) * 20))
    c.v = c.put(c.randn(c.pool, 2, 32, 128))
    out, lse = c.cache().decode(q, c.ints(c.lens), sm_scale=0.002, return_lse=True)
    check_decode(c, q, out, lse, [(b, np.arange(n)) for b, n in enumerate(c.lens)], scale=float(np.float32(0.002)))


def test_decode_nan_query_gives_nan():
    c = Case([200, 200], hq=16, hkv=2, d=64, page=16, kv="bf16", seed=15)
    q = c.randn(2, 16, 64).to(c.qt).to(c.device)
    q[1, 3, 7] = math.nan
    out, lse = c.cache().decode(q, c.ints([200, 200]), return_lse=True)
    o = f64(out)
    assert np.isnan(o[1, 3]).all() and bool(lse[1, 3].isnan())
    assert np.isfinite(o[0]).all() and np.isfinite(np.delete(o[1], 3, 0)).all()


def test_decode_many_ragged_rows():
    """More rows than every CTA plans by itself, empty ones among them, split ones too."""
    r = np.random.default_rng(8)
    lens = np.where(r.random(700) < 0.3, 0, r.integers(1, 60, 700))
    lens[123], lens[699] = 9000, 3000
    run_decode(Case(lens.tolist(), hq=3, hkv=1, d=64, page=16, kv="fp16", seed=16))


@pytest.mark.parametrize("group", [1, 5, 8, 16, 64])
def test_select_chunk_rows(group):
    """Runs of rows of one sequence inside and across the blocks that share a read of the bounds;
    groups whose heads are laid out in several goes."""
    c = Case([1300, 700, 2500], hq=group, hkv=1, d=64, page=16, kv="fp16", seed=group)
    bounds = torch.from_numpy(stored_bounds(c)).float().to(c.kt).to(c.device)
    seq = [0] * 3 + [1] * 9 + [0] * 2 + [2] * 20 + [1]
    r = np.random.default_rng(group)
    n = [int(r.integers(0, c.lens[b] + 1)) for b in seq]
    x = c.randn(len(seq), group, 64).to(c.qt).to(c.device)
    sel, cnt = c.cache(bounds=bounds).select_pages(x, c.ints(n), 12, row_seq=c.ints(seq), n_first=1, n_recent=1)
    for i, b in enumerate(seq):
        want = page_choice(c, f64(bounds), f64(x)[i], b, n[i], 0, 12, 1, 1)
        assert sel[i, 0].tolist() == want + [-1] * (12 - len(want)) and int(cnt[i, 0]) == len(want)


# ---------------------------------------------------------------- layouts, offsets, many lists


def padded(x, rows=1, dims=16):
    """The same values in a larger allocation: pages, heads and slots with gaps between them."""
    p, h, s, d = x.shape
    big = torch.zeros((p, h + 1, s + rows, d + dims), dtype=x.dtype, device=x.device)
    view = big[:, :h, :s, :d]
    view.copy_(x)
    return view


@pytest.mark.parametrize("kv,q", [("fp16", "fp16"), ("e4m3", "bf16")])
def test_padded_strides(kv, q):
    """Strides that are no multiples of one another, different for K and V."""
    c = Case([300, 0, 77], hq=8, hkv=2, d=64, page=32, kv=kv, q=q, seed=41, room=40, **SCALES.get(kv, {}))
    c.k, c.v = padded(c.k), padded(c.v, 3, 32)
    run_decode(c)
    x = c.randn(3, 12, 64).to(c.qt).to(c.device)
    cache = c.cache(bounds=torch.zeros((c.pool, 2, 2, 64), device=c.device).to(c.kt))
    out = cache.append(x[:, :8], x[:, 8:10], x[:, 10:], c.ints(c.lens))
    c.lens = [n + 1 for n in c.lens]
    lens = c.ints(c.lens)
    o, lse = cache.decode(out, lens, return_lse=True)
    cache.check()
    check_decode(c, out, o, lse, [(b, np.arange(n)) for b, n in enumerate(c.lens)])
    cache.update_bounds(lens)
    assert np.array_equal(f64(cache.bounds), stored_bounds(c))
    run_evict(c, 64, 8, 2, 1)


def test_pool_beyond_32_bits():
    """Pages whose element offsets pass 2^31 (and byte offsets 2^32): append, bounds, decode, evict."""
    free, _ = torch.cuda.mem_get_info()
    pages, hkv, ps, d = 70000, 4, 64, 128
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    c = Case([200, 130], hq=8, hkv=hkv, d=d, page=ps, kv="bf16", seed=42, room=80)
    small_k, small_v, small_table = c.k, c.v, c.table.clone()
    c.k, c.v = (torch.empty((pages, hkv, ps, d), dtype=c.kt, device=c.device) for _ in "kv")
    far = torch.arange(pages - c.pool, pages)
    c.k[far[0]:], c.v[far[0]:] = small_k, small_v
    c.table = torch.where(small_table >= 0, small_table + (pages - c.pool), small_table).to(torch.int32)
    bounds = torch.zeros((pages, hkv, 2, d), dtype=c.kt, device=c.device)
    cache = c.cache(bounds=bounds)
    x = c.randn(2, 16, d).to(c.qt).to(c.device)
    q = cache.append(x[:, :8], x[:, 8:12], x[:, 12:], c.ints(c.lens))
    lens = c.ints([201, 131])
    cache.update_bounds(lens)
    out, lse = cache.decode(q, lens, return_lse=True)
    sel, cnt = cache.select_pages(q, lens, 2)
    cache.check()
    base = pages - c.pool  # back to a small copy for the fp64 side
    c.k, c.v, c.table, c.lens = c.k[base:].clone(), c.v[base:].clone(), small_table, [201, 131]
    check_decode(c, q, out, lse, [(b, np.arange(n)) for b, n in enumerate(c.lens)])
    b64 = stored_bounds(c)
    assert np.array_equal(f64(bounds[base:]), b64)
    for r in range(2):
        for g in range(hkv):
            assert sel[r, g].tolist() == page_choice(c, b64, f64(q)[r], r, c.lens[r], g, 2, 0, 1)
    # eviction moves rows between far pages
    cap = cache.capacity
    scores = torch.rand((2, hkv, cap), device=c.device)
    pos = torch.arange(cap, device=c.device, dtype=torch.int32).expand(2, hkv, cap).contiguous()
    s0 = scores.cpu().numpy()
    cache.evict(lens, 100, scores, pos, n_recent=10)
    after = f64(cache.k[base:])
    before = f64(c.k)
    for b, n in enumerate(c.lens):
        for g in range(hkv):
            _, src = evict_choice(s0[b, g], np.arange(cap), n, 100, 10, 0)
            j = np.arange(100)
            t = c.table[b].numpy()
            assert np.array_equal(after[t[j // ps], g, j % ps], before[t[src // ps], g, src % ps])


@pytest.mark.parametrize("page", [16, 64, 128])
def test_many_page_lists(page):
    """More lists than every CTA plans by itself, from empty to full, short and long pages."""
    c = Case([page * 20 - 3, page * 7], hq=6, hkv=3, d=64, page=page, kv="fp16", seed=page)
    r = np.random.default_rng(page)
    rows = 130
    seq = r.integers(0, 2, rows)
    n = np.array([int(r.integers(0, c.lens[b] + 1)) for b in seq])
    sel = np.full((rows, 3, 9), -1, dtype=np.int32)
    cnt = r.integers(0, 10, (rows, 3)).astype(np.int32)
    want = []
    for i in range(rows):
        per = []
        for g in range(3):
            pages = r.permutation(20)[:cnt[i, g]]
            sel[i, g, :cnt[i, g]] = pages
            per.append(np.array([j for p in pages for j in range(p * page, p * page + page) if j < n[i]], dtype=int))
        want.append((int(seq[i]), per))
    q = c.randn(rows, 6, 64).to(c.qt).to(c.device)
    cache = c.cache()
    out, lse = cache.decode(q, c.ints(n.tolist()), row_seq=c.ints(seq.tolist()), return_lse=True,
                            pages=(torch.from_numpy(sel).to(c.device), torch.from_numpy(cnt).to(c.device)))
    cache.check()
    check_decode(c, q, out, lse, want)


def test_decode_writes_over_its_queries():
    c = Case([700, 64, 0, 2100], hq=16, hkv=2, d=128, page=64, kv="bf16", seed=51)
    q = c.randn(4, 16, 128).to(c.qt).to(c.device)
    cache = c.cache()
    want = cache.decode(q, c.ints(c.lens))
    got = q.clone()
    assert cache.decode(got, c.ints(c.lens), out=got) is got
    assert torch.equal(got, want)


def test_wider_slot_arrays_and_captured_eviction():
    """Scores and positions with more slots than the table; append of a chunk, eviction and the bounds
    behind it captured and replayed with other contents."""
    c = Case([150, 90, 33], hq=4, hkv=2, d=64, page=16, kv="fp16", seed=61, room=50)
    bounds = torch.zeros((c.pool, 2, 2, 64), dtype=c.kt, device=c.device)
    cache = c.cache(bounds=bounds)
    S = cache.capacity + 37
    scores = torch.zeros((3, 2, S), device=c.device)
    pos = torch.full((3, 2, S), -1, dtype=torch.int32, device=c.device)
    lens = c.ints(c.lens)
    cu = c.ints([0, 40, 41, 60])
    x = c.randn(64, 8, 64).to(c.qt).to(c.device)
    out = torch.zeros((64, 4, 64), dtype=c.qt, device=c.device)

    def step():
        cache.append(x[:, :4], x[:, 4:6], x[:, 6:], lens, cu_new=cu, max_new=1, q_out=out, slot_positions=pos)
        n = lens + (cu[1:] - cu[:-1])
        cache.decode(out[:3], n, scores=scores)
        return cache.evict(n, 64, scores, pos, n_recent=8, n_sink=2)

    k0, v0 = c.k.clone(), c.v.clone()

    def reset(seed):
        g = torch.Generator().manual_seed(seed)
        c.k.copy_(k0)
        c.v.copy_(v0)
        bounds.zero_()
        out.zero_()
        x.copy_(torch.randn(x.shape, generator=g).to(c.qt))
        scores.copy_(torch.rand(scores.shape, generator=g))
        pos.copy_(torch.arange(S, dtype=torch.int32).expand(3, 2, S))
        for b, n in enumerate(c.lens):
            scores[b, :, n:] = 0.0
            pos[b, :, n:] = -1

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        reset(1)
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    reset(2)
    with torch.cuda.graph(graph):
        new, _, _ = step()
    for seed in (3, 4):
        reset(seed)
        graph.replay()
        got = [t.clone() for t in (c.k, c.v, bounds, scores, pos, out, new)]
        reset(seed)
        n2, _, _ = step()
        want = [c.k, c.v, bounds, scores, pos, out, n2]
        # unused slots hold NaN
        assert all(torch.equal(a.nan_to_num(7.0) if a.is_floating_point() else a, b.nan_to_num(7.0) if b.is_floating_point() else b)
                   for a, b in zip(got, want))
        assert new.tolist() == [64, 64, 52]
        assert bool((out[60:] == 0).all())  # rows behind the last sequence
        assert bool((pos[:, :, 64:] == -1).all()) and bool((scores[:, :, 64:] == 0).all())
    cache.check()


def test_two_graphs_at_once():
    """Two captured steps on two streams, replayed together, keep their own workspaces."""
    c = Case([4000, 900, 17], hq=8, hkv=2, d=128, page=64, kv="fp16", seed=71)
    bounds = torch.from_numpy(stored_bounds(c)).float().to(c.kt).to(c.device)
    cache = c.cache(bounds=bounds)
    lens = c.ints(c.lens)
    qs = [c.randn(3, 8, 128).to(c.qt).to(c.device) for _ in range(2)]

    def step(q):
        pages = cache.select_pages(q, lens, 9, n_first=1)
        return cache.decode(q, lens), cache.decode(q, lens, pages=pages), pages[0]

    want = [[t.clone() for t in step(q)] for q in qs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for q, st in zip(qs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(step(q))
        graphs.append(g)
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(a, b) for a, b in zip(w, o))
