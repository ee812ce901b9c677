"""Refusals of the paged-cache operators, at the C entry points and in the binding (no GPU needed)."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import long_context_sparse_idx16_b200 as rtp  # noqa: E402
from long_context_sparse_idx16_b200 import PagedKV, build as rtp_build  # noqa: E402

BASE = 1 << 20  # a 16-byte aligned address that no host check dereferences


@pytest.fixture(scope="module")
def lib():
    rtp_build.build()
    return rtp.lib()


def _kv(**kw):
    a = dict(k=BASE, v=BASE, n_pages=10, page_size=16, n_kv_heads=2, head_dim=64, dtype=rtp_dtype("fp16"), k_scale=1.0,
             v_scale=1.0, block_table=BASE, table_stride=5, max_pages=5, n_seqs=3, bounds=BASE, err=None)
    ks, vs = kw.pop("k_stride", (2048, 1024, 64)), kw.pop("v_stride", (2048, 1024, 64))
    a.update(kw)
    return rtp.rtp_paged_kv(k_stride=(C.c_int64 * 3)(*ks), v_stride=(C.c_int64 * 3)(*vs), **a)


def rtp_dtype(name):
    return {"fp16": 0, "bf16": 1, "e4m3": 2}[name]


def _append(lib, kv=None, **kw):
    a = dict(q=BASE, k=BASE, v=BASE, dtype=0, qs=256, ks=128, vs=128, T=3, hq=4, cu=None, max_new=1, lens=BASE, pos=None,
             qw=None, kw=None, eps=1e-6, base=1e6, q_out=BASE, os=256, sp=None, sps=0, st=None)
    a.update(kw)
    return lib.rtp_paged_append(C.byref(kv) if kv is not None else None, *a.values())


def _decode(lib, kv=None, **kw):
    a = dict(q=BASE, dtype=0, qs=256, rows=3, hq=4, seq=None, lens=BASE, window=0, sink=0, scale=0.0, sel=None, cnt=None,
             ss=0, out=BASE, os=256, lse=None, scores=None, scs=0, ws=BASE, wb=1 << 40, st=None)
    a.update(kw)
    return lib.rtp_paged_decode(C.byref(kv) if kv is not None else None, *a.values())


def _select(lib, kv=None, **kw):
    a = dict(q=BASE, dtype=0, qs=256, rows=3, hq=4, seq=None, lens=BASE, top=3, first=1, recent=1, sel=BASE, ss=3,
             cnt=BASE, ws=BASE, wb=1 << 40, st=None)
    a.update(kw)
    return lib.rtp_paged_select(C.byref(kv) if kv is not None else None, *a.values())


def _evict(lib, kv=None, **kw):
    a = dict(lens=BASE, budget=20, recent=4, sink=2, scores=BASE, pos=BASE, stride=80, os=BASE, op=BASE, ol=BASE, ws=BASE,
             wb=1 << 40, st=None)
    a.update(kw)
    return lib.rtp_paged_evict(C.byref(kv) if kv is not None else None, *a.values())


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(block_table=None), dict(dtype=3), dict(dtype=-1), dict(page_size=8),
    dict(page_size=48), dict(page_size=256), dict(head_dim=96), dict(head_dim=256), dict(n_kv_heads=0), dict(n_pages=0),
    dict(n_seqs=0), dict(n_seqs=70000), dict(max_pages=0), dict(max_pages=6), dict(max_pages=1 << 28, table_stride=1 << 28),
    dict(k_scale=0.0), dict(v_scale=float("nan")), dict(k_scale=float("inf")), dict(k=BASE + 8), dict(bounds=BASE + 4),
    dict(k_stride=(2048, 1024, 60)), dict(k_stride=(2048, 1024, 32)), dict(v_stride=(0, 1024, 64)),
    dict(v_stride=(-2048, 1024, 64)), dict(v_stride=(2048, 1028, 64))])
def test_bad_caches_are_refused(lib, bad):
    kv = _kv(**bad)
    for call in (_append, _decode, _select, _evict):
        assert call(lib, kv) == rtp.RTP_EINVAL
        assert rtp.rtp_last_error(None).startswith("rtp_paged_")
    assert lib.rtp_paged_bounds(C.byref(kv), BASE, None) == rtp.RTP_EINVAL
    assert lib.rtp_paged_decode_workspace(C.byref(kv), 3, 4, 0) == 0
    assert lib.rtp_paged_select_workspace(C.byref(kv), 3, 4) == 0
    assert lib.rtp_paged_evict_workspace(C.byref(kv), 80) == 0


def test_null_cache_is_refused(lib):
    for call in (_append, _decode, _select, _evict):
        assert call(lib) == rtp.RTP_EINVAL
    assert lib.rtp_paged_bounds(None, BASE, None) == rtp.RTP_EINVAL


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(lens=None), dict(q=None), dict(q_out=None), dict(T=0), dict(T=2), dict(dtype=1),
    dict(dtype=2), dict(max_new=0), dict(max_new=4), dict(hq=0), dict(eps=-1.0), dict(eps=float("nan")), dict(base=1.0),
    dict(base=float("inf")), dict(qs=250), dict(ks=120), dict(ks=132), dict(vs=64), dict(os=255), dict(os=512),
    dict(k=BASE + 2), dict(q=BASE + 8), dict(q_out=BASE + 8), dict(qw=BASE + 2), dict(kw=BASE + 4), dict(sp=BASE, sps=79)])
def test_append_refusals(lib, bad):
    assert _append(lib, _kv(), **bad) == rtp.RTP_EINVAL, bad


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(lens=None), dict(out=None), dict(rows=0), dict(rows=4), dict(rows=70000, seq=BASE), dict(hq=3),
    dict(hq=0), dict(hq=130, qs=65536, os=65536), dict(dtype=1), dict(dtype=7), dict(qs=128), dict(qs=257), dict(os=128),
    dict(q=BASE + 8), dict(out=BASE + 8), dict(window=-1), dict(sink=-1), dict(scale=-1.0), dict(scale=float("nan")),
    dict(sel=BASE), dict(sel=BASE, cnt=BASE, ss=0), dict(sel=BASE, cnt=BASE, ss=2, window=4),
    dict(sel=BASE, cnt=BASE, ss=2, scores=BASE, scs=80), dict(scores=BASE, scs=79), dict(scores=BASE, scs=80, seq=BASE),
    dict(ws=None), dict(ws=BASE + 8), dict(wb=0)])
def test_decode_refusals(lib, bad):
    assert _decode(lib, _kv(), **bad) == rtp.RTP_EINVAL, bad


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(lens=None), dict(sel=None), dict(cnt=None), dict(top=0), dict(top=4), dict(first=3), dict(first=-1),
    dict(recent=-1), dict(recent=3), dict(ws=None), dict(wb=8), dict(rows=0), dict(hq=5), dict(dtype=2)])
def test_select_refusals(lib, bad):
    assert _select(lib, _kv(), **bad) == rtp.RTP_EINVAL, bad
    assert _select(lib, _kv(bounds=None)) == rtp.RTP_EINVAL


@pytest.mark.parametrize("bad", [
    dict(lens=None), dict(scores=None), dict(pos=None), dict(os=None), dict(op=None), dict(ol=None), dict(budget=0),
    dict(budget=5), dict(recent=-1), dict(sink=-1), dict(recent=19), dict(stride=79), dict(stride=1 << 25), dict(ws=None),
    dict(wb=100)])
def test_evict_refusals(lib, bad):
    assert _evict(lib, _kv(), **bad) == rtp.RTP_EINVAL, bad


def test_struct_layout_matches_c(tmp_path):
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    f = [n for n, _ in rtp.rtp_paged_kv._fields_]
    src = tmp_path / "p.c"
    src.write_text('#include <stdio.h>\n#include "rtp_paged.h"\nint main(void){printf("%zu", sizeof(rtp_paged_kv));'
                   + "".join(f'printf(" %zu", offsetof(rtp_paged_kv, {n}));' for n in f) + "return 0;}\n")
    exe = str(tmp_path / "p")
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), "-I", "/usr/local/cuda/include", str(src), "-o", exe])
    got = [int(x) for x in subprocess.check_output([exe]).split()]
    assert got == [C.sizeof(rtp.rtp_paged_kv)] + [getattr(rtp.rtp_paged_kv, n).offset for n in f]


# ---------------------------------------------------------------- the binding


def _cache(dtype=torch.float16, d=64, bounds=True, **kw):
    k, v = (torch.zeros((10, 2, 16, d), dtype=dtype) for _ in "kv")
    b = torch.zeros((10, 2, 2, d), dtype=dtype) if bounds else None
    return PagedKV(k, v, torch.zeros((3, 5), dtype=torch.int32), bounds=b, **kw)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_cache_checks():
    k = torch.zeros((10, 2, 16, 64), dtype=torch.float16)
    t = _i(3, 5)
    with pytest.raises(TypeError):
        PagedKV(k.numpy(), k, t)
    for bad in ((k.float(), k.float(), t), (k, k[:5], t), (k, k.bfloat16(), t), (k, k, t.long()), (k, k, t.flatten()),
                (k, k, t.t()), (k.transpose(2, 3), k.transpose(2, 3), t)):
        with pytest.raises(ValueError):
            PagedKV(*bad)
    with pytest.raises(ValueError, match="bounds"):
        PagedKV(k, k, t, bounds=k)
    PagedKV(k.transpose(1, 2).contiguous().transpose(1, 2), k, t)
    PagedKV(k[:1, :1], k[:1, :1], t)


def test_cpu_tensors_reach_no_kernel(lib):
    kv = _cache()
    x, q = torch.zeros((3, 2, 64), dtype=torch.float16), torch.zeros((3, 4, 64), dtype=torch.float16)
    s = torch.zeros((3, 2, 80))
    for call in (lambda: kv.append(q, x, x, _i(3)), lambda: kv.decode(q, _i(3)), lambda: kv.select_pages(q, _i(3), 2),
                 lambda: kv.evict(_i(3), 4, s, _i(3, 2, 80)), lambda: kv.update_bounds(_i(3))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_append_checks():
    kv = _cache()
    x, q = torch.zeros((3, 2, 64), dtype=torch.float16), torch.zeros((3, 4, 64), dtype=torch.float16)
    w = torch.zeros(64, dtype=torch.float16)
    for bad in (dict(k=x[:2]), dict(k=x[:, :1]), dict(v=x.bfloat16()), dict(q=q.float()), dict(k=x.bfloat16(), v=x.bfloat16()),
                dict(seq_lens=_i(2)), dict(seq_lens=_i(3).long()), dict(cu_new=_i(3)), dict(positions=_i(4)),
                dict(q_weight=w.float()), dict(k_weight=w[:32]), dict(slot_positions=_i(3, 2, 79)),
                dict(slot_positions=_i(2, 2, 80)), dict(q_out=q[:, :2]), dict(q=None, q_out=q),
                dict(q=torch.zeros((3, 64, 4), dtype=torch.float16).transpose(1, 2))):
        with pytest.raises(ValueError):
            kv.append(**{**dict(q=q, k=x, v=x, seq_lens=_i(3)), **bad})
    with pytest.raises(TypeError):
        kv.append(q, x, x.numpy(), _i(3))
    two = torch.zeros((2, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="cu_new"):
        kv.append(None, two, two, _i(3))


def test_decode_checks():
    kv = _cache()
    q, s = torch.zeros((3, 4, 64), dtype=torch.float16), torch.zeros((3, 2, 80))
    sel, cnt = _i(3, 2, 4), _i(3, 2)
    for bad in (dict(q=q.bfloat16()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(seq_lens=_i(4)), dict(row_seq=_i(2)),
                dict(scores=s[:, :1]), dict(scores=s.half()), dict(scores=s[..., :79]), dict(out=q[:2]),
                dict(out=q.bfloat16()), dict(pages=(sel[:2], cnt)), dict(pages=(sel, cnt[:, :1])),
                dict(pages=(sel.long(), cnt)), dict(q=torch.zeros((4, 4, 64), dtype=torch.float16), seq_lens=_i(4))):
        with pytest.raises(ValueError):
            kv.decode(**{**dict(q=q, seq_lens=_i(3)), **bad})


def test_select_and_evict_checks():
    kv = _cache()
    q, s, p = torch.zeros((3, 4, 64), dtype=torch.float16), torch.zeros((3, 2, 80)), _i(3, 2, 80)
    with pytest.raises(ValueError, match="bounds"):
        _cache(bounds=False).select_pages(q, _i(3), 2)
    with pytest.raises(ValueError, match="bounds"):
        _cache(bounds=False).update_bounds(_i(3))
    with pytest.raises(ValueError):
        kv.select_pages(q, _i(3), 0)
    for bad in (dict(scores=s.double()), dict(positions=s), dict(scores=s[:, :, :64]), dict(seq_lens=_i(2)),
                dict(positions=_i(3, 2, 96)), dict(out_scores=s[:2]), dict(out_positions=p.long())):
        with pytest.raises(ValueError):
            kv.evict(**{**dict(seq_lens=_i(3), budget=4, scores=s, positions=p), **bad})
