"""Paged-cache operators: host checks at the edges of what the arguments allow (no GPU needed)."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import long_context_sparse_idx16_b200 as rtp  # noqa: E402
from long_context_sparse_idx16_b200 import build as rtp_build  # noqa: E402

BASE = 1 << 20  # a 16-byte aligned address that no host check dereferences


@pytest.fixture(scope="module")
def lib():
    rtp_build.build()
    return rtp.lib()


def _kv(**kw):
    a = dict(k=BASE, v=BASE, n_pages=10, page_size=16, n_kv_heads=2, head_dim=64, dtype=0, k_scale=1.0, v_scale=1.0,
             block_table=BASE, table_stride=5, max_pages=5, n_seqs=3, bounds=BASE, err=BASE)
    a.update(kw)
    s = (C.c_int64 * 3)(2048, 1024, 64)
    return rtp.rtp_paged_kv(k_stride=s, v_stride=s, **a)


def test_take_errors_refusals(lib):
    assert lib.rtp_paged_take_errors(None, BASE, None) == rtp.RTP_EINVAL
    for kv, bits in ((_kv(err=None), BASE), (_kv(), None)):
        assert lib.rtp_paged_take_errors(C.byref(kv), bits, None) == rtp.RTP_EINVAL
        assert rtp.rtp_last_error(None).startswith("rtp_paged_take_errors")


def _decode(lib, kv, **kw):
    a = dict(q=BASE, dtype=0, qs=256, rows=3, hq=4, seq=None, lens=BASE, window=0, sink=0, scale=0.0, sel=None, cnt=None,
             ss=0, out=BASE, os=256, lse=None, scores=None, scs=0, ws=BASE, wb=0, st=None)
    a.update(kw)
    return lib.rtp_paged_decode(C.byref(kv), *a.values())


def test_decode_refuses_scales_beyond_fp32(lib):
    """Infinite, the product made every row NaN; as zero, it stood for the default."""
    assert _decode(lib, _kv(k_scale=1e30), scale=1e30, wb=1 << 40) == rtp.RTP_EINVAL
    assert "sm_scale" in rtp.rtp_last_error(None)
    assert _decode(lib, _kv(k_scale=1e30), scale=1e-30) == rtp.RTP_EINVAL  # (passes, up to the workspace)
    assert "workspace" in rtp.rtp_last_error(None)
    with pytest.raises(ValueError, match="sm_scale"):
        _cache().decode(torch.zeros((3, 4, 64), dtype=torch.float16), _ints(3), sm_scale=1e-50)


FAR = 1 << 30  # between the arrays: each of three sequences, two heads and 80 slots is 1920 bytes


def _evict(lib, **kw):
    a = dict(lens=BASE, budget=20, recent=4, sink=2, scores=2 * FAR, pos=3 * FAR, stride=80, os=4 * FAR, op=5 * FAR, ol=6 * FAR,
             ws=7 * FAR, wb=8, st=None)
    a.update(kw)
    return lib.rtp_paged_evict(C.byref(_kv()), *a.values())


def test_evict_refuses_arrays_that_share_memory(lib):
    """The heads' CTAs would write what others still read; a call in place is none of these.  (The
    workspace given is too small: what passes ends there.)"""
    def why(**kw):
        assert _evict(lib, **kw) == rtp.RTP_EINVAL
        return rtp.rtp_last_error(None)

    small = why()
    assert "workspace" in small
    for ok in (dict(os=2 * FAR, op=3 * FAR), dict(os=2 * FAR), dict(op=3 * FAR), dict(os=2 * FAR + 1920), dict(ol=BASE + 12)):
        assert why(**ok) == small, ok
    for bad in (dict(ol=BASE), dict(ol=BASE + 8), dict(os=2 * FAR + 4), dict(os=2 * FAR - 1916), dict(op=3 * FAR + 1916),
                dict(os=3 * FAR), dict(op=2 * FAR), dict(op=4 * FAR + 320), dict(ol=2 * FAR + 64), dict(ol=3 * FAR),
                dict(ol=4 * FAR + 1912), dict(ol=5 * FAR - 8), dict(lens=4 * FAR), dict(lens=5 * FAR + 640)):
        got = why(**bad)
        assert got != small and ("must not" in got), (bad, got)


# ---------------------------------------------------------------- the binding


def _cache():
    k = torch.zeros((10, 2, 16, 64), dtype=torch.float16)
    return rtp.PagedKV(k, k, torch.zeros((3, 5), dtype=torch.int32), bounds=torch.zeros((10, 2, 2, 64), dtype=torch.float16))


def _ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_page_lists_of_no_pages_are_refused():
    """They were taken for no list at all: attention to every slot."""
    q = torch.zeros((3, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="at least 1"):
        _cache().decode(q, _ints(3), pages=(_ints(3, 2, 0), _ints(3, 2)))
    with pytest.raises(ValueError, match="CUDA device"):  # the next thing that is looked at
        _cache().decode(q, _ints(3), pages=(_ints(3, 2, 1), _ints(3, 2)))


# ---------------------------------------------------------------- building


@pytest.fixture
def binding(tmp_path, monkeypatch):
    """build_binding() in a folder of its own, with the compiler's calls recorded instead of run."""
    calls = []

    def run(cmd):
        calls.append(cmd)
        open(rtp_build.EXT, "w").close()

    monkeypatch.setattr(rtp_build, "EXT", str(tmp_path / "_paged.so"))
    monkeypatch.setattr(rtp_build, "EXT_FOR", str(tmp_path / "_paged.torch"))
    monkeypatch.setattr(rtp_build.subprocess, "check_call", run)
    return calls


def test_library_builds_without_torch(lib, binding, monkeypatch, capsys):
    import sys

    monkeypatch.setitem(sys.modules, "torch", None)  # an import of it fails
    assert rtp_build.build() == rtp_build.LIB
    assert not binding and "torch is not installed" in capsys.readouterr().err


def test_binding_is_rebuilt_for_another_torch(lib, binding, monkeypatch):
    rtp_build.build()
    rtp_build.build()
    assert len(binding) == 1
    monkeypatch.setattr(rtp_build.importlib.metadata, "version", lambda name: "0.0")
    rtp_build.build()
    rtp_build.build()
    assert len(binding) == 2
