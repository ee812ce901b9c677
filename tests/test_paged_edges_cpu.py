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
    for kv, bits in ((_kv(err=None), BASE), (_kv(), None), (_kv(page_size=8), BASE)):
        assert lib.rtp_paged_take_errors(C.byref(kv), bits, None) == rtp.RTP_EINVAL
        assert rtp.rtp_last_error(None).startswith("rtp_paged_take_errors")
