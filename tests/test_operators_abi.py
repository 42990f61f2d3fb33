"""Host-side refusals of the rotated append, scored attention and shared-prefix
attention: documented statuses before anything touches a GPU.  CPU only."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from kv_cache_decode_append_gb300 import build as kbuild
    from kv_cache_decode_append_gb300 import kvd
    kbuild.build()
    return kvd.load()


# A fake, 256-byte aligned address: every call below is refused on the host
# before any pointer is dereferenced or any CUDA call is made.
A = 1 << 20
OK, INVALID, CAPACITY, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
F32, BF16, F16, E4M3 = 0, 1, 2, 3


def _rope(lib, q=A, q_out=A, k=A, v=A, kn=A, vn=A, strides=None, past=A, positions=None, freq=A, rot=64, pairs=0, B=1,
          H_q=4, H_kv=2, T_max=64, D=64, N=1, max_past=10, dtype=BF16):
    return lib.kvd_rope_append(q, q_out, k, v, kn, vn, strides, past, positions, 0, freq, rot, pairs, B, H_q, H_kv,
                               T_max, D, N, max_past, dtype, None, None)


def _paged_rope(lib, q=A, q_out=A, k=A, v=A, kn=A, vn=A, strides=None, table=A, past=A, positions=None, freq=A, rot=64,
                pairs=0, B=1, H_q=4, H_kv=2, D=64, N=1, page_size=64, max_pages=1, num_pages=8, max_past=10,
                dtype=BF16):
    return lib.kvd_paged_rope_append(q, q_out, k, v, kn, vn, strides, table, past, positions, 0, freq, rot, pairs, B,
                                     H_q, H_kv, D, N, page_size, max_pages, num_pages, max_past, dtype, None, None)


@pytest.mark.parametrize("call", [_rope, _paged_rope])
def test_rope_append_refusals(lib, call):
    for name in ("q", "q_out", "k", "v", "kn", "vn", "past", "freq"):
        assert call(lib, **{name: None}) == INVALID, name
    for name in ("q", "q_out", "k", "v", "kn", "vn"):
        assert call(lib, **{name: A + 8}) == INVALID, name
    assert call(lib, freq=A + 4) == INVALID
    assert call(lib, B=-1) == INVALID
    assert call(lib, H_q=0) == INVALID
    assert call(lib, N=0) == INVALID
    assert call(lib, max_past=-1) == INVALID
    assert call(lib, rot=0) == INVALID
    assert call(lib, rot=33) == INVALID
    assert call(lib, rot=66) == INVALID           # more than the row
    assert call(lib, rot=24) == UNSUPPORTED       # halves of 12: not whole 16-byte chunks
    assert call(lib, rot=20, pairs=1) == UNSUPPORTED
    assert call(lib, rot=24, pairs=1, B=0) == OK
    assert call(lib, D=68) == UNSUPPORTED
    assert call(lib, D=8192) == UNSUPPORTED
    assert call(lib, dtype=E4M3) == UNSUPPORTED
    assert call(lib, dtype=9) == UNSUPPORTED
    assert call(lib, max_past=60, N=5) == CAPACITY
    assert call(lib, max_past=(1 << 31) - 1) == CAPACITY
    assert call(lib, strides=(ctypes.c_int64 * 9)(256, 64, 64, 128, 64, 64, 128, -64, 64)) == INVALID
    assert call(lib, strides=(ctypes.c_int64 * 9)(256, 64, 60, 128, 64, 64, 128, 64, 64)) == INVALID
    assert call(lib, B=0) == OK


def test_paged_rope_append_geometry(lib):
    assert _paged_rope(lib, table=None) == INVALID
    assert _paged_rope(lib, page_size=48) == INVALID
    assert _paged_rope(lib, page_size=32) == INVALID
    assert _paged_rope(lib, max_pages=0) == INVALID
    assert _paged_rope(lib, num_pages=0) == INVALID
    assert _paged_rope(lib, max_pages=1 << 26) == INVALID


class _Score(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("window", ctypes.c_int),
                ("doc_start", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p)]


def _scored(lib, score=(), q=A, k=A, v=A, out=A, past=A, B=1, H_q=4, H_kv=2, T_max=64, D=64, N=1, max_past=10,
            dtype=BF16):
    s = None if score is None else ctypes.byref(_Score(*score))
    return lib.kvd_decode_attention_scored(q, k, v, out, past, _cast(s), B, H_q, H_kv, T_max, D, N, max_past, 0.0,
                                           dtype, None, 0, None, None)


def _paged_scored(lib, score=(), q=A, k=A, v=A, out=A, table=A, past=A, B=1, H_q=4, H_kv=2, D=64, N=1, page_size=64,
                  max_pages=1, num_pages=8, max_past=10, dtype=BF16):
    s = None if score is None else ctypes.byref(_Score(*score))
    return lib.kvd_paged_decode_attention_scored(q, k, v, out, table, past, _cast(s), B, H_q, H_kv, D, N, page_size,
                                                 max_pages, num_pages, max_past, 0.0, dtype, None, 0, None, None)


def _cast(s):
    from kv_cache_decode_append_gb300 import kvd
    return None if s is None else ctypes.cast(s, ctypes.POINTER(kvd.Score))


@pytest.mark.parametrize("call", [_scored, _paged_scored])
def test_scored_attention_refusals(lib, call):
    assert call(lib, score=None) == INVALID
    for name in ("q", "k", "v", "out", "past"):
        assert call(lib, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "out"):
        assert call(lib, **{name: A + 8}) == INVALID, name
    for cap in (-1.0, float("inf"), float("nan")):
        assert call(lib, score=(cap,)) == INVALID
    assert call(lib, score=(0.0, None, -1)) == INVALID
    assert call(lib, score=(0.0, A + 2)) == INVALID
    assert call(lib, score=(0.0, None, 0, A + 1)) == INVALID
    assert call(lib, score=(0.0, None, 0, None, A + 3)) == INVALID
    assert call(lib, H_q=3) == INVALID
    assert call(lib, N=0) == INVALID
    assert call(lib, D=96) == UNSUPPORTED
    assert call(lib, dtype=E4M3) == UNSUPPORTED
    assert call(lib, H_q=16, H_kv=1, N=65, max_past=0) == UNSUPPORTED
    assert call(lib, max_past=64) == CAPACITY
    assert call(lib, score=(2.0, A, 5, A, A), B=0) == OK


def test_scored_workspace_query_rejects_bad_shapes(lib):
    assert lib.kvd_decode_scored_workspace_bytes(1, 3, 2, 64, 1, 10, BF16) == 0
    assert lib.kvd_decode_scored_workspace_bytes(1, 4, 2, 80, 1, 10, BF16) == 0
    assert lib.kvd_decode_scored_workspace_bytes(1, 4, 2, 128, 1, 10, E4M3) == 0


def _prefix(lib, q=A, kp=A, vp=A, k=A, v=A, out=A, past=A, B=1, H_q=4, H_kv=2, S_max=64, T_max=64, D=64, N=1, S=10,
            max_past=10, dtype=BF16):
    return lib.kvd_shared_prefix_attention(q, kp, vp, k, v, out, past, B, H_q, H_kv, S_max, T_max, D, N, S, max_past,
                                           0.0, dtype, None, 0, None, None)


def _paged_prefix(lib, q=A, k=A, v=A, out=A, ptable=A, table=A, past=A, B=1, H_q=4, H_kv=2, D=64, N=1, page_size=64,
                  max_pages=1, num_pages=8, S=10, max_past=10, dtype=BF16):
    return lib.kvd_paged_shared_prefix_attention(q, k, v, out, ptable, table, past, B, H_q, H_kv, D, N, page_size,
                                                 max_pages, num_pages, S, max_past, 0.0, dtype, None, 0, None, None)


@pytest.mark.parametrize("call", [_prefix, _paged_prefix])
def test_shared_prefix_refusals(lib, call):
    for name in ("q", "k", "v", "out", "past"):
        assert call(lib, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "out"):
        assert call(lib, **{name: A + 8}) == INVALID, name
    assert call(lib, S=-1) == INVALID
    assert call(lib, H_q=3) == INVALID
    assert call(lib, N=0) == INVALID
    assert call(lib, B=-1) == INVALID
    assert call(lib, D=96) == UNSUPPORTED
    assert call(lib, dtype=E4M3) == UNSUPPORTED
    assert call(lib, H_q=16, H_kv=1, N=65, max_past=0) == UNSUPPORTED
    assert call(lib, max_past=64) == CAPACITY
    assert call(lib, B=0) == OK


def test_shared_prefix_refuses_its_own_arguments(lib):
    assert _prefix(lib, kp=None) == INVALID
    assert _prefix(lib, vp=A + 4) == INVALID
    assert _prefix(lib, S=65) == CAPACITY
    assert _prefix(lib, kp=None, vp=None, S=0, B=0) == OK
    assert _paged_prefix(lib, ptable=None) == INVALID
    assert _paged_prefix(lib, ptable=A + 2) == INVALID
    assert _paged_prefix(lib, S=8 * 64 + 1) == CAPACITY
    assert _paged_prefix(lib, page_size=32) == INVALID
    assert lib.kvd_shared_prefix_workspace_bytes(1, 4, 2, 64, 1, -1, 10, BF16) == 0
    assert lib.kvd_shared_prefix_workspace_bytes(1, 3, 2, 64, 1, 10, 10, BF16) == 0


def test_rope_append_unit_bound(lib):
    """A token's 16-byte units: below 2^26, as their divisions assume."""
    assert _rope(lib, H_q=(1 << 24), H_kv=1, D=64, dtype=BF16) == UNSUPPORTED  # 4 pairs of chunks a row
    assert _rope(lib, H_q=(1 << 24), H_kv=1, D=64, dtype=BF16, B=0) == OK
