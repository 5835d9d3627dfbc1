"""Arguments of the calls for drafted tokens and for the bounded cache that are
refused, or taken, on the host (none of these addresses is ever read)."""
import ctypes

import pytest

import paged_kv_cache_106_gb300 as pk

A = 1 << 24            # an aligned address that nothing reads
DESC = pk.PoolDesc(8, 16, num_layers=2, num_heads=2, head_dim=64)
SIZE = 8 * 16 * 2 * 64 * 2             # bytes of a cache


def _compact(k, v):
    L = len(k)
    return pk._lib.pa_compact_kv((ctypes.c_void_p * L)(*k), (ctypes.c_void_p * L)(*v), L, A, A, A, None,
                                 A, A, 1, 4, 2, 4, DESC.ref, None, 0)


@pytest.mark.parametrize("k,v", [([A], [A]), ([A, A], [A + SIZE, A + 2 * SIZE]),
                                 ([A, A + SIZE], [A + 2 * SIZE, A + SIZE]),
                                 ([A], [A + SIZE - 16]), ([A + SIZE - 16], [A]),
                                 ([A + 3 * SIZE, A], [A + SIZE, A + 3 * SIZE - 16])])
def test_moves_refuse_caches_that_overlap(k, v):
    """Each cache is moved by blocks of its own, in any order: moved twice, its
    rows would be read after they were written over."""
    assert _compact(k, v) == pk.PA_ERR_INVALID_ARG
    assert "overlap" in pk.pa_last_error_string()
