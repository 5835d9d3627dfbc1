"""Arguments of the calls for drafted tokens, for the bounded cache and of the
one-call steps that are refused, or taken, on the host (none of these addresses
is ever read)."""
import ctypes

import pytest
import torch

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


def test_one_call_steps_refuse_addresses_of_new_rows():
    """How many rows lie there cannot be checked."""
    q, tables, ctx = torch.zeros(3, 2, 64), torch.zeros(3, 4), torch.zeros(3)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="k_new"):
        pk.pa_decode_step_attention(q, q, A, q, slots, q, q, tables, ctx, 0.1, DESC)
    with pytest.raises(ValueError, match="slot_mapping"):
        pk.pa_decode_step_attention(q, q, q, q, A, q, q, tables, ctx, 0.1, DESC)
    with pytest.raises(ValueError, match="v_new"):
        pk.pa_prefill_step_attention(q, q, q, A, q, q, tables, ctx, ctx, 0.1, DESC, max_q_len=3)
