"""Host side of drafts and of a bounded cache (no GPU): pa_seq_truncate and
pa_seq_compact against a model of tables and reference counts, their
refusals, and the argument checks of the device calls that use them."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_106_gb300 as pk


class Model:
    """Tables, counts and the free queue, by the calls' descriptions."""

    def __init__(self, order, B):
        self.B, self.free, self.ref = B, list(order), {b: 0 for b in order}
        self.seqs = {}

    def take(self):
        b = self.free.pop(0)
        self.ref[b] = 1
        return b

    def drop(self, b):
        self.ref[b] -= 1
        if self.ref[b] == 0:
            self.free.append(b)

    def add(self, s, n):
        self.seqs[s] = [[self.take() for _ in range(-(-n // self.B))], n]

    def fork(self, a, b):
        self.seqs[b] = [list(self.seqs[a][0]), self.seqs[a][1]]
        for x in self.seqs[b][0]:
            self.ref[x] += 1

    def truncate(self, s, n):
        t = self.seqs[s]
        while len(t[0]) > -(-n // self.B):
            self.drop(t[0].pop())
        t[1] = n

    def compact(self, ids, lens):
        shared = [(i, j) for i, (s, n) in enumerate(zip(ids, lens)) if n != self.seqs[s][1]
                  for j in range(-(-n // self.B)) if self.ref[self.seqs[s][0][j]] > 1]
        if len(shared) > len(self.free):
            return False
        for i, j in shared:
            t = self.seqs[ids[i]][0]
            old, t[j] = t[j], self.take()
            self.drop(old)
        for s, n in zip(ids, lens):
            self.truncate(s, n)
        return True


def _same(pool, m, NB):
    assert pk.pa_pool_free_queue(pool, NB).tolist() == m.free
    assert pk.pa_pool_refcounts(pool, NB).tolist() == [m.ref[b] for b in range(NB)]
    for s, (t, n) in m.seqs.items():
        tables, ctx = pk.pa_get_block_tables(pool, [s], NB)
        assert tables[0].tolist() == t + [-1] * (NB - len(t)) and ctx[0] == n


@pytest.mark.parametrize("seed", range(6))
def test_random_shortening_against_the_model(seed):
    r = np.random.default_rng(seed)
    NB, B = 40, int(r.choice([1, 3, 4, 8]))
    order = r.permutation(NB).tolist()
    pool = pk.pa_pool_create(pk.PoolDesc(NB, B, free_order=order))
    m, next_id = Model(order, B), 0
    for _ in range(300):
        op = r.integers(0, 5)
        ids = list(m.seqs)
        if op == 0 or not ids:
            n = int(r.integers(0, 6 * B))
            if -(-n // B) <= len(m.free):
                pk.pa_seq_add(pool, next_id, n)
                m.add(next_id, n)
                next_id += 1
        elif op == 1 and len(ids) < 12:
            a = int(r.choice(ids))
            pk.pa_seq_fork(pool, a, next_id)
            m.fork(a, next_id)
            next_id += 1
        elif op == 2:
            s = int(r.choice(ids))
            pk.pa_seq_free(pool, s)
            m.truncate(s, 0)
            del m.seqs[s]
        else:
            some = [int(x) for x in r.permutation(ids)[:r.integers(1, 4)]]
            lens = [int(r.integers(0, m.seqs[s][1] + 1)) for s in some]
            if op == 3:
                pk.pa_seq_truncate(pool, some, lens)
                for s, n in zip(some, lens):
                    m.truncate(s, n)
            else:
                before = [(list(m.seqs[s][0]), m.seqs[s][1]) for s in some]
                if m.compact(some, lens):
                    src, src_lens, dst = pk.pa_seq_compact(pool, some, lens, NB)
                    for i, s in enumerate(some):
                        t, n = before[i]
                        assert src[i].tolist() == t + [-1] * (NB - len(t)) and src_lens[i] == n
                        t = m.seqs[s][0]
                        assert dst[i].tolist() == t + [-1] * (NB - len(t))
                    # a destination is the block that was there, or none that is read
                    read = set(src[src >= 0].tolist())
                    assert all(d == x or d not in read for d, x in zip(dst.ravel(), src.ravel())
                               if d >= 0)
                else:
                    with pytest.raises(pk.OutOfBlocks):
                        pk.pa_seq_compact(pool, some, lens, NB)
        _same(pool, m, NB)
    pk.pa_pool_destroy(pool)


def test_a_shortened_prompt_block_leaves_the_prefix_cache():
    B = 4
    pool = pk.pa_pool_create(pk.PoolDesc(12, B, flags=pk.PA_POOL_PREFIX_CACHING))
    toks = list(range(13))
    pk.pa_seq_add_tokens(pool, 0, toks)
    assert pk.pa_pool_cached_blocks(pool) == 3
    pk.pa_seq_truncate(pool, [0], [8])         # whole blocks: both stay cached, the third too (free)
    assert pk.pa_pool_cached_blocks(pool) == 3
    pk.pa_seq_truncate(pool, [0], [6])         # its second block will be written into
    assert pk.pa_pool_cached_blocks(pool) == 2
    assert pk.pa_seq_add_tokens(pool, 1, toks)[1] == 4      # one block to reuse
    src, lens, dst = pk.pa_seq_compact(pool, [0], [3], 4)
    # block 0 is shared with sequence 1: replaced, and cached as it was
    assert dst[0, 0] != src[0, 0] and lens[0] == 6
    assert pk.pa_seq_add_tokens(pool, 2, toks)[1] == 12
    pk.pa_seq_free_batch(pool, [1, 2])
    src, lens, dst = pk.pa_seq_compact(pool, [0], [2], 4)
    assert dst[0, 0] == src[0, 0]              # alone: in place
    pk.pa_pool_destroy(pool)


def test_a_block_rewritten_in_place_leaves_the_prefix_cache():
    pool = pk.pa_pool_create(pk.PoolDesc(8, 4, flags=pk.PA_POOL_PREFIX_CACHING))
    toks = list(range(12))
    pk.pa_seq_add_tokens(pool, 0, toks)
    src, lens, dst = pk.pa_seq_compact(pool, [0], [8], 3)
    assert (dst[0, :2] == src[0, :2]).all() and dst[0, 2] == -1
    assert pk.pa_seq_add_tokens(pool, 1, toks)[1] == 0
    pk.pa_pool_destroy(pool)


def test_refusals_change_nothing():
    pool = pk.pa_pool_create(pk.PoolDesc(6, 4))
    pk.pa_seq_add(pool, 0, 9)
    pk.pa_seq_add(pool, 1, 8)
    pk.pa_seq_fork(pool, 0, 2)
    free = pk.pa_pool_free_queue(pool, 6).tolist()
    for call in (lambda i, n: pk.pa_seq_truncate(pool, i, n),
                 lambda i, n: pk.pa_seq_compact(pool, i, n, 8)):
        for ids, lens, code in (([0, 7], [1, 1], pk.PA_ERR_NO_SEQ),
                                ([0, 0], [1, 1], pk.PA_ERR_INVALID_ARG),
                                ([1, 0], [1, 10], pk.PA_ERR_INVALID_ARG),
                                ([1, 0], [1, -1], pk.PA_ERR_INVALID_ARG)):
            with pytest.raises(pk.PagedKVError) as e:
                call(ids, lens)
            assert e.value.code == code
        with pytest.raises(ValueError):
            call([0], [1, 2])
    with pytest.raises(pk.PagedKVError):
        pk.pa_seq_compact(pool, [1, 0], [1, 1], 2)        # three blocks, two columns
    with pytest.raises(pk.OutOfBlocks):
        pk.pa_seq_compact(pool, [0, 2], [8, 8], 3)        # four shared blocks, one free
    assert pk.pa_pool_free_queue(pool, 6).tolist() == free
    assert [pk.pa_seq_info(pool, s) for s in (0, 1, 2)] == [(9, 3), (8, 2), (9, 3)]
    pk.pa_pool_destroy(pool)


# ------------------------------------------- argument checks of device calls

I32, F = ctypes.c_int32, ctypes.c_float
A = 4096          # an aligned address that no refused call touches


def _desc(**kw):
    return pk.PoolDesc(**{"num_blocks": 8, "block_size": 16, "num_heads": 2, "head_dim": 64, **kw})


def _call(name, args, changed):
    args = {**args, **changed}
    d = args.pop("desc")
    vals = [*args.values(), None if d is None else d.ref] if d != "none" else list(args.values())
    if name == "pa_compact_kv":
        vals = [*list(args.values()), d.ref if d is not None else None]
    tail = {"pa_tree_attention": 1, "pa_decode_attention_weights": 1}.get(name)
    if tail:
        return getattr(pk._lib, name)(*vals, None)
    if name == "pa_compact_kv":
        return getattr(pk._lib, name)(*vals, A, None)
    return getattr(pk._lib, name)(*vals, None)


TREE = {"out": A, "q": A, "k": A, "v": A, "tables": A, "ctx": A, "starts": A, "parents": A,
        "n_seqs": 2, "max_blocks": 4, "max_q": 8, "rows": 9, "scale": 1.0, "ws": A, "bytes": 1 << 40,
        "status": A, "desc": _desc()}
TREE_BAD = [{"desc": None}, {"desc": _desc(head_dim=32)}, {"desc": _desc(head_dim=256)},
            {"desc": _desc(block_size=4)}, {"desc": _desc(num_blocks=0)}, {"n_seqs": -1},
            {"n_seqs": 4097}, {"max_blocks": -1}, {"max_blocks": 0}, {"max_blocks": 1 << 28},
            {"max_q": 65}, {"max_q": -1}, {"rows": -1}, {"scale": float("nan")}, {"ws": None},
            {"ws": A + 16}, {"bytes": 100}, {"out": None}, {"q": A + 2}, {"k": A + 8}, {"v": None},
            {"tables": None}, {"ctx": None}, {"starts": None}, {"starts": A + 2}, {"parents": A + 1}]


@pytest.mark.parametrize("changed", TREE_BAD, ids=str)
def test_tree_attention_refuses(changed):
    assert _call("pa_tree_attention", TREE, changed) == pk.PA_ERR_INVALID_ARG
    assert pk.pa_last_error_string().startswith("pa_tree_attention")


WEIGHTS = {"out": A, "w_out": A, "w_in": A, "w_len": 64, "q": A, "k": A, "v": A, "tables": A,
           "ctx": A, "n_seqs": 2, "max_blocks": 4, "scale": 1.0, "ws": A, "bytes": 1 << 40,
           "status": A, "desc": _desc()}


@pytest.mark.parametrize("changed", [{"desc": None}, {"desc": _desc(head_dim=16)},
                                     {"desc": _desc(block_size=4)}, {"n_seqs": 4097},
                                     {"n_seqs": -1}, {"max_blocks": 0}, {"w_len": -1},
                                     {"scale": float("inf")}, {"ws": None}, {"ws": A + 128},
                                     {"bytes": 0}, {"w_out": None}, {"w_out": A + 2},
                                     {"w_in": A + 1}, {"q": None}, {"out": A + 4}, {"ctx": None}],
                         ids=str)
def test_decode_attention_weights_refuses(changed):
    assert _call("pa_decode_attention_weights", WEIGHTS, changed) == pk.PA_ERR_INVALID_ARG
    assert pk.pa_last_error_string().startswith("pa_decode_attention_weights")


VERIFY = {"path": A, "lens": A, "next": A, "p": A, "q": A, "dtype": pk.PA_DTYPE_F32, "tokens": A,
          "parents": A, "starts": A, "u": A, "us": A, "n_seqs": 2, "max_q": 8, "rows": 9,
          "vocab": 100, "status": A, "desc": "none"}


@pytest.mark.parametrize("changed", [{"dtype": 3}, {"dtype": -1}, {"n_seqs": -1}, {"n_seqs": 65536},
                                     {"max_q": 0}, {"max_q": 65}, {"rows": -1}, {"vocab": 0},
                                     {"path": None}, {"lens": None}, {"next": None}, {"p": None},
                                     {"p": A + 2}, {"q": A + 2}, {"tokens": None}, {"starts": None},
                                     {"u": None}, {"us": None}, {"us": A + 2}], ids=str)
def test_verify_draft_refuses(changed):
    assert _call("pa_verify_draft", VERIFY, changed) == pk.PA_ERR_INVALID_ARG
    assert pk.pa_last_error_string().startswith("pa_verify_draft")


SELECT = {"keep": A, "lens": A, "w_out": A, "w_in": A, "w_len": 64, "ctx": A, "n_seqs": 2, "heads": 2,
          "budget": 8, "recent": 2, "status": A, "desc": "none"}


@pytest.mark.parametrize("changed", [{"keep": None}, {"lens": None}, {"w_out": None}, {"w_in": None},
                                     {"w_len": -1}, {"ctx": None}, {"n_seqs": -1},
                                     {"n_seqs": 65536}, {"heads": 0}, {"budget": 0}, {"recent": -1},
                                     {"recent": 9}, {"keep": A + 2}], ids=str)
def test_evict_select_refuses(changed):
    assert _call("pa_evict_select", SELECT, changed) == pk.PA_ERR_INVALID_ARG
    assert pk.pa_last_error_string().startswith("pa_evict_select")


def _caches(*addresses):
    return (ctypes.c_void_p * len(addresses))(*addresses)


COMPACT = {"k": _caches(A, A), "v": _caches(A, A), "layers": 2, "src": A, "dst": A, "src_lens": A,
           "first": A, "keep": A, "keep_lens": A, "heads": 1, "stride": 8, "n_seqs": 2,
           "max_blocks": 4, "desc": _desc()}


@pytest.mark.parametrize("changed", [{"desc": None}, {"desc": _desc(head_dim=24)}, {"layers": -1},
                                     {"layers": 129}, {"k": None}, {"v": _caches(A, None)},
                                     {"k": _caches(A, A + 8)}, {"src": None}, {"dst": None},
                                     {"src_lens": None}, {"keep": None}, {"keep_lens": None},
                                     {"heads": 3}, {"heads": 0}, {"stride": -1}, {"n_seqs": -1},
                                     {"max_blocks": -1}, {"first": A + 2}],
                         ids=lambda c: ",".join(c))
def test_compact_kv_refuses(changed):
    assert _call("pa_compact_kv", COMPACT, changed) == pk.PA_ERR_INVALID_ARG
    assert pk.pa_last_error_string().startswith("pa_compact_kv")


def test_nothing_to_do_is_no_call():
    assert _call("pa_tree_attention", TREE, {"n_seqs": 0, "ws": None}) == pk.PA_OK
    assert _call("pa_tree_attention", TREE, {"rows": 0}) == pk.PA_OK
    assert _call("pa_decode_attention_weights", WEIGHTS, {"n_seqs": 0}) == pk.PA_OK
    assert _call("pa_verify_draft", VERIFY, {"n_seqs": 0}) == pk.PA_OK
    assert _call("pa_evict_select", SELECT, {"n_seqs": 0}) == pk.PA_OK
    for changed in ({"layers": 0}, {"n_seqs": 0}, {"stride": 0}):
        assert _call("pa_compact_kv", COMPACT, changed) == pk.PA_OK


def test_workspace_sizes():
    d = _desc(num_heads=40, head_dim=128)
    assert pk.pa_tree_workspace_bytes(1, 128, 8, d) > 0
    assert pk.pa_tree_workspace_bytes(1, 128, 64, d) >= pk.pa_tree_workspace_bytes(1, 128, 8, d)
    for bad in ((0, 128, 8), (4097, 128, 8), (1, -1, 8), (1, 128, 0), (1, 128, 65)):
        assert pk.pa_tree_workspace_bytes(*bad, d) == 0
    assert pk.pa_decode_weights_workspace_bytes(2, 128, d) >= 2 * 40 * 2048 * 4
    assert pk.pa_decode_weights_workspace_bytes(0, 128, d) == 0
    assert pk.pa_decode_weights_workspace_bytes(2, 128, _desc(head_dim=32)) == 0
