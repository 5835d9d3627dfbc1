"""A bounded cache on the GPU: decode attention that adds up the positions'
weights, the selection of what a budget keeps, and the move of kept rows,
against plain evaluations in 64 bits; their reports; and decode steps of a
budgeted sequence through the block manager.

Weights: a score of D fp32-accumulated products errs by at most
D * 2^-24 * scale * log2 e * sum |q k| < 2^-13 here, which is a weight's
relative error, once more in the sum it is divided by; the running sum is
rounded once (2^-24).  Selection and moves are exact.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_106_gb300 as pk
from tests.test_gpu_drafts import Batch, _dev, _i32, _status

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- weights of positions


def _run_weights(b, w_in, w_len, in_place=False, status=None):
    S = len(b.ctx)
    desc = pk.PoolDesc(b.nb, b.B, num_heads=b.H, head_dim=b.D)
    out = torch.full((S, b.H, b.D), 7.0, dtype=torch.float16, device="cuda")
    w_out = w_in if in_place else torch.full((S, b.H, w_len), -3.0, device="cuda")
    need = pk.pa_decode_weights_workspace_bytes(S, b.tables.shape[1], desc)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    pk.pa_decode_attention_weights(out, w_out, w_in, b.q[:S], b.k, b.v, _dev(b.tables),
                                   _i32(b.ctx), b.scale, desc, workspace=ws, status=status)
    return out, w_out


def _check_weights(b, out, w_out, w_in, rest):
    for i, c in enumerate(b.ctx):
        assert torch.equal(w_out[i, :, max(c, 0):], rest[i, :, max(c, 0):])
        if c <= 0:
            assert bool((out[i] == 0).all())
            continue
        x = torch.einsum("hd,phd->hp", b.q[i].double(), b.rows64(b.k, i)) * b.scale
        p = torch.softmax(x, -1)
        v = b.rows64(b.v, i)
        ref = torch.einsum("hp,phd->hd", p, v)
        size = torch.einsum("hp,phd->hd", p, v.abs())
        tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2.0 ** -12) * size + 2.0 ** -24
        err = (out[i].double() - ref).abs()
        assert bool((err <= tol).all()), (i, c, float((err - tol).max()))
        w = p if w_in is None else p + w_in[i, :, :c].double()
        tol = 2.0 ** -12 * p + 2.0 ** -23 * w + 1e-30
        err = (w_out[i, :, :c].double() - w).abs()
        assert bool((err <= tol).all()), (i, c, float((err / tol).max()))


@pytest.mark.parametrize("D,B", [(64, 8), (64, 32), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("H", [1, 2, 3, 4])
@pytest.mark.parametrize("odd", [0, 3])
def test_weights(D, B, H, odd):
    ctx = [1, 2, B - 1, B, B + 1, 0, 5 * B + 3, 700, 1500]
    b = Batch(D + B + H, ctx, [1] * len(ctx), H, D, B, scale_q=2.0)
    S, W = len(ctx), b.tables.shape[1] * B + odd
    st = _status()
    w_in = torch.rand(S, H, W, device="cuda")
    out, w_out = _run_weights(b, w_in, W, status=st)
    _check_weights(b, out, w_out, w_in, torch.full_like(w_out, -3.0))
    before = w_in.clone()
    same, w_out2 = _run_weights(b, w_in, W, in_place=True, status=st)
    assert torch.equal(out, same)
    _check_weights(b, same, w_out2, before, before)
    out3, w_out3 = _run_weights(b, None, W, status=st)
    _check_weights(b, out3, w_out3, None, torch.full_like(w_out3, -3.0))
    assert st.item() == 0


@pytest.mark.parametrize("H,ctx", [(40, [2048]), (5, [33333, 60, 9000]), (1, [70001])])
def test_weights_of_cut_contexts(H, ctx):
    b = Batch(sum(ctx), ctx, [1] * len(ctx), H, 128, 16, scale_q=3.0)
    W = b.tables.shape[1] * 16
    w_in = torch.rand(len(ctx), H, W, device="cuda")
    out, w_out = _run_weights(b, w_in, W)
    _check_weights(b, out, w_out, w_in, torch.full_like(w_out, -3.0))


def test_weights_agree_with_decode_attention():
    b = Batch(5, [100, 1, 3000, 513], [1] * 4, 4, 128, 16)
    desc = pk.PoolDesc(b.nb, b.B, num_heads=b.H, head_dim=b.D)
    ref = torch.empty(4, b.H, b.D, dtype=torch.float16, device="cuda")
    ws = torch.empty(pk.pa_decode_workspace_bytes(4, b.tables.shape[1], desc), dtype=torch.uint8,
                     device="cuda")
    pk.pa_decode_attention(ref, b.q[:4], b.k, b.v, _dev(b.tables), _i32(b.ctx), b.scale, desc,
                           workspace=ws)
    out, _ = _run_weights(b, None, b.tables.shape[1] * 16)
    assert float((out.float() - ref.float()).abs().max()) <= 4e-3


def test_weights_reports():
    b = Batch(6, [40, 90], [1, 1], 2, 64, 8)
    st = _status()
    out, w_out = _run_weights(b, None, 64, status=st)   # 90 positions, 64 sums
    torch.cuda.synchronize()
    assert st.item() == pk.PA_ERR_INVALID_ARG
    assert bool((out[1] == 7.0).all()) and bool((w_out[1] == -3.0).all())
    b.ctx = [40, 8 * b.tables.shape[1] + 1]
    st = _status()
    out, w_out = _run_weights(b, None, 999, status=st)
    torch.cuda.synchronize()
    assert st.item() == pk.PA_ERR_BAD_BLOCK
    assert bool((out[1] == 7.0).all()) and bool((w_out[1] == -3.0).all())


# ------------------------------------------------------------------ selection


def _select(w, ctx, budget, recent, in_place=False, status=None):
    S, H, _ = w.shape
    keep = torch.full((S, H, budget), 99, dtype=torch.int32, device="cuda")
    lens = torch.full((S,), 99, dtype=torch.int32, device="cuda")
    w_out = w if in_place else torch.full_like(w, -3.0)
    pk.pa_evict_select(keep, lens, w_out, w, _i32(ctx), budget, recent, status=status)
    torch.cuda.synchronize()
    return keep.cpu().numpy(), lens.cpu().numpy(), w_out.cpu().numpy()


def _check_select(w, ctx, budget, recent, got, rest):
    keep, lens, w_out = got
    for s, c in enumerate(ctx):
        c = max(c, 0)
        n = min(c, budget)
        assert lens[s] == n
        for h in range(w.shape[1]):
            if c <= budget:
                want = np.arange(c)
            else:
                x = w[s, h, :c - recent].astype(np.float64)
                x = np.where(np.isnan(x), -np.inf, x)
                nan = np.isnan(w[s, h, :c - recent])
                order = np.lexsort((np.arange(len(x)), nan, -x))[:budget - recent]
                want = np.concatenate([np.sort(order), np.arange(c - recent, c)])
            assert keep[s, h].tolist() == want.tolist() + [-1] * (budget - n), (s, h, c)
            assert np.array_equal(w_out[s, h, :n], w[s, h, want], equal_nan=True)
            assert (w_out[s, h, n:c] == 0).all()
            assert np.array_equal(w_out[s, h, c:], rest[s, h, c:], equal_nan=True)


@pytest.mark.parametrize("W,budget,recent", [(40, 7, 3), (40, 7, 7), (40, 7, 0), (40, 1, 0),
                                             (40, 64, 9), (3000, 512, 64), (9001, 700, 1),
                                             (25000, 4096, 1000), (25000, 1, 1),
                                             (70000, 20000, 333)])
def test_select(W, budget, recent):
    r = np.random.default_rng(W + budget)
    ctx = [W, 0, 1, budget, budget + 1, W - 1, -2]
    ctx = [min(c, W) for c in ctx]
    H = 3
    w = np.exp(2 * r.standard_normal((len(ctx), H, W))).astype(np.float32)
    w[:, 1] = r.integers(0, 3, (len(ctx), W))                  # ties everywhere
    w[0, 2] = r.standard_normal(W)                             # signs, zeros, NaN, infinities
    w[0, 2, r.integers(0, W, max(4, W // 10))] = np.nan
    w[0, 2, r.integers(0, W, 4)] = [np.inf, -np.inf, 0.0, -0.0]
    st = _status()
    got = _select(_dev(w), ctx, budget, recent, status=st)
    _check_select(w, ctx, budget, recent, got, np.full_like(w, -3.0))
    got = _select(_dev(w), ctx, budget, recent, in_place=True, status=st)
    _check_select(w, ctx, budget, recent, got, w)
    assert st.item() == 0


def test_select_reports_a_context_past_the_row():
    w = np.random.default_rng(1).random((2, 2, 50)).astype(np.float32)
    st = _status()
    keep, lens, w_out = _select(_dev(w), [51, 50], 8, 2, status=st)
    assert st.item() == pk.PA_ERR_INVALID_ARG
    assert lens.tolist() == [0, 8] and (keep[0] == -1).all() and (w_out[0] == -3.0).all()
    _check_select(w[1:], [50], 8, 2, (keep[1:], lens[1:], w_out[1:]), np.full((1, 2, 50), -3.0))


# ------------------------------------------------------------------- moves


@pytest.mark.parametrize("D,B", [(8, 4), (16, 16), (32, 8), (64, 32), (128, 16), (256, 8)])
@pytest.mark.parametrize("H,shared", [(1, True), (3, True), (3, False), (10, True), (10, False)])
@pytest.mark.parametrize("apart", [False, True])
def test_compact(D, B, H, shared, apart):
    r = np.random.default_rng(D + B + H)
    L, ctx = 2, [1, B, 3 * B + 1, 700, 50, 0]
    S = len(ctx)
    first = np.array([0, 0, 1, B // 2 + 1, 49, 0])
    blocks = [-(-c // B) for c in ctx]
    NB = 2 * sum(blocks) + 2
    perm = r.permutation(NB)
    src = np.full((S, max(blocks)), -1, np.int32)
    dst = src.copy()
    at = 0
    for i, n in enumerate(blocks):
        src[i, :n] = perm[at:at + n]
        # a destination apart for every other block
        dst[i, :n] = np.where(np.arange(n) % 2 == 0, perm[at + n:at + 2 * n], src[i, :n]) if apart \
            else src[i, :n]
        at += 2 * n
    KH = 1 if shared else H
    room = 400
    lens = np.array([min(room, int(r.integers(0, c - f + 1))) if c > f else 0
                     for c, f in zip(ctx, first)], np.int32)
    lens[2] = min(room, ctx[2] - first[2])       # everything
    lens[3] = room
    keep = np.full((S, KH, room), -1, np.int32)
    for s in range(S):
        for h in range(KH):
            keep[s, h, :lens[s]] = np.sort(r.permutation(ctx[s] - first[s])[:lens[s]])
    caches = [r.standard_normal((NB, H, B, D)).astype(np.float16) for _ in range(2 * L)]
    dev = [_dev(c) for c in caches]
    desc = pk.PoolDesc(NB, B, num_layers=L, num_heads=H, head_dim=D)
    st = _status()
    k_dev = _dev(keep[:, 0]) if shared else _dev(keep)
    pk.pa_compact_kv(dev[:L], dev[L:], _dev(src), _dev(dst), _i32(ctx), k_dev, _dev(lens), desc,
                     first=_i32(first), status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for got, was in zip(dev, caches):
        want = was.copy()
        for s in range(S):
            for h in range(H):
                for j in range(lens[s]):
                    o, n = first[s] + keep[s, h % KH, j], first[s] + j
                    want[dst[s, n // B], h, n % B] = was[src[s, o // B], h, o % B]
        assert np.array_equal(got.cpu().numpy(), want)


def test_compact_reports():
    H, B, D = 2, 8, 64
    desc = pk.PoolDesc(6, B, num_heads=H, head_dim=D)
    was = np.random.default_rng(2).standard_normal((6, H, B, D)).astype(np.float16)
    table = np.array([[4, 1, 3], [0, 2, 5]], np.int32)

    def run(keep, lens, ctx=(20, 20), first=None, src=table, dst=table):
        k, v, st = _dev(was), _dev(was), _status()
        pk.pa_compact_kv([k], [v], _dev(src), _dev(dst), _i32(ctx), _i32(keep), _i32(lens), desc,
                         first=None if first is None else _i32(first), status=st)
        torch.cuda.synchronize()
        assert torch.equal(k, v)
        return st.item(), k.cpu().numpy()

    def moved(rows):
        want = was.copy()
        for s, o, n in rows:
            want[table[s, n // B], :, n % B] = was[table[s, o // B], :, o % B]
        return want

    # not ascending (the same row twice): that row stays
    code, got = run([[3, 3, 9], [0, 5, 6]], [3, 3])
    assert code == pk.PA_ERR_INVALID_ARG
    assert np.array_equal(got, moved([(0, 3, 0), (0, 9, 2), (1, 5, 1), (1, 6, 2)]))
    # outside the sequence
    code, got = run([[3, 20, 21], [-1, 5, 6]], [2, 3])
    assert code == pk.PA_ERR_INVALID_ARG
    assert np.array_equal(got, moved([(0, 3, 0), (1, 5, 1), (1, 6, 2)]))
    # more than the list holds, a negative start: the sequence stays
    for lens, first in (([4, 1], None), ([3, 1], [-1, 0])):
        code, got = run([[3, 4, 9], [1, -1, -1]], lens, first=first)
        assert code == pk.PA_ERR_INVALID_ARG and np.array_equal(got, moved([(1, 1, 0)]))
    # tables outside the pool, a position past the table
    bad = table.copy()
    bad[0, 0] = 6
    for src, dst in ((bad, table), (table, bad)):
        code, got = run([[3, 4, 5], [1, -1, -1]], [3, 1], src=src, dst=dst)
        assert code == pk.PA_ERR_BAD_BLOCK and np.array_equal(got, moved([(1, 1, 0)]))
    code, got = run([[3, 30, 31], [1, -1, -1]], [3, 1], ctx=(40, 20))
    assert code == pk.PA_ERR_BAD_BLOCK and np.array_equal(got, moved([(0, 3, 0), (1, 1, 0)]))


# ------------------------------------------------------------ a whole run


def test_budgeted_decoding_through_the_block_manager():
    """Decode steps of two sequences that share a prompt; one of them is cut to
    its budget twice.  Attention afterwards is that over each head's kept
    rows, the other sequence's rows are untouched, and the sums follow."""
    H, D, B, NB, budget, recent = 3, 64, 8, 60, 20, 5
    r = np.random.default_rng(31)
    g = torch.Generator("cuda").manual_seed(31)
    desc = pk.PoolDesc(NB, B, num_heads=H, head_dim=D, free_order=r.permutation(NB))
    pool = pk.pa_pool_create(desc)
    kc = torch.zeros(NB, H, B, D, dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    rows = torch.randn(2, 37, H, D, generator=g, device="cuda").half()
    pk.pa_write_kv(rows[0].contiguous(), rows[1].contiguous(), _dev(pk.pa_seq_add(pool, 0, 37)), kc,
                   vc, desc)
    pk.pa_seq_fork(pool, 0, 1)
    held = [[[rows[:, p, h] for p in range(37)] for h in range(H)] for _ in range(2)]
    sums = np.zeros((2, H, 256), np.float64)
    W = torch.zeros(2, H, 256, device="cuda")
    st = _status()
    for step in range(12):
        slots, copies = pk.pa_alloc_slots(pool, [0, 1])
        if len(copies):
            pk.pa_copy_blocks([kc], [vc], _dev(copies), desc)
        q, k, v = (torch.randn(2, H, D, generator=g, device="cuda").half() * s for s in (3, 1, 1))
        pk.pa_write_kv(k, v, _dev(slots), kc, vc, desc)
        for s in range(2):
            for h in range(H):
                held[s][h].append(torch.stack([k[s, h], v[s, h]]))
        tables, ctx = pk.pa_get_block_tables(pool, [0, 1], 16)
        out = torch.empty_like(q)
        need = pk.pa_decode_weights_workspace_bytes(2, 16, desc)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        pk.pa_decode_attention_weights(out, W, W, q, kc, vc, _dev(tables), _dev(ctx), 0.125, desc,
                                       workspace=ws, status=st)
        for s in range(2):
            for h in range(H):
                kv = torch.stack(held[s][h]).double()
                assert kv.shape[0] == ctx[s]
                p = torch.softmax(kv[:, 0] @ q[s, h].double() * 0.125, 0)
                assert float((out[s, h].double() - p @ kv[:, 1]).abs().max()) <= 4e-3
                sums[s, h, :ctx[s]] += p.cpu().numpy()
        assert np.allclose(W.cpu().numpy(), sums, rtol=2e-3, atol=1e-6)
        if step in (3, 9):
            # sequence 0 to its budget; 1 still holds the shared prompt
            src, src_lens, dst = pk.pa_seq_compact(pool, [0], [budget], 16)
            keep = torch.empty(1, H, budget, dtype=torch.int32, device="cuda")
            lens = torch.empty(1, dtype=torch.int32, device="cuda")
            pk.pa_evict_select(keep, lens, W[:1], W[:1], _dev(src_lens), budget, recent, status=st)
            pk.pa_compact_kv([kc], [vc], _dev(src), _dev(dst), _dev(src_lens), keep, lens, desc,
                             status=st)
            kept = keep.cpu().numpy()[0]
            assert lens.item() == budget
            w_now = W.cpu().numpy()
            for h in range(H):
                assert (kept[h][-recent:] == np.arange(src_lens[0] - recent, src_lens[0])).all()
                old = np.sort(kept[h][:budget - recent])
                others = np.setdiff1d(np.arange(src_lens[0] - recent), old)
                # what goes is no heavier than what stays, to the sums' rounding
                assert sums[0, h, others].max() <= sums[0, h, old].min() + 1e-5
                held[0][h] = [held[0][h][p] for p in kept[h]]
                sums[0, h, :budget] = sums[0, h, kept[h]]
                sums[0, h, budget:] = 0
                assert np.allclose(w_now[0, h], sums[0, h], rtol=2e-3, atol=1e-6)
    assert st.item() == 0
    pk.pa_pool_destroy(pool)
