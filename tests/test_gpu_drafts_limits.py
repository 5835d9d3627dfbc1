"""Drafted tokens and the bounded cache where calls go wrong most easily: values
that are not finite in nodes a row does not see, calls captured in one graph
that share a workspace, two streams at once, unaligned probabilities, caches
and rows past 32-bit offsets, long row lists, and lists that do not ascend.
Tolerances are those of the two files whose checks are used here; results that
are the same arithmetic have to be equal.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_106_gb300 as pk
from tests.test_gpu_bounded_cache import _check_select, _check_weights, _run_weights, _select
from tests.test_gpu_drafts import Batch, _dev, _drafts, _expect, _i32, _status, _verify

pytestmark = pytest.mark.gpu


def _sees(parents, t):
    """Node t and its ancestors."""
    seen = set()
    while t >= 0:
        seen.add(t)
        t = t - 1 if parents is None else int(parents[t])
    return seen


# ------------------------------------------------- values that are not finite


def _plant_and_check(b, up, seed, sequences):
    """Puts infinities and NaN into the keys or values of some nodes of some
    sequences: rows that see them have them in their output, the others stay
    within the tolerance of the evaluation without, and equal it in the
    dimensions without such values."""
    clean = b.run(up).float()
    r = np.random.default_rng(seed)
    odd = [math.inf, -math.inf, math.nan]
    want, k, v = clean.clone(), b.k.clone(), b.v.clone()
    hit = torch.zeros_like(want, dtype=torch.bool)
    for i in sequences:
        a, c, n = int(b.starts[i]), b.ctx[i], b.n[i]
        links = None if up is None else up[a:a + n]
        for e in range(4):
            # never the root: some row is left that does not see the node
            t, h, dim, x = int(r.integers(1, n)), int(r.integers(b.H)), int(r.integers(b.D)), odd[e % 3]
            pos = c - n + t
            at = (int(b.tables[i, pos // b.B]), h, pos % b.B, dim)
            if e < 3:
                b.v[at] = x
                hit[a:a + n, h, dim] = True
            else:
                b.k[at] = math.nan
            for row in range(n):
                if t not in _sees(links, row):
                    continue
                if e < 3:
                    want[a + row, h, dim] += x
                else:
                    want[a + row, h] = math.nan
    got = b.run(up).float()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    fine = torch.isfinite(want)
    assert torch.equal(got[fine & ~hit], clean[fine & ~hit])
    b.k, b.v = k, v
    b.check(torch.where(fine, got, clean).half(), up)
    assert bool(torch.isfinite(got[b.starts[:-1]]).all())     # the roots


@pytest.mark.parametrize("D,B", [(64, 8), (64, 32), (128, 16)])
@pytest.mark.parametrize("n", [2, 13, 32, 64])
@pytest.mark.parametrize("chain", [False, True])
def test_tree_attention_unseen_values_that_are_not_finite(D, B, n, chain):
    """Contexts put the nodes in one tile of 128 positions, across two, and
    behind a context in many parts."""
    ctx = [n, 100 + n, 128 + n // 2, 256, 9000 + n]
    b = Batch(D + n, ctx, [n] * len(ctx), 3, D, B, scale_q=2.0)
    _plant_and_check(b, None if chain else b.forest(n), n, range(len(ctx)))


def _mixed(seed, S, most_n, most_ctx):
    r = np.random.default_rng(seed)
    ctx = [int(c) for c in np.exp(r.uniform(0, math.log(most_ctx), S))]
    return ctx, [int(r.integers(1, min(most_n, c) + 1)) for c in ctx]


@pytest.mark.parametrize("D,B", [(64, 8), (64, 32), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("most_ctx", [60, 300, 2000])
def test_many_units_of_few_rows(D, B, most_ctx):
    """Batches that give every CTA several units of up to 16 rows, of one tile
    and of several, and the same contexts with weights."""
    ctx, n = _mixed(D + most_ctx, 61, 16, most_ctx)
    b = Batch(D + B, ctx, n, 10, D, B, scale_q=2.0)
    up = b.forest(2)
    b.check(b.run(up), up)
    b.check(b.run(None), None)
    one = Batch(D + B, ctx, [1] * 61, 10, D, B, scale_q=2.0)
    W = one.tables.shape[1] * B
    w_in = torch.rand(61, 10, W, device="cuda")
    st = _status()
    out, w_out = _run_weights(one, w_in, W, status=st)
    _check_weights(one, out, w_out, w_in, torch.full_like(w_out, -3.0))
    assert st.item() == 0


@pytest.mark.parametrize("D,B", [(64, 16), (128, 16)])
@pytest.mark.parametrize("n", [1, 9, 16, 31, 64])
@pytest.mark.parametrize("S", [2, 40])
def test_scores_that_grow_along_the_context(D, B, n, S):
    """Keys that raise a row's largest score by 12 in log2 units from tile to
    tile, another row's in each, so what is summed so far is rescaled.  A score
    of D products, fp32-accumulated, errs by at most e = D 2^-24 times the sum
    of their sizes; a weight by that, and once more in the sum it is divided by.
    2^(x - reference) enters the second product as fp16, which below 2^-14 has
    steps of 2^-24: half of one, 2^-25, is its error there, and the sum it is
    divided by is 1 or more, since a reference is the score of some position
    seen (that one's term is 1 and a larger score's more).  A weight of 2^-14 or
    more has a term of 2^-14 or more, so the rest add 2^-25 |v| each."""
    H = 8
    ctx = [600 + 17 * s for s in range(S)]
    b = Batch(n + D, ctx, [n] * S, H, D, B)
    up = b.forest(n)
    scale2 = b.scale / math.log(2)
    for s, c in enumerate(ctx):
        a = int(b.starts[s])
        for j, pos in enumerate((20, 140, 290, 420, 550)):
            row = b.q[a + (3 * j) % n].float()                     # [H][D]
            key = row * (12.0 * (j + 1) / (scale2 * (row * row).sum(-1, keepdim=True)))
            b.k[int(b.tables[s, pos // B]), :, pos % B] = key.half()
    out = b.run(up)
    one = None
    if n == 1:
        one = _run_weights(b, None, b.tables.shape[1] * B)
    for s, c in enumerate(ctx):
        a = int(b.starts[s])
        sees = torch.zeros(n, c, dtype=torch.bool)
        sees[:, :c - n] = True
        for t in range(n):
            sees[t, [c - n + x for x in _sees(up[a:a + n], t)]] = True
        q, k, v = b.q[a:a + n].double(), b.rows64(b.k, s), b.rows64(b.v, s)
        x = torch.einsum("thd,phd->htp", q, k) * b.scale
        w = torch.softmax(x.masked_fill(~sees.cuda(), -math.inf), -1)
        e = D * 2.0 ** -24 * float(torch.einsum("thd,phd->htp", q.abs(), k.abs()).max()) * b.scale
        ref = torch.einsum("htp,phd->thd", w, v)
        size = torch.einsum("htp,phd->thd", w, v.abs())
        small = (sees.cuda() & (w < 2.0 ** -14)).double()
        steps = 2.0 ** -25 * torch.einsum("htp,phd->thd", small, v.abs())
        tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2 * e) * size + steps + 2.0 ** -24
        err = (out[a:a + n].double() - ref).abs()
        assert bool((err <= tol).all()), (s, float((err - tol).max()))
        if one is not None:
            got = one[1][s, :, :c].double()
            assert bool(((got - w[:, 0]).abs() <= (2 * e + 2.0 ** -23) * w[:, 0] + 1e-30).all())


@pytest.mark.parametrize("D,B", [(64, 8), (128, 16)])
def test_many_units_with_values_that_are_not_finite(D, B):
    ctx, n = _mixed(D, 61, 16, 700)
    n = [max(2, k) for k in n]
    ctx = [max(c, k) for c, k in zip(ctx, n)]
    b = Batch(D + 1, ctx, n, 10, D, B, scale_q=2.0)
    _plant_and_check(b, b.forest(4), 4, range(0, 61, 3))


def test_tree_attention_rows_with_infinite_scores_leave_the_others():
    b = Batch(3, [300, 40], [20, 5], 2, 128, 16)
    up = b.forest(3)
    clean = b.run(up)
    b.q[7, 1, 5] = math.inf
    b.q[22, 0, 5] = math.nan
    got = b.run(up)
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[7, 1] = keep[22, 0] = False
    assert torch.equal(got[keep], clean[keep])
    assert bool(torch.isnan(got[22, 0]).all()) and bool(torch.isnan(got[7, 1]).all())


# ------------------------------------------------------- graphs and streams


def test_one_graph_of_all_calls_sharing_a_workspace():
    """Two tree attentions and two weighted decodes on one workspace, then
    verification, selection and moves, captured once and replayed over other
    contents of the same buffers."""
    H, D, B = 4, 128, 16
    one = Batch(31, [5000, 70, 900], [40, 9, 64], H, D, B)
    two = Batch(32, [300, 4100, 64], [3, 16, 64], H, D, B)
    ups = [one.forest(1), two.forest(2)]
    desc = [pk.PoolDesc(b.nb, B, num_heads=H, head_dim=D) for b in (one, two)]
    need = max(max(pk.pa_tree_workspace_bytes(3, b.tables.shape[1], 64, d),
                   pk.pa_decode_weights_workspace_bytes(3, b.tables.shape[1], d))
               for b, d in zip((one, two), desc))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    W = max(one.tables.shape[1], two.tables.shape[1]) * B
    dev = [(_dev(b.tables), _i32(b.ctx), _i32(b.starts), _i32(u)) for b, u in zip((one, two), ups)]
    outs = [torch.zeros_like(b.q) for b in (one, two)]
    dec = [torch.zeros(3, H, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    sums = [torch.zeros(3, H, W, device="cuda") for _ in range(2)]
    p, qd, tokens, up, starts, u, us = _drafts(9, [5, 3, 8], 5001, torch.float32)
    path = torch.empty(3, 8, dtype=torch.int32, device="cuda")
    lens, nxt = (torch.empty(3, dtype=torch.int32, device="cuda") for _ in range(2))
    d_ver = (_i32(tokens), _i32(up), _i32(starts), _dev(u), _dev(us))
    keep = torch.empty(3, H, 50, dtype=torch.int32, device="cuda")
    kept = torch.empty(3, dtype=torch.int32, device="cuda")
    st = _status()

    def calls():
        for b, d, (t, c, s, x), o, m, w in zip((one, two), desc, dev, outs, dec, sums):
            pk.pa_tree_attention(o, b.q, b.k, b.v, t, c, s, x, b.scale, d, max_q_len=64,
                                 workspace=ws, status=st)
            pk.pa_decode_attention_weights(m, w, w, b.q[:3], b.k, b.v, t, c, b.scale, d,
                                           workspace=ws, status=st)
        pk.pa_verify_draft(path, lens, nxt, p, qd, *d_ver, status=st)
        pk.pa_evict_select(keep, kept, sums[0], sums[0], dev[0][1], 50, 7, status=st)
        pk.pa_compact_kv([one.k], [one.v], dev[0][0], dev[0][0], dev[0][1], keep, kept, desc[0],
                         status=st)

    state = [one.k, one.v, two.k, two.v, one.q, two.q, *sums]
    results = state + outs + dec + [path, lens, nxt, keep, kept]

    def contents(seed):
        g = torch.Generator("cuda").manual_seed(seed)
        for x in state:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda").abs().to(x.dtype) if x.dtype == torch.float32
                    else torch.randn(x.shape, generator=g, device="cuda").half())
        logits = torch.randn(p.shape, generator=g, device="cuda")
        p.copy_(torch.softmax(logits, 1))

    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):       # loads what is loaded at the first call
        calls()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        calls()
    for seed in range(3):
        contents(seed)
        calls()
        want = [x.clone() for x in results]
        contents(seed)
        for x in results[len(state):]:
            x.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(results, want):
            if x is outs[0] or x is outs[1]:
                rows = one.rows if x is outs[0] else two.rows
                assert torch.equal(x[:rows], y[:rows])
            else:
                assert torch.equal(x, y)
    assert st.item() == 0


def test_two_streams_at_once():
    a = Batch(41, [700, 3000, 64], [12, 40, 64], 6, 128, 16)
    b = Batch(42, [2000, 33], [1, 1], 6, 128, 16)
    up = a.forest(1)
    W = b.tables.shape[1] * 16
    d = _drafts(43, [6] * 40, 9000, torch.float16)
    want = a.run(up), *_run_weights(b, None, W), _verify(*d)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            x = a.run(up)
        with torch.cuda.stream(s2):
            y, w = _run_weights(b, None, W)
            v = _verify(*d)              # (waits for both)
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])
        for i, c in enumerate(b.ctx):
            assert torch.equal(w[i, :, :c], want[2][i, :, :c])
        assert all(np.array_equal(e, f) for e, f in zip(v, want[3]))


# --------------------------------------------------------------- verification


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V,off", [(1000, 1), (4100, 2), (4099, 3), (20001, 5)])
def test_verify_probabilities_at_any_address(dtype, V, off):
    n = [3, 1, 17, 8]
    p, q, tokens, up, starts, u, us = _drafts(V + off, n, V, dtype)

    def moved(x, by):
        flat = torch.empty(x.numel() + 16, dtype=dtype, device="cuda")
        y = flat[by:by + x.numel()].view(x.shape)
        y.copy_(x)
        return y

    d = (moved(p, off), moved(q, 0), tokens, up, starts, u, us)
    _expect(*d, _verify(*d))


@pytest.mark.parametrize("S,V,dtype", [(700, 5003, torch.float32), (320, 9001, torch.float16),
                                       (3, 600_001, torch.float32), (1, 1_000_000, torch.bfloat16)])
def test_verify_batches_and_vocabularies(S, V, dtype):
    """Many sequences (a CTA each), and rows of several loads a segment."""
    n = [int(k) for k in np.random.default_rng(S).integers(1, 4, S)]
    d = _drafts(S + V, n, V, dtype)
    _expect(*d, _verify(*d))


def test_verify_rows_past_32_bits():
    V, rows, first = 131072, 16400, 16388          # rows from 2^31 elements on
    n = [3, 5, 4]
    p, q, tokens, up, starts, u, us = _drafts(1, n, V, torch.float16)
    big_p, big_q = (torch.empty(rows, V, dtype=torch.float16, device="cuda") for _ in range(2))
    big_p[first:], big_q[first:] = p, q
    want = _verify(p, q, tokens, up, starts, u, us)
    pad = np.zeros(first)
    got = _verify(big_p, big_q, np.concatenate([pad, tokens]), np.concatenate([pad, up]),
                  starts + first, np.concatenate([pad, u]), us, max_q=5)
    assert all(np.array_equal(x, y) for x, y in zip(got, want))


# ----------------------------------------------------------- 32-bit offsets


def test_caches_past_32_bits():
    """The same blocks at the end of a cache of more than 2^32 elements."""
    H, D, B = 8, 128, 32
    b = Batch(51, [900, 64, 5000], [1, 30, 64], H, D, B)
    up = b.forest(1)
    W = b.tables.shape[1] * B
    one = Batch(51, [900, 64, 5000], [1, 1, 1], H, D, B)
    want, (dec, sums) = b.run(up), _run_weights(one, None, W)
    far = 2 ** 32 // (H * D * B)
    small = [b.k, b.v, one.k, one.v]
    assert torch.equal(b.k.nan_to_num(), one.k.nan_to_num()) and b.nb == one.nb
    k, v = (torch.empty(far + b.nb, H, B, D, dtype=torch.float16, device="cuda") for _ in range(2))
    k[far:], v[far:] = b.k, b.v
    for x in (b, one):
        x.k, x.v = k, v
        x.tables = np.where(x.tables >= 0, x.tables + far, -1).astype(np.int32)
        x.nb += far
    assert torch.equal(b.run(up), want)
    again, w = _run_weights(one, None, W)
    assert torch.equal(again, dec)
    for i, c in enumerate(one.ctx):
        assert torch.equal(w[i, :, :c], sums[i, :, :c])
    # moves, by one list and by one a head, against the same in the small cache
    keep = np.full((3, H, 40), -1, np.int32)
    lens = np.array([40, 33, 40], np.int32)
    r = np.random.default_rng(5)
    for s in range(3):
        for h in range(H):
            keep[s, h, :lens[s]] = np.sort(r.permutation(one.ctx[s])[:lens[s]])
    for lists in (keep[:, 0], keep):
        for caches, tables, nb in ((small[:2], one.tables - far * (one.tables >= 0), one.nb - far),
                                   ([k, v], one.tables, one.nb)):
            desc = pk.PoolDesc(nb, B, num_heads=H, head_dim=D)
            t = _i32(tables)
            pk.pa_compact_kv(caches[:1], caches[1:], t, t, _i32(one.ctx), _dev(lists), _dev(lens), desc)
        for x, y in ((k, small[0]), (v, small[1])):
            assert torch.equal(x[far:].nan_to_num(), y.nan_to_num())


def test_sums_past_32_bits():
    """Rows of accumulated weights that begin past 2^31 elements."""
    W, H = 2 ** 30 + 4, 3
    w = torch.empty(1, H, W, device="cuda")
    b = Batch(61, [500], [1], H, 64, 16)
    start = torch.rand(1, H, 500, device="cuda")
    w[:, :, :500] = start
    w[:, :, 500:600] = -3.0
    out, w_out = _run_weights(b, w, W, in_place=True)
    _check_weights(b, out, w_out[:, :, :600], start, torch.full((1, H, 600), -3.0, device="cuda"))
    now = w[:, :, :600].cpu().numpy()
    keep = torch.full((1, H, 100), 99, dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.pa_evict_select(keep, lens, w, w, _i32([500]), 100, 10)
    _check_select(now, [500], 100, 10,
                  (keep.cpu().numpy(), lens.cpu().numpy(), w[:, :, :600].cpu().numpy()), now)


# --------------------------------------------------------------------- moves


@pytest.mark.parametrize("L,H,D,S", [(1, 40, 128, 2), (24, 3, 64, 40), (128, 5, 8, 17),
                                     (7, 1, 256, 200)])
@pytest.mark.parametrize("room", [1, 5, 64, 65])
def test_short_lists_for_all_heads(L, H, D, S, room):
    """Accepted drafts: a short list of each sequence, keys and values of all
    layers, in place."""
    B, n = 8, 70
    r = np.random.default_rng(L + room)
    ctx = r.integers(n, 200, S).astype(np.int32)
    first = (ctx - n).astype(np.int32)
    blocks = -(-ctx // B)
    NB = int(blocks.sum())
    tables = np.full((S, int(blocks.max())), -1, np.int32)
    perm, at = r.permutation(NB), 0
    for s in range(S):
        tables[s, :blocks[s]] = perm[at:at + blocks[s]]
        at += blocks[s]
    lens = r.integers(0, room + 1, S).astype(np.int32)
    keep = np.full((S, room), -1, np.int32)
    for s in range(S):
        keep[s, :lens[s]] = np.sort(r.permutation(n)[:lens[s]])
    caches = [torch.randn(NB, H, B, D, device="cuda").half() for _ in range(2 * L)]
    was = [c.clone() for c in caches]
    desc = pk.PoolDesc(NB, B, num_layers=L, num_heads=H, head_dim=D)
    st = _status()
    t = _dev(tables)
    pk.pa_compact_kv(caches[:L], caches[L:], t, t, _dev(ctx), _dev(keep), _dev(lens), desc,
                     first=_dev(first), status=st)
    rows = [(s, first[s] + keep[s, j], first[s] + j) for s in range(S) for j in range(lens[s])]
    s, o, d = (np.array(x, np.int64) for x in zip(*rows)) if rows else (np.zeros(0, np.int64),) * 3
    src, dst = _dev(tables[s, o // B]).long(), _dev(tables[s, d // B]).long()
    for got, x in zip(caches, was):
        want = x.clone()
        want[dst, :, _dev(d % B)] = x[src, :, _dev(o % B)]
        assert torch.equal(got, want)
    assert st.item() == 0


@pytest.mark.parametrize("heads", [1, 2])
def test_moves_never_go_up(heads):
    """After an entry out of order later ones can lie below their own index:
    they are reported, and nothing past the table is looked up."""
    H, B, D, room = 2, 8, 64, 24
    desc = pk.PoolDesc(7, B, num_heads=H, head_dim=D)
    was = torch.randn(7, H, B, D, device="cuda").half()
    table = np.array([[4, 1, 3], [0, 2, 5]], np.int32)
    keep = np.stack([np.arange(room) - 1, np.arange(room)]).astype(np.int32)   # -1, 0, 1, ...
    keep[0, 9] = 11
    lists = keep if heads == 1 else np.repeat(keep[:, None], H, 1)
    k, v, st = was.clone(), was.clone(), _status()
    t = _dev(table)
    pk.pa_compact_kv([k], [v], t, t, _i32([24, 24]), _dev(np.ascontiguousarray(lists)),
                     _i32([room, room]), desc, status=st)
    want = was.clone()
    want[table[0, 1], :, 1] = was[table[0, 1], :, 3]      # entry 9 alone
    assert torch.equal(k, want) and torch.equal(v, want)
    assert st.item() == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("W,budget,recent", [(4096, 1000, 100), (4097, 1000, 100), (26624, 5000, 1),
                                             (26625, 5000, 1)])
def test_select_at_the_edges_of_its_forms(W, budget, recent):
    r = np.random.default_rng(W)
    w = np.exp(2 * r.standard_normal((2, 3, W))).astype(np.float32)
    w[0, 1, :] = 1.0                                       # all equal
    w[1, 1, : W // 2] = 2.5                                # more equal ones than are ranked
    for in_place in (False, True):
        got = _select(_dev(w), [W, W - 1], budget, recent, in_place=in_place)
        _check_select(w, [W, W - 1], budget, recent, got, w if in_place else np.full_like(w, -3.0))
