"""Drafted tokens on the GPU: pa_tree_attention and pa_verify_draft against
plain evaluations in 64 bits, their reports of bad input, and a whole
speculative step (append, slot write, tree attention, verification, commit,
truncate) through the block manager.

Attention tolerance, per output element (fp16 half step 2^-11 relative):
the output is rounded once (2^-11 |o|), every weight enters the second product
as fp16 (2^-11 sum p |v|), and a score of 128 fp32-accumulated products errs by
at most 128 * 2^-24 * scale * log2 e * sum |q k| (below 2^-13 here, a weight's
relative error; once more in the sum it is divided by).  Verification is in
whole numbers and has to be equal.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_106_gb300 as pk

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _i32(a):
    return _dev(np.asarray(a, np.int32))


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ tree attention


class Batch:
    """Random cache, tables and queries; NaN in every slot that no sequence uses."""

    def __init__(self, seed, ctx, n, H, D, B, spare=3, scale_q=1.0):
        r = np.random.default_rng(seed)
        self.B, self.H, self.D, self.ctx, self.n = B, H, D, list(ctx), list(n)
        blocks = [-(-c // B) for c in ctx]
        self.nb = sum(blocks) + spare
        free = r.permutation(self.nb)
        self.tables = np.full((len(ctx), max(1, max(blocks)) + 1), -1, np.int32)
        k = torch.full((self.nb, H, B, D), float("nan"), dtype=torch.float16, device="cuda")
        v = torch.full_like(k, float("nan"))
        g = torch.Generator("cuda").manual_seed(seed)
        at = 0
        for i, c in enumerate(ctx):
            self.tables[i, :blocks[i]] = free[at:at + blocks[i]]
            at += blocks[i]
            if c:
                pos = torch.arange(c, device="cuda")
                t = _dev(self.tables[i]).long()[pos // B]
                for cache in (k, v):
                    cache[t, :, pos % B] = torch.randn(c, H, D, generator=g, device="cuda").half()
        self.k, self.v = k, v
        self.starts = np.concatenate([[0], np.cumsum(n)])
        self.rows = int(self.starts[-1])
        self.q = (torch.randn(self.rows + 2, H, D, generator=g, device="cuda") * scale_q).half()
        self.scale = float(np.float32(1 / math.sqrt(D)))

    def forest(self, seed, none=0.15):
        r = np.random.default_rng(seed)
        up = np.full(self.rows + 2, -1, np.int32)
        for i, n in enumerate(self.n):
            for t in range(1, n):
                up[self.starts[i] + t] = -1 if r.random() < none else r.integers(0, t)
        return up

    def run(self, parents, max_q=None, status=None, stream=None):
        desc = pk.PoolDesc(self.nb, self.B, num_heads=self.H, head_dim=self.D)
        max_q = max(1, max(self.n)) if max_q is None else max_q
        out = torch.full_like(self.q, 7.0)
        need = pk.pa_tree_workspace_bytes(len(self.ctx), self.tables.shape[1], max_q, desc)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        pk.pa_tree_attention(out, self.q, self.k, self.v, _dev(self.tables), _i32(self.ctx),
                             _i32(self.starts), None if parents is None else _i32(parents),
                             self.scale, desc, max_q_len=max_q, workspace=ws, status=status,
                             stream=stream)
        return out

    def rows64(self, cache, i):
        pos = torch.arange(self.ctx[i], device="cuda")
        return cache[_dev(self.tables[i]).long()[pos // self.B], :, pos % self.B].double()

    def check(self, out, parents, only=None):
        assert bool((out[self.rows:] == 7.0).all())
        for i, c in enumerate(self.ctx):
            n, a = self.n[i], int(self.starts[i])
            if n == 0 or (only is not None and i not in only):
                continue
            sees = torch.zeros(n, c, dtype=torch.bool)
            sees[:, :c - n] = True
            for t in range(n):
                up = t
                while up >= 0:
                    sees[t, c - n + up] = True
                    up = (up - 1) if parents is None else int(parents[a + up])
            x = torch.einsum("thd,phd->htp", self.q[a:a + n].double(), self.rows64(self.k, i))
            x = (x * self.scale).masked_fill(~sees.cuda(), -math.inf)
            w = torch.softmax(x, -1)
            v = self.rows64(self.v, i)
            ref = torch.einsum("htp,phd->thd", w, v)
            size = torch.einsum("htp,phd->thd", w, v.abs())
            tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2.0 ** -12) * size + 2.0 ** -24
            err = (out[a:a + n].double() - ref).abs()
            assert bool((err <= tol).all()), (i, c, n, float((err - tol).max()))


def _ctx_for(n, B):
    """Contexts around what matters for n nodes: nothing before them, a block's
    edges, many blocks."""
    return [n, n + 1, n + B - 1, n + B, 2 * B + n, 5 * B + 3 + n, 40 * B + 1 + n]


@pytest.mark.parametrize("D,B", [(64, 8), (64, 16), (64, 32), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("H", [1, 2, 3, 4])
@pytest.mark.parametrize("n", [1, 2, 16, 17, 33, 64])
def test_tree_attention(D, B, H, n):
    ctx = _ctx_for(n, B)
    ns = [n] * len(ctx)
    ctx += [n + 9, 0, 300]      # fewer nodes, none at all, one
    ns += [max(1, n // 2), 0, 1]
    b = Batch(1000 * D + 10 * B + H + n, ctx, ns, H, D, B, scale_q=2.0)
    st = _status()
    up = b.forest(n)
    out = b.run(up, status=st)
    b.check(out, up)
    b.check(b.run(None, status=st), None)
    assert st.item() == 0


@pytest.mark.parametrize("H,ctx,n", [(40, [2048], [8]), (3, [20011, 9000, 70], [5, 64, 33]),
                                     (8, [4099, 17, 16385, 2], [1, 16, 13, 2]),
                                     (1, [40000], [20])])
@pytest.mark.parametrize("D,B", [(128, 16), (64, 8), (64, 32)])
def test_tree_attention_cut_contexts(H, ctx, n, D, B):
    """Few sequences: contexts cut into parts and joined."""
    b = Batch(sum(ctx) + D, ctx, n, H, D, B, scale_q=3.0)
    up = b.forest(5)
    b.check(b.run(up), up)


def test_tree_attention_large_batches():
    r = np.random.default_rng(3)
    # more sequences than the GPU has slots, one of them long
    ctx = [int(c) for c in r.integers(1, 60, 4096)]
    n = [min(int(k), c) for k, c in zip(r.integers(0, 9, 4096), ctx)]
    ctx[77], n[77] = 30000, 8
    b = Batch(4, ctx, n, 2, 64, 8)
    up = b.forest(6)
    b.check(b.run(up), up, only=set(range(0, 4096, 97)) | {77, 4095})


def test_tree_attention_equals_prefill_of_a_chunk_and_decode():
    b = Batch(9, [700, 65, 33], [33, 64, 33], 5, 128, 16)
    desc = pk.PoolDesc(b.nb, b.B, num_heads=b.H, head_dim=b.D)
    out = b.run(None)
    ref = torch.full_like(b.q, 7.0)
    pk.pa_prefill_attention(ref, b.q, b.k, b.v, _dev(b.tables), _i32(b.ctx), _i32(b.starts),
                            b.scale, desc, max_q_len=64)
    # both are within the fp16 output rounding and the weights' of the same value
    assert float((out.float() - ref.float()).abs().max()) <= 4e-3


def test_tree_attention_does_not_depend_on_where_blocks_are():
    b = Batch(10, [1500, 37, 4000], [12, 30, 7], 4, 128, 16)
    up = b.forest(1)
    out = b.run(up)
    perm = torch.randperm(b.nb, device="cuda")
    k, v = torch.empty_like(b.k), torch.empty_like(b.v)
    k[perm], v[perm] = b.k, b.v
    b.k, b.v = k, v
    b.tables = np.where(b.tables >= 0, perm.cpu().numpy()[b.tables], -1).astype(np.int32)
    assert torch.equal(out, b.run(up))


def test_tree_attention_in_a_graph_and_on_another_stream():
    b = Batch(11, [900, 2100], [9, 40], 4, 128, 16)
    up = b.forest(2)
    want = b.run(up)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.run(up)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    desc = pk.PoolDesc(b.nb, b.B, num_heads=b.H, head_dim=b.D)
    need = pk.pa_tree_workspace_bytes(2, b.tables.shape[1], 40, desc)
    out, ws = torch.zeros_like(b.q), torch.empty(need, dtype=torch.uint8, device="cuda")
    t, c, s, u = _dev(b.tables), _i32(b.ctx), _i32(b.starts), _i32(up)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.pa_tree_attention(out, b.q, b.k, b.v, t, c, s, u, b.scale, desc, max_q_len=40,
                             workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:b.rows], want[:b.rows])


def test_tree_attention_reports():
    # more nodes than positions; a row past the end: reported, left as they were
    b = Batch(12, [5, 50], [4, 6], 2, 64, 8)
    b.ctx[0] = 3
    st = _status()
    out = b.run(None, status=st)
    torch.cuda.synchronize()
    assert st.item() == pk.PA_ERR_INVALID_ARG
    assert bool((out[:4] == 7.0).all())
    b.check(out, None, only={1})
    # more nodes than max_q_len
    b = Batch(12, [5, 50], [4, 6], 2, 64, 8)
    st = _status()
    out = b.run(None, max_q=5, status=st)
    torch.cuda.synchronize()
    assert st.item() == pk.PA_ERR_INVALID_ARG and bool((out[4:10] == 7.0).all())
    b.check(out, None, only={0})
    # a context that the table cannot hold
    b = Batch(12, [5, 50], [4, 6], 2, 64, 8)
    b.ctx[1] = 8 * b.tables.shape[1] + 1
    st = _status()
    out = b.run(None, status=st)
    torch.cuda.synchronize()
    assert st.item() == pk.PA_ERR_BAD_BLOCK and bool((out[4:10] == 7.0).all())
    b.check(out, None, only={0})
    # a table entry outside the pool: reported, the others unaffected
    b = Batch(12, [5, 50], [4, 6], 2, 64, 8)
    b.tables[1, 2] = b.nb
    st = _status()
    out = b.run(None, status=st)
    torch.cuda.synchronize()
    assert st.item() == pk.PA_ERR_BAD_BLOCK
    b.check(out, None, only={0})
    # a parent that is no earlier node counts as none
    b = Batch(12, [5, 50], [4, 6], 2, 64, 8)
    up = b.forest(3, none=0.0)
    up[6] = 2          # node 2 of sequence 1: itself
    st = _status()
    out = b.run(up, status=st)
    torch.cuda.synchronize()
    assert st.item() == pk.PA_ERR_INVALID_ARG
    up[6] = -1
    b.check(out, up)


# -------------------------------------------------------------- verification


def _clean(x):
    x = np.asarray(x, np.float64)
    return np.where((x > 0) & np.isfinite(x), x, 0.0)


def _walk(p, q, tokens, parents, u, us):
    """One sequence, in 64 bits: path, next token (None where nothing can be drawn)."""
    V, n = p.shape[1], len(tokens)
    cur, path, w, z = 0, [0], _clean(p[0]), 1.0
    for i in range(1, n):
        if parents[i] != cur or not 0 <= tokens[i] < V:
            continue
        if q is None:
            row = np.zeros(V)
            row[tokens[i]] = 1
        else:
            row = _clean(q[cur])
        if float(u[i]) * row[tokens[i]] * z < w[tokens[i]]:
            cur, w, z = i, _clean(p[i]), 1.0
            path.append(i)
            continue
        rest = np.maximum(w - row * z, 0)
        if rest.sum() > 0:
            w, z = rest, rest.sum()
    c = np.cumsum(w)
    if not c[-1] > 0:
        return path, -1
    past = np.nonzero(c > float(us) * c[-1])[0]
    return path, int(past[0]) if len(past) else int(np.nonzero(w)[0][-1])


def _verify(p, q, tokens, parents, starts, u, us, max_q=None, status=None):
    S = len(starts) - 1
    mq = max(1, int(np.max(np.diff(starts)))) if max_q is None else max_q
    path = torch.full((S, mq), 99, dtype=torch.int32, device="cuda")
    lens, nxt = (torch.full((S,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    pk.pa_verify_draft(path, lens, nxt, p, q, _i32(tokens),
                       None if parents is None else _i32(parents), _i32(starts),
                       _dev(np.asarray(u, np.float32)), _dev(np.asarray(us, np.float32)),
                       status=status)
    torch.cuda.synchronize()
    return path.cpu().numpy(), lens.cpu().numpy(), nxt.cpu().numpy()


def _expect(p, q, tokens, parents, starts, u, us, got):
    path, lens, nxt = got
    p64 = p.double().cpu().numpy()
    q64 = None if q is None else q.double().cpu().numpy()
    for s in range(len(starts) - 1):
        a, b = int(starts[s]), int(starts[s + 1])
        if a == b:
            assert lens[s] == 0 and nxt[s] == -1 and (path[s] == -1).all()
            continue
        up = np.arange(b - a) - 1 if parents is None else parents[a:b]
        want, token = _walk(p64[a:b], None if q is None else q64[a:b], tokens[a:b], up, u[a:b], us[s])
        assert lens[s] == len(want), (s, lens[s], want)
        assert path[s].tolist() == want + [-1] * (path.shape[1] - len(want))
        assert nxt[s] == token, (s, nxt[s], token)


def _drafts(seed, n, V, dtype, chain=False, onehot=False, close=0.7):
    r = np.random.default_rng(seed)
    g = torch.Generator("cuda").manual_seed(seed)
    starts = np.concatenate([[0], np.cumsum(n)])
    rows = int(starts[-1])
    logits = torch.randn(rows, V, generator=g, device="cuda") * 2
    p = torch.softmax(logits, 1).to(dtype)
    q = torch.softmax(logits + close * torch.randn(rows, V, generator=g, device="cuda"), 1).to(dtype)
    up = np.full(rows, -1, np.int32)
    for i, k in enumerate(n):
        for t in range(1, k):
            up[starts[i] + t] = t - 1 if chain else max(0, t - int(r.integers(1, 4)))
    row = np.repeat(starts[:-1], n) + np.maximum(up, 0)
    src = (p if onehot else q).float()[_dev(row)]
    tokens = torch.multinomial(src, 1, generator=g)[:, 0].int().cpu().numpy()
    return p, None if onehot else q, tokens, up, starts, \
        r.random(rows).astype(np.float32), r.random(len(n)).astype(np.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 3, 32, 33, 1000, 2049, 4100, 20001])
@pytest.mark.parametrize("onehot", [False, True])
def test_verify_trees(dtype, V, onehot):
    r = np.random.default_rng(V)
    n = [1, 2, 64, 0, 5] + [int(k) for k in r.integers(1, 30, 20)]
    d = _drafts(V + 7, n, V, dtype, onehot=onehot)
    st = _status()
    _expect(*d, _verify(*d, status=st))
    assert st.item() == 0


@pytest.mark.parametrize("V", [50272, 131072])
def test_verify_chains_of_a_batch(V):
    n = [int(k) for k in np.random.default_rng(1).integers(1, 9, 24)]
    p, q, tokens, up, starts, u, us = _drafts(3, n, V, torch.float32, chain=True)
    got = _verify(p, q, tokens, None, starts, u, us)
    _expect(p, q, tokens, None, starts, u, us, got)
    again = _verify(p, q, tokens, up, starts, u, us)
    assert all(np.array_equal(x, y) for x, y in zip(got, again))


def test_verify_edges():
    V = 70
    n = [2, 3, 4, 4, 2, 2, 3]
    p, q, tokens, up, starts, u, us = _drafts(5, n, V, torch.float32)
    rows = {s: int(starts[s]) for s in range(7)}
    for s in range(7):
        up[rows[s] + 1:rows[s] + n[s]] = 0        # all drafted after the root
    # 0: the drafter is the target: a rejection leaves nothing, w stays
    q[rows[0]] = p[rows[0]]
    u[rows[0] + 1] = 1.0
    # 1: the same token twice; its second trial meets weight 0 or what is left
    tokens[rows[1] + 2] = tokens[rows[1] + 1]
    u[rows[1] + 1:rows[1] + 3] = 1.0 - 2.0 ** -24
    # 2: NaN, infinities and negative entries count as 0
    p[rows[2], :5] = torch.tensor([math.nan, math.inf, -math.inf, -1.0, 0.0], device="cuda")
    q[rows[2], 2:6] = torch.tensor([math.nan, math.inf, -2.0, 0.0], device="cuda")
    # 3: the numbers' ends
    u[rows[3] + 1:rows[3] + 4] = [0.0, 1.0 - 2.0 ** -24, 0.5]
    us[3] = 0.0
    us[2] = 1.0 - 2.0 ** -24
    # 4: a certain target
    p[rows[4]] = 0
    p[rows[4], 31] = 1
    # 5: what the drafter never draws is always accepted where the target has it
    q[rows[5], int(tokens[rows[5] + 1])] = 0
    u[rows[5] + 1] = 1.0 - 2.0 ** -24
    # 6: tiny weights: 2^-140 is below fp32's normal range
    p[rows[6]] *= 2.0 ** -130
    d = (p, q, tokens, up, starts, u, us)
    st = _status()
    _expect(*d, _verify(*d, status=st))
    assert st.item() == 0


def test_verify_reports():
    n = [3, 4, 2, 3]
    p, q, tokens, up, starts, u, us = _drafts(6, n, 40, torch.float32)
    up[1:3] = 0
    u[:] = 0.0           # everything reached is accepted
    # a parent that is no earlier node, a token outside: not reached
    st = _status()
    bad = up.copy()
    bad[2] = 2
    got = _verify(p, q, tokens, bad, starts, u, us, status=st)
    assert st.item() == pk.PA_ERR_INVALID_ARG
    bad[2] = -1
    _expect(p, q, tokens, bad, starts, u, us, got)
    for token in (-1, 40):
        t = tokens.copy()
        t[4] = token
        st = _status()
        got = _verify(p, q, t, up, starts, u, us, status=st)
        assert st.item() == pk.PA_ERR_INVALID_ARG
        _expect(p, q, t, up, starts, u, us, got)
    # a row without weight
    z = p.clone()
    z[7:9] = 0
    st = _status()
    path, lens, nxt = _verify(z, q, tokens, up, starts, u, us, status=st)
    assert st.item() == pk.PA_ERR_INVALID_ARG and nxt[2] == -1 and lens[2] == 1
    # rows past the end, more nodes than max_q_len
    for s2, mq in ((np.array([0, 3, 7, 9, 13]), 4), (starts, 3)):
        st = _status()
        path, lens, nxt = _verify(p, q, tokens, up, s2, u, us, max_q=mq, status=st)
        i = 3 if mq == 4 else 1
        assert st.item() == pk.PA_ERR_INVALID_ARG
        assert lens[i] == 0 and nxt[i] == -1 and (path[i] == -1).all()
        assert lens[0] > 0


def test_verified_tokens_are_distributed_as_the_target():
    """Two siblings from one drafter row: the token decided after the root has
    the target's distribution.  20000 draws, 12 tokens: every frequency within
    5 standard deviations."""
    S, V = 20000, 12
    r = np.random.default_rng(8)
    p1, q1 = r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V))
    starts = np.arange(S + 1) * 3
    p, q = (torch.from_numpy(np.tile(x, (3 * S, 1))).float().cuda() for x in (p1, q1))
    tokens = r.choice(V, 3 * S, p=q1).astype(np.int32)
    up = np.tile(np.array([-1, 0, 0], np.int32), S)
    path, lens, nxt = _verify(p, q, tokens, up, starts, r.random(3 * S), r.random(S))
    first = np.where(lens > 1, tokens[starts[:-1] + path[:, 1]], nxt)
    f = np.bincount(first, minlength=V) / S
    assert (np.abs(f - p1) <= 5 * np.sqrt(p1 * (1 - p1) / S)).all()


# ------------------------------------------------------------ a whole step


def test_speculative_steps_through_the_block_manager():
    """Three steps for three sequences, one of them forked: after each commit
    the caches hold, at every kept position, the K/V that the accepted nodes
    had, and shared blocks of the parent are as they were."""
    H, D, B, L, NB, V = 3, 64, 8, 2, 64, 50
    r = np.random.default_rng(21)
    g = torch.Generator("cuda").manual_seed(21)
    desc = pk.PoolDesc(NB, B, num_layers=L, num_heads=H, head_dim=D,
                       free_order=r.permutation(NB))
    pool = pk.pa_pool_create(desc)
    kc = [torch.zeros(NB, H, B, D, dtype=torch.float16, device="cuda") for _ in range(L)]
    vc = [torch.zeros_like(kc[0]) for _ in range(L)]
    ids = [0, 1, 2]
    held = {i: [] for i in ids}          # per sequence: rows [2 L, H, D] of its positions

    def write(slots, rows):
        for layer in range(L):
            pk.pa_write_kv(rows[:, 2 * layer].contiguous(), rows[:, 2 * layer + 1].contiguous(),
                           _dev(slots), kc[layer], vc[layer], desc)

    def fresh(n):
        return torch.randn(n, 2 * L, H, D, generator=g, device="cuda").half()

    for i, n in ((0, 13), (1, 30)):
        rows = fresh(n)
        write(pk.pa_seq_add(pool, i, n), rows)
        held[i] = list(rows)
    pk.pa_seq_fork(pool, 1, 2)
    held[2] = list(held[1])
    for step in range(3):
        n = [int(k) for k in r.integers(1, 12, 3)]
        starts = np.concatenate([[0], np.cumsum(n)])
        rows = int(starts[-1])
        slots, copies = pk.pa_alloc_slots_n(pool, ids, n)
        if len(copies):
            pk.pa_copy_blocks(kc, vc, _dev(copies), desc)
        new = fresh(rows)
        write(slots, new)
        tables, ctx = pk.pa_get_block_tables(pool, ids, 16)
        up = np.concatenate([[max(0, t - int(r.integers(1, 3))) - (t == 0) for t in range(k)]
                             for k in n]).astype(np.int32)
        q = torch.randn(rows, H, D, generator=g, device="cuda").half()
        out = torch.empty_like(q)
        need = pk.pa_tree_workspace_bytes(3, 16, max(n), desc)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        st = _status()
        d_tables, d_ctx, d_starts, d_up = _dev(tables), _dev(ctx), _i32(starts), _i32(up)
        for layer in range(L):
            pk.pa_tree_attention(out, q, kc[layer], vc[layer], d_tables, d_ctx, d_starts, d_up,
                                 0.125, desc, max_q_len=max(n), workspace=ws, status=st)
        for i in ids:         # the last layer's output
            a, b = int(starts[i]), int(starts[i + 1])
            rows_kv = torch.stack(held[i] + list(new[a:b])).double()
            base = len(held[i])
            sees = torch.zeros(b - a, base + b - a, dtype=torch.bool)
            sees[:, :base] = True
            for t in range(b - a):
                x = t
                while x >= 0:
                    sees[t, base + x] = True
                    x = int(up[a + x])
            s = torch.einsum("thd,phd->htp", q[a:b].double(), rows_kv[:, 2 * L - 2]) * 0.125
            w = torch.softmax(s.masked_fill(~sees.cuda(), -math.inf), -1)
            ref = torch.einsum("htp,phd->thd", w, rows_kv[:, 2 * L - 1])
            assert float((out[a:b].double() - ref).abs().max()) <= 4e-3
        p, qd, tokens, _, _, u, us = _drafts(30 + step, n, V, torch.float32)
        path = torch.empty(3, max(n), dtype=torch.int32, device="cuda")
        lens, nxt = (torch.empty(3, dtype=torch.int32, device="cuda") for _ in range(2))
        pk.pa_verify_draft(path, lens, nxt, p, qd, _i32(tokens), d_up, d_starts,
                           _dev(u), _dev(us), status=st)
        first = d_ctx - _i32(n)
        pk.pa_compact_kv(kc, vc, d_tables, d_tables, d_ctx, path, lens, desc, first=first,
                         status=st)
        path_h, lens_h = path.cpu().numpy(), lens.cpu().numpy()
        assert st.item() == 0
        for i in ids:
            held[i] += [new[int(starts[i]) + int(t)] for t in path_h[i, :lens_h[i]]]
        pk.pa_seq_truncate(pool, ids, [len(held[i]) for i in ids])
        tables, ctx = pk.pa_get_block_tables(pool, ids, 16)
        for i in ids:
            assert ctx[i] == len(held[i])
            want = torch.stack(held[i])
            pos = np.arange(ctx[i])
            t, off = _dev(tables[i][pos // B]).long(), _dev(pos % B)
            for layer in range(L):
                assert torch.equal(kc[layer][t, :, off], want[:, 2 * layer])
                assert torch.equal(vc[layer][t, :, off], want[:, 2 * layer + 1])
    pk.pa_pool_destroy(pool)
