"""Drafted tokens and the bounded cache where rounding decides: one position
that takes almost all of a row's weight, rows beside rows whose scores jump,
and random numbers that fall on the border between two tokens.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_106_gb300 as pk
from tests.test_gpu_drafts import Batch, _dev, _i32, _status, _verify

pytestmark = pytest.mark.gpu


# --------------------------------------------------- one dominant position


def _dominated(D, n, ctx, gaps, seed):
    """One sequence whose first key lies `gaps[row]` binary orders above all
    others in every row and whose first value is 0.  All blocks but the first
    are one and the same, so a long context costs no memory; enough heads that
    no context is cut into parts (a part without the first position has no such
    gap)."""
    B, H = 16, 4 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator("cuda").manual_seed(seed)
    k = torch.zeros(2, H, B, D, dtype=torch.float16, device="cuda")
    v = (torch.rand(2, H, B, D, generator=g, device="cuda") + 0.5).half()
    k[0, :, 0, 0] = 8.0
    v[0, :, 0] = 0
    scale = float(np.float32(1 / math.sqrt(D)))
    q = torch.zeros(n, H, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = torch.tensor(gaps, device="cuda")[:, None] * math.log(2) / (8.0 * scale)
    table = np.ones((1, ctx // B), np.int32)
    table[0, 0] = 0
    return k, v, q, scale, _dev(table), pk.PoolDesc(2, B, num_heads=H, head_dim=D)


def _check_dominated(out, k, v, q, scale, n, ctx, heads=(0, 1, 100)):
    """Against 64 bits.  The output is rounded once (2^-11), and every weight
    enters the product as an fp16 number (2^-11 of it).  A row's terms are taken
    relative to a reference that lies 7 to 15 binary orders below its largest
    score, so a weight of 2^-21 of the largest one or more is a normal fp16
    number; below, its error is half a step of 2^-24 where the largest term is
    2^7 or more: 2^-32 of the largest weight, which is 1 at most."""
    at = torch.arange(ctx, device="cuda")
    for h in heads:
        block = (at >= 16).long()
        kk, vv = k[block, h, at % 16].double(), v[block, h, at % 16].double()
        x = q[:, h].double() @ kk.T * scale
        x.masked_fill_(at[None] > ctx - n + torch.arange(n, device="cuda")[:, None], -math.inf)
        w = torch.softmax(x, -1)
        ref, size = w @ vv, w @ vv.abs()
        small = (w > 0) & (w < 2.0 ** -21 * w.amax(-1, keepdim=True))
        tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2.0 ** -12) * size + 2.0 ** -24 \
            + 2.0 ** -32 * (small.double() @ vv.abs())
        err = (out[:, h].double() - ref).abs()
        assert bool((err <= tol).all()), (h, float((err / tol).max()))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 8, 20, 40])
@pytest.mark.parametrize("low,high", [(15.0, 18.0), (18.5, 20.9), (22.0, 25.0)])
def test_tree_attention_beside_a_dominant_position(D, n, low, high):
    ctx = 32768
    gaps = np.random.default_rng(n).uniform(low, high, n)
    k, v, q, scale, table, desc = _dominated(D, n, ctx, gaps, D + n)
    out, st = torch.empty_like(q), _status()
    need = pk.pa_tree_workspace_bytes(1, table.shape[1], n, desc)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    pk.pa_tree_attention(out, q, k, v, table, _i32([ctx]), _i32([0, n]), None, scale, desc,
                         max_q_len=n, workspace=ws, status=st)
    assert st.item() == 0
    _check_dominated(out, k, v, q, scale, n, ctx)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gap", [15.6, 18.6, 20.6, 22.6])
def test_weights_beside_a_dominant_position(D, gap):
    ctx = 32768
    k, v, q, scale, table, desc = _dominated(D, 1, ctx, [gap], D)
    out, st = torch.empty_like(q), _status()
    w = torch.empty(1, desc.num_heads, ctx, device="cuda")
    need = pk.pa_decode_weights_workspace_bytes(1, table.shape[1], desc)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    pk.pa_decode_attention_weights(out, w, None, q, k, v, table, _i32([ctx]), scale, desc,
                                   workspace=ws, status=st)
    assert st.item() == 0
    _check_dominated(out, k, v, q, scale, 1, ctx)
    # The weights themselves.  The one score that is not 0, at most 23 binary
    # orders, is a product of three roundings (the scale's two and its own) of
    # 2^-24 and loses half a step of 2^-19 with the reference: 2^-17.6 in all, of
    # which a power of 2 makes 2^-18.1 of itself, below 2^-17 with its own error.
    # The sum it is divided by: a thread adds up every 128th term, ctx / 128 of
    # them, and each addition rounds the running sum, which is almost all of the
    # row's where the large term is in it, by 2^-24 of it, alike for equal terms.
    x = q[0, 0, 0].double() * k[0, 0, 0, 0].double() * scale
    one = torch.exp(-x) / (1 + (ctx - 1) * torch.exp(-x))
    assert bool(((w[0, :, 1:].double() - one).abs() <= (2.0 ** -17 + ctx / 128 * 2.0 ** -24) * one).all())


# ------------------------------------------- rows beside rows that jump


@pytest.mark.parametrize("D,B", [(64, 16), (128, 16)])
@pytest.mark.parametrize("n,S", [(7, 24), (16, 24), (16, 90), (30, 24), (64, 24)])
def test_tree_attention_rows_do_not_depend_on_keys_they_do_not_see(D, B, n, S):
    """A node whose finite key lifts the scores of the rows that see it by some
    20 binary orders: every other row is the same to the bit."""
    H = 8
    ctx = [300 + 7 * s for s in range(S)]
    b = Batch(n + D + S, ctx, [n] * S, H, D, B, scale_q=2.0)
    up = b.forest(n)
    clean = b.run(up)
    seen = torch.zeros(b.rows + 2, dtype=torch.bool, device="cuda")
    r = np.random.default_rng(n)
    for s, c in enumerate(ctx):
        a, t = int(b.starts[s]), int(r.integers(1, n))
        row = b.q[a + t].float()
        key = row * (20.0 * math.log(2) / (b.scale * (row * row).sum(-1, keepdim=True)))
        pos = c - n + t
        b.k[int(b.tables[s, pos // B]), :, pos % B] = key.half()
        for x in range(t, n):
            y = x
            while y > t:
                y = int(up[a + y])
            seen[a + x] = y == t
    assert bool(seen.any())
    got = b.run(up)
    assert torch.equal(got[~seen], clean[~seen])
    # (the scores' error, D 2^-24 of the sum of |q k| <= 20 binary orders and some,
    # stays below the 2^-12 that the check allows)
    b.check(got, up)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 5, 13, 21])
def test_tree_attention_does_not_depend_on_the_next_sequence(D, n):
    """Rows are handled by eight: those of the next sequence among them, whose
    queries here are large."""
    S, H = 40, 8
    b = Batch(n + D, [500 + 9 * s for s in range(S)], [n] * S, H, D, 16)
    up = b.forest(n)
    clean = b.run(up)
    odd = torch.arange(b.rows, device="cuda") // n % 2 == 1
    b.q[:b.rows][odd] = b.q[:b.rows][odd] * 40
    got = b.run(up)
    assert torch.equal(got[:b.rows][~odd], clean[:b.rows][~odd])


# ------------------------------------------------- verification's borders


@pytest.mark.parametrize("V,front,back,S", [(1020, 768, 1000, 4096), (20476, 1536, 2053, 1000)])
def test_verify_random_numbers_on_a_border(V, front, back, S):
    """u_sample = 1/2 falls, to the rounding of the sums, on the border between
    the tokens before `front` and two at `back` that weigh as much together;
    nothing between them weighs anything.  The next token is the last one before
    the border or the first one behind it."""
    r = np.random.default_rng(V)
    p = np.zeros((S, V), np.float32)
    # over so many binary orders that sums in another order round otherwise
    p[:, :front] = np.exp2(-24 * r.random((S, front))) / front
    for s in range(S):
        total = math.fsum(p[s, :front].tolist())
        hi = np.float32(total)
        if float(hi) >= total:
            hi = np.nextafter(hi, np.float32(0))
        p[s, back], p[s, back + 1] = hi, np.float32(total - float(hi))
    assert (p[:, [front - 1, back, back + 1]] > 0).all()
    st = _status()
    starts = np.arange(S + 1)
    path, lens, nxt = _verify(_dev(p), None, np.zeros(S), None, starts, np.zeros(S), np.full(S, 0.5), status=st)
    assert st.item() == 0
    assert np.isin(nxt, [front - 1, back]).all(), np.unique(nxt[~np.isin(nxt, [front - 1, back])])
    # beside the border there is no doubt
    for us, want in ((0.5 - 2.0 ** -12, range(front)), (0.5 + 2.0 ** -12, [back])):
        _, _, nxt = _verify(_dev(p), None, np.zeros(S), None, starts, np.zeros(S), np.full(S, us), status=st)
        assert np.isin(nxt, list(want)).all()


def test_picked_tokens_leave_the_target_its_distribution():
    """Siblings that are always the drafter's three most probable tokens, without
    draft probabilities: the token decided after the root has the target's
    distribution.  40000 draws, 12 tokens: every frequency within 5 standard
    deviations."""
    S, V = 40000, 12
    r = np.random.default_rng(9)
    p1 = r.dirichlet(np.ones(V))
    starts = np.arange(S + 1) * 4
    p = torch.from_numpy(np.tile(p1, (4 * S, 1))).float().cuda()
    tokens = np.tile(np.array([0, 7, 2, 5], np.int32), S)
    up = np.tile(np.array([-1, 0, 0, 0], np.int32), S)
    path, lens, nxt = _verify(p, None, tokens, up, starts, r.random(4 * S), r.random(S))
    first = np.where(lens > 1, tokens[starts[:-1] + path[:, 1]], nxt)
    f = np.bincount(first, minlength=V) / S
    assert (np.abs(f - p1) <= 5 * np.sqrt(p1 * (1 - p1) / S)).all()
