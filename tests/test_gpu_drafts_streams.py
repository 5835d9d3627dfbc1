"""Calls for drafted tokens and for the bounded cache in flight on two streams at
once: everything is prepared first, the calls are enqueued in turn without a
wait between them, and the results are compared at the end."""
import pytest
import torch

import paged_kv_cache_106_gb300 as pk
from tests.test_gpu_drafts import Batch, _dev, _drafts, _i32, _status

pytestmark = pytest.mark.gpu


def _tree_call(b, up, st):
    desc = pk.PoolDesc(b.nb, b.B, num_heads=b.H, head_dim=b.D)
    out, n = torch.empty_like(b.q[:b.rows]), max(b.n)
    ws = torch.empty(pk.pa_tree_workspace_bytes(len(b.ctx), b.tables.shape[1], n, desc),
                     dtype=torch.uint8, device="cuda")
    t, c, s, u = _dev(b.tables), _i32(b.ctx), _i32(b.starts), _i32(up)
    return [out], lambda: pk.pa_tree_attention(out, b.q, b.k, b.v, t, c, s, u, b.scale, desc,
                                               max_q_len=n, workspace=ws, status=st)


def _weights_call(b, st):
    S, W = len(b.ctx), b.tables.shape[1] * b.B
    desc = pk.PoolDesc(b.nb, b.B, num_heads=b.H, head_dim=b.D)
    out = torch.empty(S, b.H, b.D, dtype=torch.float16, device="cuda")
    w = torch.zeros(S, b.H, W, device="cuda")
    ws = torch.empty(pk.pa_decode_weights_workspace_bytes(S, b.tables.shape[1], desc),
                     dtype=torch.uint8, device="cuda")
    t, c = _dev(b.tables), _i32(b.ctx)
    return [out, w], lambda: pk.pa_decode_attention_weights(out, w, w, b.q[:S], b.k, b.v, t, c,
                                                            b.scale, desc, workspace=ws, status=st)


def _verify_call(d, st):
    p, q, tokens, up, starts, u, us = d
    S, mq = len(us), int((starts[1:] - starts[:-1]).max())
    path = torch.empty(S, mq, dtype=torch.int32, device="cuda")
    lens, nxt = (torch.empty(S, dtype=torch.int32, device="cuda") for _ in range(2))
    args = _i32(tokens), _i32(up), _i32(starts), _dev(u), _dev(us)
    return [path, lens, nxt], lambda: pk.pa_verify_draft(path, lens, nxt, p, q, *args, status=st)


def _select_call(seed, S, H, W, budget, st):
    g = torch.Generator("cuda").manual_seed(seed)
    w = torch.randn(S, H, W, generator=g, device="cuda").exp()
    kept, c = torch.zeros_like(w), _i32([W] * S)
    keep = torch.empty(S, H, budget, dtype=torch.int32, device="cuda")
    lens = torch.empty(S, dtype=torch.int32, device="cuda")
    return [kept, keep, lens], lambda: pk.pa_evict_select(keep, lens, kept, w, c, budget, 9, status=st)


def test_calls_in_flight_on_two_streams():
    st = _status()
    trees = [Batch(71, [4000, 900, 64, 2500], [12, 40, 64, 3], 24, 128, 16),
             Batch(72, [700 + 50 * s for s in range(20)], [1 + s % 16 for s in range(20)], 24, 64, 32)]
    one = Batch(73, [3000, 33, 1500] * 8, [1] * 24, 16, 128, 16)
    calls = [[_tree_call(trees[0], trees[0].forest(1), st),
              _verify_call(_drafts(74, [6] * 100, 20011, torch.float16), st),
              _weights_call(one, st)],
             [_tree_call(trees[1], trees[1].forest(2), st), _select_call(75, 12, 24, 30000, 700, st),
              _tree_call(trees[0], trees[0].forest(3), st),
              _verify_call(_drafts(76, [9, 1, 20], 50001, torch.float32), st)]]
    # one after another, each stream's outputs by round (the weights add up)
    rounds, want = 12, [[], []]
    for side in (0, 1):
        for _ in range(rounds):
            for outs, call in calls[side]:
                call()
                torch.cuda.synchronize()
            want[side].append([x.clone() for outs, _ in calls[side] for x in outs])
    for outs, _ in calls[0] + calls[1]:
        for x in outs:
            x.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[[torch.empty_like(x) for x in r] for r in want[side]] for side in (0, 1)]
    torch.cuda.synchronize()
    for i in range(rounds):
        for k in range(4):
            for side in (0, 1):
                with torch.cuda.stream(streams[side]):
                    if k < len(calls[side]):
                        calls[side][k][1]()
                    if k == 3:
                        for x, y in zip(got[side][i], (x for outs, _ in calls[side] for x in outs)):
                            x.copy_(y)
    torch.cuda.synchronize()
    for side in (0, 1):
        for i in range(rounds):
            for k, (x, y) in enumerate(zip(got[side][i], want[side][i])):
                assert torch.equal(x, y), (side, i, k)
    assert st.item() == 0
