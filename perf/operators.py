"""Operators of speculative decoding and of a bounded cache, as they are measured.

Four kinds of pass over the paged cache:

* ``tree``     attention of a tree of drafted tokens over each sequence's cached
               context (the drafted tokens are its last positions);
* ``verify``   acceptance of the drafted tokens against the target's
               probabilities, and the next token, from given random numbers;
* ``weights``  decode attention that adds each position's attention weight to
               a running sum per (sequence, head, position);
* ``compact``  rows of the cache moved to the front of a sequence: after a
               verification the accepted drafts (all layers, ``by="path"``), or
               after a selection by accumulated weight the positions that a
               budget keeps (one layer, a set per head, ``by="weight"``).

``run`` computes them in elementary torch operations, or, with ``own`` set,
through the package's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    layer = {"heads": 40, "dim": 128, "block": 16}     # the benchmark's attention layer
    return [
        # one interactive request, eight drafted tokens in a row: latency counts
        {"name": "tree_1x8", "kind": "tree", "seqs": 1, "ctx_lo": 2048, "ctx_hi": 2048,
         "n_lo": 8, "n_hi": 8, "chain": True, **layer},
        # a serving batch of mixed lengths with small draft trees of uneven size
        {"name": "tree_64_mixed", "kind": "tree", "seqs": 64, "ctx_lo": 128, "ctx_hi": 2048,
         "n_lo": 4, "n_hi": 16, "chain": False, **layer},
        # a full batch with the largest trees: 64 nodes a sequence
        {"name": "tree_256x64", "kind": "tree", "seqs": 256, "ctx_lo": 128, "ctx_hi": 1536,
         "n_lo": 64, "n_hi": 64, "chain": False, **layer},
        # few sequences with long contexts, narrow heads, a wide block
        {"name": "tree_long", "kind": "tree", "seqs": 3, "ctx_lo": 40001, "ctx_hi": 65536,
         "n_lo": 17, "n_hi": 31, "chain": False, "heads": 32, "dim": 64, "block": 32},
        # one request, eight drafts in a row, one row of probabilities to sample from
        {"name": "verify_1x8", "kind": "verify", "seqs": 1, "vocab": 32000, "n_lo": 8, "n_hi": 8,
         "chain": True, "dtype": "f32", "onehot": False},
        # a full batch of draft chains against a 50 k vocabulary
        {"name": "verify_256x8", "kind": "verify", "seqs": 256, "vocab": 50272, "n_lo": 5,
         "n_hi": 9, "chain": True, "dtype": "f32", "onehot": False},
        # draft trees (several candidates per position), an odd vocabulary in half precision
        {"name": "verify_trees", "kind": "verify", "seqs": 64, "vocab": 100003, "n_lo": 10,
         "n_hi": 26, "chain": False, "dtype": "f16", "onehot": False},
        # a decode step of the mixed batch that keeps score of every position
        {"name": "weights_64", "kind": "weights", "seqs": 64, "ctx_lo": 128, "ctx_hi": 2048,
         **layer},
        # two long conversations
        {"name": "weights_long", "kind": "weights", "seqs": 2, "ctx_lo": 50001, "ctx_hi": 65536,
         **layer},
        # a batch cut back to 512 positions a head, the last 64 among them; some are shorter
        {"name": "evict_64", "kind": "compact", "by": "weight", "seqs": 64, "ctx_lo": 256,
         "ctx_hi": 2048, "budget": 512, "recent": 64, **layer},
        # long conversations cut to an eighth
        {"name": "evict_long", "kind": "compact", "by": "weight", "seqs": 4, "ctx_lo": 20001,
         "ctx_hi": 32768, "budget": 4096, "recent": 511, **layer},
        # accepted drafts of a full batch moved into place in 24 layers
        {"name": "commit_256", "kind": "compact", "by": "path", "seqs": 256, "layers": 24,
         "n_lo": 8, "n_hi": 26, "most": 8, "ctx_lo": 128, "ctx_hi": 2048, **layer},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        kind = rng.choice(["tree", "tree", "verify", "weights", "compact", "compact"])
        geo = {"heads": _log(rng, 1, 48), "dim": rng.choice([64, 128, 128]),
               "block": rng.choice([8, 16, 16, 32])}
        if kind == "verify":
            n = _log(rng, 1, 64)
            c = {"kind": kind, "seqs": _log(rng, 1, 256), "vocab": _log(rng, 500, 130000),
                 "n_lo": rng.randint(1, n), "n_hi": n, "chain": rng.random() < 0.4,
                 "dtype": rng.choice(["f32", "f32", "f16", "bf16"]),
                 "onehot": rng.random() < 0.25}
            if c["seqs"] * c["n_hi"] * c["vocab"] <= 256 * 9 * 50272 and \
                    c["seqs"] * c["vocab"] * c["n_hi"] ** 0.5 <= 256 * 50272 * 3:
                return c
            continue
        seqs, top = _log(rng, 1, 256), _log(rng, 33, 65536)
        lo = rng.randint(max(1, top // 16), top)
        tokens = seqs * (lo + top) / 2 * geo["heads"] * geo["dim"]
        if kind == "tree":
            n = _log(rng, 1, 64)
            n_lo = rng.randint(1, n)
            c = {"kind": kind, "seqs": seqs, "ctx_lo": max(lo, n), "ctx_hi": max(top, n),
                 "n_lo": n_lo, "n_hi": n, "chain": rng.random() < 0.3, **geo}
            if tokens <= 7e8 and seqs * top <= 4e5 and tokens * n <= 4e10:
                return c
        elif kind == "weights":
            if tokens <= 5e8 and seqs * top <= 2.5e5:
                return {"kind": kind, "seqs": seqs, "ctx_lo": lo, "ctx_hi": top, **geo}
        elif rng.random() < 0.5:
            budget = _log(rng, 16, 8192)
            if tokens <= 5e8 and seqs * top <= 1.5e5 and tokens > 1e5:
                return {"kind": kind, "by": "weight", "seqs": seqs, "ctx_lo": lo, "ctx_hi": top,
                        "budget": budget, "recent": rng.randint(0, budget), **geo}
        else:
            n, layers = _log(rng, 2, 64), _log(rng, 1, 30)
            if seqs * layers * geo["heads"] * geo["dim"] * (n + 64) <= 256 * 24 * 40 * 128 * 90:
                return {"kind": kind, "by": "path", "seqs": seqs, "layers": layers,
                        "n_lo": rng.randint(1, n), "n_hi": n, "most": rng.randint(1, 16),
                        "ctx_lo": 1, "ctx_hi": _log(rng, 32, 4096), **geo}


# ------------------------------------------------------------------- inputs


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _lens(case, what):
    """One length a sequence: a case's own, whatever the seed of the values."""
    r = np.random.RandomState([case["seqs"], case[what + "_lo"], case[what + "_hi"]])
    return r.randint(case[what + "_lo"], case[what + "_hi"] + 1, case["seqs"])


def _forest(r, lens, chain):
    """Parent of every node (node 0 of a sequence is its root), rows of all sequences."""
    rows = []
    for n in lens:
        up = np.arange(n) - 1
        if not chain:   # mostly recent nodes, some high up: wide and deep trees
            back = np.minimum(r.geometric(0.35, n), np.maximum(np.arange(n), 1))
            up = np.arange(n) - back
            up[0] = -1
        rows.append(up)
    return np.concatenate(rows)


def _tables(r, blocks, spare=0):
    """Scattered block tables padded with -1, and the pool's size."""
    total = int(blocks.sum()) + spare + max(1, int(blocks.sum()) // 8)
    free, at = r.permutation(total), 0
    t = np.full((len(blocks), int(blocks.max())), -1)
    for i, n in enumerate(blocks):
        t[i, :n] = free[at:at + n]
        at += n
    return t, total, free[at:]


def prepare(case, seed):
    r = np.random.RandomState(seed % (1 << 32))
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}

    def normal(*shape, scale=1.0):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
        return x if scale == 1.0 else x.mul_(scale)

    if case["kind"] == "verify":
        n = _lens(case, "n")
        starts = np.concatenate([[0], np.cumsum(n)])
        rows, V = int(starts[-1]), case["vocab"]
        t = DTYPES[case["dtype"]]
        logits = torch.randn((rows, V), generator=g, device="cuda") * 2.5
        s["p"] = torch.softmax(logits, 1).to(t)
        logits += torch.randn((rows, V), generator=g, device="cuda") * 0.7
        q = torch.softmax(logits, 1).to(t)
        del logits
        s["parents"] = up = _i32(_forest(r, n, case["chain"]))
        # each drafted token is drawn from the drafter's row of its parent
        row = torch.from_numpy(np.repeat(starts[:-1], n)).cuda() + up.clamp(min=0)
        pick = torch.empty(rows, dtype=torch.int64, device="cuda")
        for a in range(0, rows, 256):
            pick[a:a + 256] = torch.multinomial(q[row[a:a + 256]].float(), 1, generator=g)[:, 0]
        s["tokens"] = pick.int()
        s["q"] = None if case["onehot"] else q
        s["starts"], s["nmax"] = _i32(starts), int(n.max())
        s["u"] = torch.rand(rows, generator=g, device="cuda")
        s["us"] = torch.rand(case["seqs"], generator=g, device="cuda")
        if own:
            S = case["seqs"]
            s["path"] = torch.empty((S, s["nmax"]), dtype=torch.int32, device="cuda")
            s["n_path"] = torch.empty(S, dtype=torch.int32, device="cuda")
            s["next"] = torch.empty(S, dtype=torch.int32, device="cuda")
        return s

    H, D, B, S = case["heads"], case["dim"], case["block"], case["seqs"]
    ctx = _lens(case, "ctx")
    s["scale"] = float(np.float32(1 / math.sqrt(D)))
    if case["kind"] == "compact":
        if case["by"] == "path":
            # drafted nodes lie in scratch blocks of their own; the accepted
            # ones go behind the sequence's `ctx` tokens
            n = _lens(case, "n")
            base = ctx % B      # the front of the table is not needed here
            keep = np.full((S, 1, case["most"]), -1)
            length = np.minimum(r.randint(1, case["most"] + 1, S), n)
            for i in range(S):
                keep[i, 0, :length[i]] = np.concatenate(
                    [[0], 1 + np.sort(r.permutation(n[i] - 1)[:length[i] - 1])])
            total = base + n
        else:
            base, total = np.zeros(S, np.int64), ctx
        src, blocks, left = _tables(r, -(-total // B), spare=int(sum(-(-total // B))))
        dst = np.full_like(src, -1)
        dst[src >= 0] = left[:(src >= 0).sum()]
        L = case.get("layers", 1)
        s["k"] = [normal(blocks, H, B, D) for _ in range(L)]
        s["v"] = [normal(blocks, H, B, D) for _ in range(L)]
        s["src"], s["dst"], s["ctx"], s["first"] = _i32(src), _i32(dst), _i32(total), _i32(base)
        if case["by"] == "path":
            s["keep"], s["keep_lens"] = _i32(keep), _i32(length)
        else:
            # sums of weights over many steps: few positions hold most of it
            W = src.shape[1] * B
            w = torch.randn((S, H, W), generator=g, device="cuda").mul_(2).exp_()
            inside = torch.arange(W, device="cuda") < s["ctx"][:, None, None]
            s["w"] = torch.where(inside, w, 0.0)
            s["w_out"] = torch.zeros_like(s["w"])
        if own:
            import paged_kv_cache_106_gb300 as pk
            s["desc"] = pk.PoolDesc(blocks, B, num_layers=L, num_heads=H, head_dim=D)
            if case["by"] == "weight":
                s["keep"] = torch.empty((S, H, case["budget"]), dtype=torch.int32, device="cuda")
                s["keep_lens"] = torch.empty(S, dtype=torch.int32, device="cuda")
        return s

    tables, blocks, _ = _tables(r, -(-ctx // B))
    s["k"], s["v"] = normal(blocks, H, B, D), normal(blocks, H, B, D)
    s["tables"], s["ctx"] = _i32(tables), _i32(ctx)
    n = _lens(case, "n") if case["kind"] == "tree" else np.ones(S, np.int64)
    starts = np.concatenate([[0], np.cumsum(n)])
    s["q"] = normal(int(starts[-1]), H, D, scale=2.0)
    if case["kind"] == "tree":
        s["starts"], s["nmax"] = _i32(starts), int(n.max())
        s["parents"] = _i32(_forest(r, n, case["chain"]))
    else:
        W = tables.shape[1] * B
        s["w"] = torch.rand((S, H, W), generator=g, device="cuda")
        s["w_out"] = torch.zeros_like(s["w"])
    if own:
        import paged_kv_cache_106_gb300 as pk
        s["desc"] = desc = pk.PoolDesc(blocks, B, num_heads=H, head_dim=D)
        s["out"] = torch.empty_like(s["q"])
        need = (pk.pa_tree_workspace_bytes(S, tables.shape[1], s["nmax"], desc)
                if case["kind"] == "tree" else
                pk.pa_decode_weights_workspace_bytes(S, tables.shape[1], desc))
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"tree": _own_tree, "verify": _own_verify, "weights": _own_weights,
                "compact": _own_compact}[kind](s)
    return {"tree": _tree, "verify": _verify, "weights": _weights, "compact": _compact}[kind](s)


def _own_tree(s):
    import paged_kv_cache_106_gb300 as pk
    pk.pa_tree_attention(s["out"], s["q"], s["k"], s["v"], s["tables"], s["ctx"], s["starts"],
                         s["parents"], s["scale"], s["desc"], max_q_len=s["nmax"],
                         workspace=s["ws"])
    return s["out"]


def _own_verify(s):
    import paged_kv_cache_106_gb300 as pk
    pk.pa_verify_draft(s["path"], s["n_path"], s["next"], s["p"], s["q"], s["tokens"],
                       s["parents"], s["starts"], s["u"], s["us"], max_q_len=s["nmax"])
    return {"path": s["path"], "n_path": s["n_path"], "next": s["next"]}


def _own_weights(s):
    import paged_kv_cache_106_gb300 as pk
    pk.pa_decode_attention_weights(s["out"], s["w_out"], s["w"], s["q"], s["k"], s["v"],
                                   s["tables"], s["ctx"], s["scale"], s["desc"],
                                   workspace=s["ws"])
    return {"out": s["out"], "weights": s["w_out"]}


def _own_compact(s):
    import paged_kv_cache_106_gb300 as pk
    c = s["case"]
    if c["by"] == "weight":
        pk.pa_evict_select(s["keep"], s["keep_lens"], s["w_out"], s["w"], s["ctx"], c["budget"],
                           c["recent"])
    pk.pa_compact_kv(s["k"], s["v"], s["src"], s["dst"], s["ctx"], s["keep"], s["keep_lens"],
                     s["desc"], first=s["first"])
    moved = {"k": s["k"], "v": s["v"]}
    if c["by"] == "weight":
        moved.update(keep=s["keep"], keep_lens=s["keep_lens"], weights=s["w_out"])
    return moved


def _context(s, cache):
    """The sequences' rows of a cache in order of position, in 32 bits: [S, H, positions, D]."""
    t = s["tables"].long().clamp(min=0)
    x = cache[t].permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4]).float()


def _tree(s):
    S, N = s["ctx"].shape[0], s["nmax"]
    starts, n = s["starts"][:-1].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    node = torch.arange(N, device="cuda")
    have = node < n[:, None]                                       # [S, N]
    rows = torch.where(have, starts[:, None] + node, 0)
    # a node sees itself and its ancestors: the reachable ones of its parent links
    up = torch.where(have, s["parents"][rows].long(), -1)
    sees = (up[:, :, None] == node) | (node[:, None] == node)
    for _ in range(max(1, (N - 1).bit_length())):
        sees = torch.matmul(sees.float(), sees.float()) > 0
    k = _context(s, s["k"])
    pos = torch.arange(k.shape[2], device="cuda")
    ctx, base = s["ctx"].long(), s["ctx"].long() - n
    j = (pos - base[:, None]).clamp(0, N - 1)                      # the draft node at a position
    drafted = torch.gather(sees, 2, j[:, None, :].expand(S, N, -1))
    visible = torch.where(pos < base[:, None, None], True, drafted & (pos < ctx[:, None, None]))
    q = s["q"][rows].float().permute(0, 2, 1, 3)                   # [S, H, N, D]
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    del k
    x = x.masked_fill_(~visible[:, None], -math.inf)
    x = x.sub_(x.amax(3, keepdim=True)).exp_()
    o = torch.matmul(x, _context(s, s["v"])) / x.sum(3, keepdim=True)
    # back to the rows of q: sequence by sequence, node by node
    at = torch.repeat_interleave(torch.arange(S, device="cuda"), n, output_size=s["q"].shape[0])
    i = torch.arange(s["q"].shape[0], device="cuda") - starts[at]
    return o[at, :, i].half()


def _verify(s):
    p, tokens, parents = s["p"], s["tokens"].long(), s["parents"].long()
    starts, n = s["starts"][:-1].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    S = starts.shape[0]
    every = torch.arange(S, device="cuda")
    cur = torch.zeros_like(starts)
    w, z = p[starts].double(), torch.ones(S, dtype=torch.float64, device="cuda")
    path = torch.full((S, s["nmax"]), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    n_path = torch.ones_like(starts)
    for i in range(1, s["nmax"]):      # nodes in order: a walk from the root, siblings in turn
        row = starts + torch.clamp(n - 1, max=i)
        tried = (i < n) & (parents[row] == cur)
        x = tokens[row][:, None]
        if s["q"] is None:
            q = torch.zeros_like(w).scatter_(1, x, 1.0)
        else:
            q = s["q"][starts + cur].double()
        yes = tried & (s["u"][row].double() * q.gather(1, x)[:, 0] * z < w.gather(1, x)[:, 0])
        rest = (w - q * z[:, None]).clamp_(min=0)
        left = rest.sum(1)
        no = tried & ~yes & (left > 0)
        w = torch.where(no[:, None], rest, w)
        z = torch.where(no, left, z)
        w = torch.where(yes[:, None], p[row].double(), w)
        z = torch.where(yes, 1.0, z)
        cur = torch.where(yes, i, cur)
        at = torch.clamp(n_path, max=s["nmax"] - 1)
        path[every, at] = torch.where(yes, i, path[every, at]).int()
        n_path = n_path + yes
    c = w.cumsum(1)
    nxt = (c <= s["us"].double()[:, None] * c[:, -1:]).sum(1)
    last = p.shape[1] - 1 - (w > 0).flip(1).int().argmax(1)
    return {"path": path, "n_path": n_path.int(), "next": torch.minimum(nxt, last).int()}


def _weights(s):
    k = _context(s, s["k"])
    inside = torch.arange(k.shape[2], device="cuda") < s["ctx"].long()[:, None, None]
    x = (k * s["q"].float()[:, :, None]).sum(3) * s["scale"]
    del k
    x = x.masked_fill(~inside, -math.inf)
    x = (x - x.amax(2, keepdim=True)).exp()
    x = x / x.sum(2, keepdim=True)
    o = torch.matmul(x[:, :, None], _context(s, s["v"]))[:, :, 0]
    return {"out": o.half(), "weights": torch.where(inside, s["w"] + x, s["w_out"])}


def _compact(s):
    c, ctx = s["case"], s["ctx"].long()
    moved = {}
    if c["by"] == "weight":
        W, budget, recent = s["w"].shape[2], c["budget"], c["recent"]
        pos = torch.arange(W, device="cuda")
        length = torch.clamp(ctx, max=budget)
        key = torch.where(pos >= (ctx - recent)[:, None, None], math.inf, s["w"])
        key = torch.where(pos < ctx[:, None, None], key, -math.inf)
        first = torch.sort(key, dim=2, descending=True, stable=True)[1][:, :, :budget]
        j = torch.arange(first.shape[2], device="cuda")
        have = j < length[:, None, None]
        kept = torch.sort(torch.where(have, first, W), dim=2)[0]
        moved["keep_lens"] = length.int()
        moved["keep"] = torch.full((*kept.shape[:2], budget), -1, dtype=torch.int32, device="cuda")
        moved["keep"][:, :, :kept.shape[2]] = torch.where(have, kept, -1).int()
        w = torch.where(pos < ctx[:, None, None], 0.0, s["w_out"])
        gathered = s["w"].gather(2, kept.clamp(max=W - 1))
        w[:, :, :kept.shape[2]] = torch.where(have, gathered, w[:, :, :kept.shape[2]])
        moved["weights"] = w
        keep, lens = kept, length
    else:
        keep, lens = s["keep"].long(), s["keep_lens"].long()
    S, H, B = ctx.shape[0], c["heads"], c["block"]
    j = torch.arange(keep.shape[2], device="cuda").expand(S, H, -1)
    keep = keep.expand(S, H, -1)
    have = j < lens[:, None, None]
    first = s["first"].long()[:, None, None]
    # what is not kept repeats the first row's move
    old = first + torch.where(have, keep, keep[:, :, :1])
    new = first + torch.where(have, j, 0)
    seq = torch.arange(S, device="cuda")[:, None, None]
    head = torch.arange(H, device="cuda")[None, :, None]
    a = (s["src"].long()[seq, old // B], head, old % B)
    b = (s["dst"].long()[seq, new // B], head, new % B)
    for cache in s["k"] + s["v"]:
        cache[b] = cache[a]
    return {"k": s["k"], "v": s["v"], **moved}


# ----------------------------------------------------------- what it takes


def work(case):
    c = case
    S = c["seqs"]
    if c["kind"] == "verify":
        # one row of the target's and one of the drafter's probabilities a sequence
        size = 4 if c["dtype"] == "f32" else 2
        rows = S * (c["n_lo"] + c["n_hi"]) / 2
        both = 1 if c["onehot"] else 2
        return {"bytes": S * c["vocab"] * size * both + rows * 20, "flops": 4 * S * c["vocab"]}
    H, D = c["heads"], c["dim"]
    tokens = S * (c["ctx_lo"] + c["ctx_hi"]) / 2
    if c["kind"] == "compact":
        if c["by"] == "path":
            rows = S * c["layers"] * min((c["most"] + 1) / 2, (c["n_lo"] + c["n_hi"]) / 2)
            return {"bytes": rows * H * D * 2 * 4, "flops": 0}
        kept = S * min(c["budget"], (c["ctx_lo"] + c["ctx_hi"]) / 2)
        # rows read and written, the sums read, kept and zeroed
        return {"bytes": kept * H * (D * 2 * 4 + 4) + tokens * H * 8, "flops": tokens * H}
    rows = S * (c["n_lo"] + c["n_hi"]) / 2 if c["kind"] == "tree" else S
    flops = 4 * D * H * tokens * rows / S
    sums = tokens * H * 8 if c["kind"] == "weights" else 0
    return {"bytes": tokens * H * D * 4 + rows * H * D * 4 + tokens / c["block"] * 4 + sums,
            "flops": flops}


# ------------------------------------------------ the definition, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "weights": _exact_weights,
            "compact": _exact_compact}[case["kind"]](s)


def _rows64(s, cache, i, count):
    """The first `count` positions of sequence i, in 64 bits: [positions, H, D]."""
    B = s["case"]["block"]
    at = torch.arange(count, device="cuda")
    return cache[s["tables"][i].long()[at // B], :, at % B].double()


def _exact_tree(s):
    starts, ctx = s["starts"].tolist(), s["ctx"].tolist()
    parents = s["parents"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, c in enumerate(ctx):
        a, b = starts[i], starts[i + 1]
        bar = torch.zeros(b - a, c, dtype=torch.float64)
        bar[:, c - (b - a):] = -math.inf
        for t in range(b - a):
            up = t
            while up >= 0:
                bar[t, c - (b - a) + up] = 0
                up = parents[a + up]
        x = torch.einsum("thd,phd->htp", s["q"][a:b].double(), _rows64(s, s["k"], i, c))
        x = torch.softmax(x * s["scale"] + bar.cuda(), -1)
        out[a:b] = torch.einsum("htp,phd->thd", x, _rows64(s, s["v"], i, c))
    return out


def _exact_verify(s):
    starts, parents, tokens = s["starts"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    u, us = s["u"].double().tolist(), s["us"].double().tolist()
    path = torch.full((len(us), s["nmax"]), -1, dtype=torch.int32)
    n_path, nxt = [], []
    for i in range(len(us)):
        a, b = starts[i], starts[i + 1]
        node, walked, moved = 0, [0], True
        while moved:
            w, total, moved = s["p"][a + node].double(), 1.0, False
            for child in (t for t in range(1, b - a) if parents[a + t] == node):
                x = tokens[a + child]
                q = s["q"][a + node].double() if s["q"] is not None else \
                    torch.nn.functional.one_hot(torch.tensor(x), w.shape[0]).double().cuda()
                if u[a + child] * float(q[x]) * total < float(w[x]):
                    node, moved = child, True
                    walked.append(child)
                    break
                rest = torch.relu(w - total * q)
                if float(rest.sum()) > 0:
                    w, total = rest, float(rest.sum())
        c = torch.cumsum(w, 0)
        past = torch.searchsorted(c, c[-1:] * us[i], right=True)
        nxt.append(min(int(past), int(w.nonzero()[-1])))
        path[i, :len(walked)] = torch.tensor(walked, dtype=torch.int32)
        n_path.append(len(walked))
    return {"path": path, "n_path": torch.tensor(n_path, dtype=torch.int32),
            "next": torch.tensor(nxt, dtype=torch.int32)}


def _exact_weights(s):
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    w = s["w_out"].double()
    for i, c in enumerate(s["ctx"].tolist()):
        x = torch.einsum("hd,phd->hp", s["q"][i].double(), _rows64(s, s["k"], i, c))
        x = torch.softmax(x * s["scale"], -1)
        out[i] = torch.einsum("hp,phd->hd", x, _rows64(s, s["v"], i, c))
        w[i, :, :c] = s["w"][i, :, :c].double() + x
    return {"out": out, "weights": w}


def _exact_compact(s):
    c, ctx, first = s["case"], s["ctx"].tolist(), s["first"].tolist()
    S, H, B = len(ctx), c["heads"], c["block"]
    src, dst = s["src"].cpu().numpy().astype(np.int64), s["dst"].cpu().numpy().astype(np.int64)
    by_weight = c["by"] == "weight"
    moved, chosen = {}, []
    if by_weight:
        w = s["w"].cpu().numpy()
        w_out = s["w_out"].cpu().numpy()
        lens = [min(t, c["budget"]) for t in ctx]
        keep = np.full((S, H, c["budget"]), -1, np.int32)
        for i, t in enumerate(ctx):
            heavy = max(0, lens[i] - min(c["recent"], t))
            old = t - (lens[i] - heavy)
            w_out[i, :, :t] = 0
            for h in range(H):
                order = np.argsort(-w[i, h, :old], kind="stable")[:heavy]
                keep[i, h, :lens[i]] = np.concatenate([np.sort(order), np.arange(old, t)])
                w_out[i, h, :lens[i]] = w[i, h][keep[i, h, :lens[i]]]
        moved = {"keep": torch.from_numpy(keep),
                 "keep_lens": torch.tensor(lens, dtype=torch.int32),
                 "weights": torch.from_numpy(w_out).double()}
    else:
        keep, lens = s["keep"].cpu().numpy(), s["keep_lens"].tolist()
        keep = np.broadcast_to(keep, (S, H, keep.shape[2]))
    for i in range(S):
        old = first[i] + keep[i, :, :lens[i]].astype(np.int64)        # [H, rows]
        new = first[i] + np.broadcast_to(np.arange(lens[i]), old.shape)
        head = np.broadcast_to(np.arange(H)[:, None], old.shape)
        chosen.append(np.stack([src[i][old // B], old % B, dst[i][new // B], new % B, head]))
    at = torch.from_numpy(np.concatenate([x.reshape(5, -1) for x in chosen], 1)).cuda()
    caches = {}
    for name in ("k", "v"):
        caches[name] = []
        for cache in s[name]:
            x = cache.clone()
            x[at[2], at[4], at[3]] = cache[at[0], at[4], at[1]]
            caches[name].append(x)
    return {**caches, **moved}
