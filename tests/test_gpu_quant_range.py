"""Attention over a quantised cache with queries and scales at the ends of their
types' ranges, against the evaluation in 64 bits (tolerances: test_gpu_quant_attention)."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_106_gb300 as pk
from tests.test_gpu_quant_attention import BF16, Batch

pytestmark = pytest.mark.gpu

LAST = float(torch.finfo(torch.float32).max)


def _queries(b, top):
    """Rows whose largest magnitude is just below 2^top (bf16's largest number is, of 2^128)."""
    x = b.q.double()
    x = x / x.abs().amax(2, keepdim=True) * 0.99          # largest 0.99, so just below 2^top
    return (x * 2.0 ** top).to(BF16)


@pytest.mark.parametrize("bits,H,rep,D,B", [(8, 2, 4, 128, 16), (8, 2, 1, 128, 16), (8, 1, 8, 128, 32), (8, 2, 3, 64, 16),
                                            (8, 1, 20, 64, 8), (4, 2, 4, 128, 16), (4, 2, 2, 128, 32), (4, 1, 9, 128, 8),
                                            (4, 3, 2, 64, 32)])
@pytest.mark.parametrize("top", [128, 127, 126, 100, 97, 96, 0, -94, -95, -96, -98, -110, -124, -128, -132])
def test_bf16_queries_to_the_ends_of_their_range(bits, H, rep, D, B, top):
    """Scales bring their scores into the usual range: largest query elements of 2^(top - 1) to 2^top."""
    b = Batch(61, [90, 400, 1], H, rep, D, B, bits, dtype=BF16)
    b.q = _queries(b, top)
    assert bool(b.q.isfinite().all()) and bool((b.q.abs().float().amax(2) > 0).all())
    b.scale = float(np.float32(min(4.0 / math.sqrt(D) * 2.0 ** -top, LAST)))
    b.check(b.run())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("scale", [LAST, -LAST, 1e30])
def test_the_largest_scales(bits, scale):
    """Queries of zeros weigh every position alike; small ones give ordinary scores."""
    b = Batch(62, [90, 400, 1], 2, 4, 128, 16, bits, dtype=BF16)
    b.q = torch.zeros_like(b.q)
    b.scale = scale
    b.check(b.run())
    b.q = (torch.randn(b.q.shape, generator=torch.Generator("cuda").manual_seed(63), device="cuda").double() / abs(scale) / 8).to(BF16)
    b.scale = float(np.float32(scale))
    b.check(b.run())


SHAPES = [(4, 1, 128, 16), (2, 4, 128, 16), (2, 8, 128, 32), (3, 2, 64, 16), (1, 6, 64, 8), (1, 20, 128, 16)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H,rep,D,B", SHAPES)
@pytest.mark.parametrize("top", [20, 22, 23, 24, 26, 28, 40, 70, 100])
def test_scores_far_apart(bits, H, rep, D, B, top):
    """Scores of about +-2^top: one position has all the weight where the next is further
    away than the scores' error E (the tolerances' of test_gpu_quant_attention, and
    2^-22 of the score for its product with the scale and the reference) by 40 or more,
    so that what is left is 400 * e^-40 of the values.  Weight * scale is rounded once
    (2^-11), the sums and the join of that position's value add 34 * 2^-24 of what is summed (231
    scales in 4 bits), as there; the output is rounded once."""
    b = Batch(64 + top, [400, 1, 2100], H, rep, D, B, bits, dtype=BF16)
    b.scale = 2.0 ** (top - 5)
    out = b.run()
    assert bool(out.isfinite().all())
    seen = 0
    for i, n in enumerate(b.ctx):
        k, ks, v, vs = b.rows64(i, n)
        q = b.q[i].double().reshape(H, rep, D)
        y = torch.einsum("hrd,phd->hrp", q, k) * b.scale
        g = q.unflatten(2, (-1, 32))
        M = b._constant(g) + (272.0 if bits == 4 else 1280.0) * g.abs().amax(-1) + (7 if bits == 4 else 127) * g.abs().sum(-1)
        E = b.scale * 34 * 2.0 ** -24 * torch.einsum("hrg,phg->hrp", M, ks).amax(-1) + \
            b.scale * 2.0 ** -21 * q.abs().amax(-1) * k.abs().sum(-1).amax(0)[:, None] + 2.0 ** -22 * y.abs().amax(-1)
        best = y.topk(min(2, n), -1)
        alone = torch.ones_like(E, dtype=torch.bool) if n == 1 else best.values[..., 0] - best.values[..., 1] > 2 * E + 40
        at = best.indices[..., 0]
        ref = torch.stack([v[at[h], h] for h in range(H)])
        scale = torch.stack([vs[at[h], h] for h in range(H)]).repeat_interleave(32, -1)
        summed = 231 * scale if bits == 4 else ref.abs()
        tol = torch.finfo(BF16).eps / 2 * ref.abs() + 2.0 ** -11 * ref.abs() + 34 * 2.0 ** -24 * summed + 2.0 ** -24 + \
            n * math.exp(-40) * v.abs().max()
        err = (out[i].double().reshape_as(ref) - ref).abs()
        assert bool((err <= tol)[alone].all())
        seen += int(alone.sum())
    assert seen >= H * rep * 2           # (a context of one, and as many rows of the others)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H,rep,D,B", SHAPES)
@pytest.mark.parametrize("scale", [2.0 ** 18, -2.0 ** 21, 2.0 ** 40, -2.0 ** 90])
def test_equal_scores_far_from_zero(bits, H, rep, D, B, scale):
    """The same key everywhere: the mean of the values, however large the score, and
    also where the values' scales grow along the context."""
    b = Batch(67, [3000, 77], H, rep, D, B, bits, dtype=BF16)
    n = b.nb * b.B
    g = torch.Generator("cuda").manual_seed(68)
    key = torch.randn(1, H, D, generator=g, device="cuda").half().expand(n, H, D)
    grow = torch.linspace(-8, 8, n, device="cuda").exp2()[:, None, None]
    value = torch.empty(n, H, D, device="cuda")
    order = torch.cat([torch.from_numpy(t[:-(-c // B)].astype(np.int64)).cuda() for t, c in zip(b.tables, b.ctx)])
    rest = torch.from_numpy(np.setdiff1d(np.arange(b.nb), order.cpu().numpy())).cuda()
    value.copy_(torch.randn(n, H, D, generator=g, device="cuda") * grow)
    slots = (torch.cat([order, rest])[:, None] * B + torch.arange(B, device="cuda")).flatten()
    pk.pa_write_kv_quant(key, value.half(), slots, *b.caches, b.desc())
    # (weights are equal: only weight * scale's rounding and the sums are left of the tolerance)
    b.scale = scale
    out = b.run()
    assert bool(out.isfinite().all())
    small = b.scale
    b.check(out, scale=small / 2.0 ** 140)          # scores of nothing: the mean, without an error of theirs
