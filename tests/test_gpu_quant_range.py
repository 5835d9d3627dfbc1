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
