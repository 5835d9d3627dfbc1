"""Norm of heads where its formula has no number, and at the ends of the range that
the header gives for rows of bf16 (reference and tolerance: test_gpu_norm_rope)."""
import pytest
import torch

import paged_kv_cache_106_gb300 as pk
from tests.test_gpu_norm_rope import BF16, F16, _close, _reference, _table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_head_of_zeros(D, dtype):
    """0 / 0 with a weight and an eps of 0, in that head alone; 0 otherwise."""
    x = torch.randn(3, 5, D, device="cuda").to(dtype)
    x[1, 2] = 0
    w, table, pos = torch.ones(D, device="cuda").to(dtype), _table(9, D), torch.arange(3, device="cuda", dtype=torch.int32)
    for weight, eps, none in ((w, 0.0, True), (w, 1e-6, False), (None, 0.0, False)):
        q, k = (torch.full((3, h, D), 7.0, dtype=dtype, device="cuda") for h in (4, 1))
        pk.pa_norm_rope(q, k, x[:, :4], x[:, 4:], weight, None, eps, table, pos)
        assert bool(q[1, 2].isnan().all()) if none else bool((q[1, 2] == 0).all())
        ref, size = _reference(x[:, :4], weight, eps, table, pos, D, False)
        rest = torch.ones(3, 4, dtype=torch.bool, device="cuda")
        rest[1, 2] = False
        _close(q[rest], ref[rest], size[rest])
        _close(k, *_reference(x[:, 4:], None, eps, table, pos, D, False))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("top", [59, 30, -30, -54])
def test_bf16_rows_within_the_range(D, top):
    """Largest magnitudes just below 2^top, without an eps."""
    x = torch.randn(40, 6, D, device="cuda").double()
    x = (x / x.abs().amax(2, keepdim=True) * 0.99 * 2.0 ** top).to(BF16)
    w = (1 + 0.3 * torch.randn(D, device="cuda")).to(BF16)
    table, pos = _table(50, D), torch.arange(40, device="cuda", dtype=torch.int32)
    q, k = (torch.empty(40, h, D, dtype=BF16, device="cuda") for h in (4, 2))
    pk.pa_norm_rope(q, k, x[:, :4], x[:, 4:], w, w, 0.0, table, pos)
    _close(q, *_reference(x[:, :4], w, 0.0, table, pos, D, False))
    _close(k, *_reference(x[:, 4:], w, 0.0, table, pos, D, False))
