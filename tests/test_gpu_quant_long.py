"""Calls in which every CTA goes through its rings of stages many times: attention of
many and of long contexts by each form of its kernel (references: test_gpu_quant_attention),
norm and rotation of many tokens with and without the slot write (test_gpu_norm_rope)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_106_gb300 as pk
from tests import quantised as qz
from tests.test_gpu_norm_rope import _close, _reference, _table
from tests.test_gpu_quant_attention import BF16, F16, Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,rep,D,B,bits", [
    (40, 1, 128, 16, 4), (8, 2, 128, 16, 4), (3, 2, 128, 16, 4), (8, 4, 128, 32, 4), (2, 8, 128, 8, 4), (4, 12, 128, 16, 4),
    (2, 40, 128, 16, 4), (16, 2, 64, 32, 4), (8, 4, 64, 16, 4), (5, 8, 64, 8, 4), (8, 1, 128, 16, 8), (8, 2, 128, 16, 8),
    (8, 4, 128, 16, 8), (8, 8, 128, 16, 8), (4, 20, 128, 32, 8), (6, 3, 128, 32, 8), (8, 2, 64, 16, 8), (8, 8, 64, 32, 8)])
@pytest.mark.parametrize("spread", [0.0, 1.5])
def test_many_tiles_a_cta(H, rep, D, B, bits, spread):
    """Contexts of 128 to 3000; with `spread`, references move along them."""
    r = np.random.RandomState(H + rep)
    ctx = r.randint(128, 3001, 96).tolist()
    ctx[17], ctx[40], ctx[95] = 0, 1, 2999
    b = Batch(71 + H, ctx, H, rep, D, B, bits, BF16 if rep % 2 else F16, scale_q=1.0 if spread else 2.0, spread=spread)
    out = b.run()
    b.check(out, only={0, 17, 40, 95, *r.randint(0, 96, 5).tolist()})
    assert torch.equal(b.run(), out)


@pytest.mark.parametrize("H,rep,D,B,bits", [(16, 2, 64, 32, 4), (4, 1, 128, 16, 4), (2, 8, 128, 16, 8), (1, 3, 64, 8, 8)])
def test_long_contexts(H, rep, D, B, bits):
    b = Batch(73 + H, [40001, 65536, 50017], H, rep, D, B, bits)
    b.check(b.run())


@pytest.mark.parametrize("D,rot,pairs,hq,hk,norm", [(128, 128, False, 40, 40, True), (128, 64, True, 32, 8, True),
                                                     (128, 24, False, 40, 8, False), (64, 64, False, 71, 9, True),
                                                     (256, 256, True, 16, 4, True)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_norm_and_rotation_of_many_tokens(D, rot, pairs, hq, hk, norm, dtype):
    n = 20011
    g = torch.Generator("cuda").manual_seed(D + rot)
    x = torch.randn(n, hq + hk, D, generator=g, device="cuda").mul_(3).to(dtype)
    q, k = x[:, :hq], x[:, hq:]
    w = [(1 + 0.5 * torch.randn(D, generator=g, device="cuda")).to(dtype) if norm else None for _ in range(2)]
    table, pos = _table(700, rot), torch.randint(0, 700, (n,), generator=g, device="cuda", dtype=torch.int32)
    out = [torch.empty((n, h, D), dtype=dtype, device="cuda") for h in (hq, hk)]
    st = qz.status()
    pk.pa_norm_rope(*out, q, k, *w, 1e-5, table, pos, interleaved=pairs, status=st)
    assert st.item() == 0
    for got, src, wt in zip(out, (q, k), w):
        for a in range(0, n, 4000):
            _close(got[a:a + 4000], *_reference(src[a:a + 4000], wt, 1e-5, table, pos[a:a + 4000], rot, pairs))


@pytest.mark.parametrize("D,B,bits,dtype,hq,hk,rot,pairs", [
    (128, 16, 16, F16, 32, 8, 64, True), (128, 16, 8, BF16, 32, 8, 128, False), (128, 16, 4, F16, 40, 40, 128, False),
    (64, 32, 4, BF16, 8, 8, 64, False), (64, 8, 8, F16, 9, 3, 24, True), (128, 32, 8, F16, 0, 5, 8, False),
    (256, 16, 16, F16, 8, 4, 256, False)])
def test_slot_write_of_many_tokens(D, B, bits, dtype, hq, hk, rot, pairs):
    """Bit for bit what the rows of pa_norm_rope (above) and the slot write give."""
    n, blocks = 25013, -(-25013 // B) + 5
    g = torch.Generator("cuda").manual_seed(D + B + bits)
    x = torch.randn(n, hq + 2 * hk, D, generator=g, device="cuda").to(dtype)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    table, pos = _table(90, rot), torch.randint(0, 90, (n,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(blocks * B, generator=g, device="cuda")[:n]
    slots[::911] = -1
    desc = pk.PoolDesc(blocks, B, num_heads=hk, head_dim=D) if bits == 16 else qz.desc(blocks, B, hk, D, bits)
    shape = (blocks, hk, B, D) if bits == 16 else (blocks, hk, qz.block_bytes(D, bits, B))
    one = [torch.full(shape, 3, dtype=F16 if bits == 16 else torch.uint8, device="cuda") for _ in range(2)]
    two = [t.clone() for t in one]
    q1, q2 = (torch.full((n, hq, D), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    k2 = torch.empty(n, hk, D, dtype=dtype, device="cuda")
    st = qz.status()
    pk.pa_norm_rope_write_kv(q1, q, k, v, *w, 1e-6, table, pos, slots, *one, desc, interleaved=pairs, status=st)
    pk.pa_norm_rope(q2, k2, q, k, *w, 1e-6, table, pos, interleaved=pairs, status=st)
    _close(k2, *_reference(k, w[1], 1e-6, table, pos, rot, pairs))
    (pk.pa_write_kv if bits == 16 else pk.pa_write_kv_quant)(k2, v.contiguous(), slots, *two, desc, status=st)
    assert st.item() == 0 and torch.equal(q1, q2)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
