"""Attention over a quantised cache whose bounded waits may give up, without a fault:
with a status word that already holds PA_ERR_TIMEOUT a wait gives up as soon as its
barrier has not come by the hardware's own limit (which copies rarely exceed, so most
runs see few or none).  Whichever do, the call ends, keeps to its own output, and
leaves nothing that the next call on its workspace meets."""
import time

import numpy as np
import pytest
import torch

import paged_kv_cache_106_gb300 as pk
from tests import quantised as qz
from tests.test_gpu_quant_attention import Batch

pytestmark = pytest.mark.gpu


def _given_up(b, ws):
    """The call with such a status word and that workspace, its output between rows of others."""
    wide = torch.full((len(b.ctx) + 2, *b.q.shape[1:]), 7.0, dtype=b.q.dtype, device="cuda")
    st = torch.full((1,), pk.PA_ERR_TIMEOUT, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.monotonic()
    b.run(st, out=wide[1:-1], ws=ws)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 10
    assert st.item() == pk.PA_ERR_TIMEOUT
    assert bool((wide[0] == 7).all()) and bool((wide[-1] == 7).all())
    for i, n in enumerate(b.ctx):
        if n <= 0:
            assert bool((wide[i + 1] == 0).all())


@pytest.mark.parametrize("H,rep,D,B,bits", [(8, 4, 128, 16, 4), (1, 2, 64, 8, 4), (3, 8, 128, 32, 8), (2, 12, 64, 16, 8)])
def test_many_sequences(H, rep, D, B, bits):
    """More units than CTAs, with one warp and with several to a head's positions."""
    ctx = np.random.RandomState(H).randint(0, 300, 700).tolist()
    b = Batch(H + rep, ctx, H, rep, D, B, bits)
    good = b.run()
    ws = torch.zeros(pk.pa_decode_quant_workspace_bytes(len(ctx), H * rep, b.desc()), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        _given_up(b, ws)
        assert torch.equal(b.run(qz.status(), ws=ws), good)


@pytest.mark.parametrize("H,rep,D,B,bits,units", [(8, 4, 128, 16, 4, 2), (2, 20, 64, 32, 4, 2), (4, 8, 128, 16, 8, 1),
                                                  (1, 70, 128, 16, 4, 3)])
def test_entries_of_few_sequences(H, rep, D, B, bits, units):
    """Units whose parts are joined by an entry each, several to a CTA: every entry
    is written (they come first in the workspace: first CTA, parts, sequence, unit, or
    zeros), whatever stood there, and no other sequence's."""
    ctx = [60000, 0] + [40] * 60 + [-3, 9000] + [17] * 30
    b = Batch(H + rep, ctx, H, rep, D, B, bits)
    good = b.run()
    ws = torch.empty(pk.pa_decode_quant_workspace_bytes(len(ctx), H * rep, b.desc()), dtype=torch.uint8, device="cuda")
    want = np.stack(np.divmod(np.arange(len(ctx) * units), units), 1)
    empty = np.repeat(np.array(ctx) <= 0, units)
    ctas = torch.cuda.get_device_properties(0).multi_processor_count * 3
    assert len(want) <= ctas * 2 // 3
    for before in (-99, 0):
        ws.view(torch.int32).fill_(before)
        _given_up(b, ws)
        entry = ws[:16 * len(want)].view(torch.int32).reshape(-1, 4).cpu().numpy()
        assert (entry[empty] == 0).all()
        first, parts = entry[~empty, 0], entry[~empty, 1]
        assert (entry[~empty, 2:] == want[~empty]).all()
        assert (first >= 0).all() and (parts >= 1).all() and (first + parts <= ctas).all()
    assert torch.equal(b.run(qz.status(), ws=ws), good)
