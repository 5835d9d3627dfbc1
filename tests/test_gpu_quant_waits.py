"""Attention over a quantised cache whose bounded waits give up, without a fault: a
status word that already holds PA_ERR_TIMEOUT ends every wait that does not
succeed at once.  Such a call ends, keeps to its own output, and leaves nothing that the
next call on its workspace meets."""
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
