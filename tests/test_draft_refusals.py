"""What the calls for drafted tokens and for the bounded cache refuse before
anything reaches the GPU: tensors by the bindings, scalars and addresses by the
library (none of these addresses is ever read)."""
import math

import pytest
import torch

import paged_kv_cache_106_gb300 as pk

A = 1 << 20            # an aligned address that nothing reads
DESC = pk.PoolDesc(8, 16, num_heads=2, head_dim=64)


def _zeros(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def _tree(desc=DESC, n=2, mb=4, rows=4, max_q=4, scale=0.1, out=A, q=A, k=A, v=A, tables=A, ctx=A,
          starts=A, parents=None, ws=None, ws_bytes=0, status=None):
    return pk._lib.pa_tree_attention(out, q, k, v, tables, ctx, starts, parents, n, mb, max_q, rows,
                                     scale, ws, ws_bytes, status, desc.ref, 0)


def _weights(desc=DESC, n=2, mb=4, wl=64, scale=0.1, out=A, w_out=A, w_in=None, q=A, k=A, v=A,
             tables=A, ctx=A, ws=None, ws_bytes=0, status=None):
    return pk._lib.pa_decode_attention_weights(out, w_out, w_in, wl, q, k, v, tables, ctx, n, mb,
                                               scale, ws, ws_bytes, status, desc.ref, 0)


GEOMETRIES = [pk.PoolDesc(8, 16, num_heads=2, head_dim=32), pk.PoolDesc(8, 16, num_heads=2, head_dim=256),
              pk.PoolDesc(8, 4, num_heads=2, head_dim=64)]


@pytest.mark.parametrize("bad", [
    *({"desc": d} for d in GEOMETRIES), {"n": -1}, {"n": 4097}, {"mb": -1}, {"mb": 0},
    {"mb": (1 << 31) // 16}, {"rows": -1}, {"max_q": -1}, {"max_q": 65}, {"scale": math.inf},
    {"scale": math.nan}, {"out": None}, {"q": None}, {"k": None}, {"v": None}, {"tables": None},
    {"ctx": None}, {"starts": None}, {"out": A + 8}, {"q": A + 8}, {"k": A + 8}, {"v": A + 8},
    {"tables": A + 2}, {"ctx": A + 1}, {"starts": A + 2}, {"parents": A + 2}, {"status": A + 2},
    {"ws": None}, {"ws": A, "ws_bytes": 100}, {"ws": A + 128, "ws_bytes": 1 << 30}])
def test_tree_attention_refuses(bad):
    assert _tree(**bad) == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    *({"desc": d} for d in GEOMETRIES), {"n": -1}, {"n": 4097}, {"mb": -1}, {"mb": 0},
    {"mb": (1 << 31) // 16}, {"wl": -1}, {"scale": math.inf}, {"out": None}, {"w_out": None},
    {"q": None}, {"k": None}, {"v": None}, {"tables": None}, {"ctx": None}, {"out": A + 8},
    {"w_out": A + 2}, {"w_in": A + 1}, {"q": A + 8}, {"k": A + 4}, {"status": A + 3}, {"ws": None},
    {"ws": A, "ws_bytes": 100}, {"ws": A + 16, "ws_bytes": 1 << 30}])
def test_weights_refuse(bad):
    assert _weights(**bad) == pk.PA_ERR_INVALID_ARG


def test_empty_calls_do_nothing():
    for bad in ({"n": 0}, {"rows": 0}, {"max_q": 0}):
        assert _tree(**bad) == pk.PA_OK
    assert _weights(n=0) == pk.PA_OK


def test_workspace_sizes_are_zero_where_the_call_is_refused():
    assert pk.pa_tree_workspace_bytes(4, 8, 16, DESC) > 0
    assert pk.pa_decode_weights_workspace_bytes(4, 8, DESC) > 0
    for n, mb, mq in ((0, 8, 16), (4097, 8, 16), (4, -1, 16), (4, 8, 0), (4, 8, 65)):
        assert pk.pa_tree_workspace_bytes(n, mb, mq, DESC) == 0
    for d in GEOMETRIES:
        assert pk.pa_tree_workspace_bytes(4, 8, 16, d) == 0
        assert pk.pa_decode_weights_workspace_bytes(4, 8, d) == 0


@pytest.mark.parametrize("bad", [
    {"dtype": 3}, {"n": -1}, {"n": 65536}, {"rows": -1}, {"vocab": 0}, {"vocab": (1 << 30) + 1},
    {"max_q": 0}, {"max_q": 65}, {"path": None}, {"lens": None}, {"nxt": None}, {"p": None},
    {"tokens": None}, {"starts": None}, {"u": None}, {"us": None}, {"p": A + 2}, {"q": A + 2},
    {"path": A + 2}, {"lens": A + 1}, {"tokens": A + 2}, {"parents": A + 2}, {"u": A + 2},
    {"us": A + 2}, {"status": A + 2}])
def test_verify_refuses(bad):
    a = dict(path=A, lens=A, nxt=A, p=A, q=A, dtype=pk.PA_DTYPE_F32, tokens=A, parents=None,
             starts=A, u=A, us=A, n=2, max_q=4, rows=8, vocab=100, status=None)
    a.update(bad)
    assert pk._lib.pa_verify_draft(a["path"], a["lens"], a["nxt"], a["p"], a["q"], a["dtype"],
                                   a["tokens"], a["parents"], a["starts"], a["u"], a["us"], a["n"],
                                   a["max_q"], a["rows"], a["vocab"], a["status"],
                                   0) == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    {"n": -1}, {"n": 65536}, {"heads": 0}, {"wl": -1}, {"budget": 0}, {"recent": -1},
    {"recent": 9}, {"keep": None}, {"lens": None}, {"w_out": None}, {"w_in": None}, {"ctx": None},
    {"keep": A + 2}, {"lens": A + 2}, {"w_out": A + 2}, {"w_in": A + 1}, {"status": A + 1}])
def test_select_refuses(bad):
    a = dict(keep=A, lens=A, w_out=A, w_in=A, wl=64, ctx=A, n=2, heads=2, budget=8, recent=2, status=None)
    a.update(bad)
    assert pk._lib.pa_evict_select(a["keep"], a["lens"], a["w_out"], a["w_in"], a["wl"], a["ctx"],
                                   a["n"], a["heads"], a["budget"], a["recent"], a["status"],
                                   0) == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    {"layers": -1}, {"layers": 129}, {"n": -1}, {"n": 65536}, {"mb": -1}, {"stride": -1},
    {"heads": 3}, {"heads": 0}, {"src": None}, {"dst": None}, {"lens": None}, {"keep": None},
    {"keep_lens": None}, {"src": A + 2}, {"keep": A + 1}, {"first": A + 2}, {"status": A + 2},
    {"k": None}, {"k": A + 8}, {"v": None}, {"v": A + 4}])
def test_moves_refuse(bad):
    import ctypes
    a = dict(k=A, v=A, layers=1, src=A, dst=A, lens=A, first=None, keep=A, keep_lens=A, heads=1,
             stride=4, n=2, mb=4, status=None)
    a.update(bad)
    k, v = (ctypes.c_void_p * 1)(a["k"]), (ctypes.c_void_p * 1)(a["v"])
    assert pk._lib.pa_compact_kv(k, v, a["layers"], a["src"], a["dst"], a["lens"], a["first"],
                                 a["keep"], a["keep_lens"], a["heads"], a["stride"], a["n"],
                                 a["mb"], DESC.ref, a["status"], 0) == pk.PA_ERR_INVALID_ARG


def test_bindings_refuse_tensors_that_do_not_fit():
    h, f = torch.float16, torch.float32
    q = _zeros(4, 2, 64, dtype=h)
    with pytest.raises(ValueError, match="out"):                  # not on the GPU
        pk.pa_tree_attention(q, q, q, q, _zeros(2, 4), _zeros(2), _zeros(3), None, 0.1, DESC, 4)
    p = _zeros(4, 50, dtype=f)
    args = (_zeros(4), None, _zeros(3), _zeros(4, dtype=f), _zeros(2, dtype=f))
    with pytest.raises(ValueError, match="width"):
        pk.pa_verify_draft(_zeros(2, 4), _zeros(2), _zeros(2), p, _zeros(4, 51, dtype=f), *args)
    with pytest.raises(ValueError, match="max_q_len"):
        pk.pa_verify_draft(_zeros(2, 4), _zeros(2), _zeros(2), p, p, *args, max_q_len=3)
    with pytest.raises(ValueError, match="float64"):
        pk.pa_verify_draft(_zeros(2, 4), _zeros(2), _zeros(2), p.double(), None, *args)
    w = _zeros(2, 3, 64, dtype=f)
    with pytest.raises(ValueError, match="heads"):
        pk.pa_decode_attention_weights(q, w, None, q, q, q, _zeros(2, 4), _zeros(2), 0.1, DESC)
    with pytest.raises(ValueError, match="length"):
        pk.pa_decode_attention_weights(q, w, w[:, :, 1:], q, q, q, _zeros(2, 4), _zeros(2), 0.1, DESC)
    with pytest.raises(ValueError, match="keep"):
        pk.pa_evict_select(_zeros(2, 3, 7), _zeros(2), w, w, _zeros(2), 8, 2)
    with pytest.raises(ValueError, match="shape"):
        pk.pa_evict_select(_zeros(2, 3, 8), _zeros(2), w, w[:, 1:], _zeros(2), 8, 2)
    with pytest.raises(ValueError, match="differ in length"):
        pk.pa_compact_kv([q], [], _zeros(2, 4), _zeros(2, 4), _zeros(2), _zeros(2, 4), _zeros(2), DESC)
    with pytest.raises(ValueError, match="differ in width"):
        pk.pa_compact_kv([q], [q], _zeros(2, 4), _zeros(2, 5), _zeros(2), _zeros(2, 4), _zeros(2), DESC)
