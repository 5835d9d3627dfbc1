"""Arguments of the calls for drafted tokens, for the bounded cache and of the
one-call steps that are refused, or taken, on the host (none of these addresses
is ever read)."""
import ctypes

import pytest
import torch

import paged_kv_cache_106_gb300 as pk

A = 1 << 24            # an aligned address that nothing reads
DESC = pk.PoolDesc(8, 16, num_layers=2, num_heads=2, head_dim=64)
SIZE = 8 * 16 * 2 * 64 * 2             # bytes of a cache


def _compact(k, v):
    L = len(k)
    return pk._lib.pa_compact_kv((ctypes.c_void_p * L)(*k), (ctypes.c_void_p * L)(*v), L, A, A, A, None,
                                 A, A, 1, 4, 2, 4, DESC.ref, None, 0)


@pytest.mark.parametrize("k,v", [([A], [A]), ([A, A], [A + SIZE, A + 2 * SIZE]),
                                 ([A, A + SIZE], [A + 2 * SIZE, A + SIZE]),
                                 ([A], [A + SIZE - 16]), ([A + SIZE - 16], [A]),
                                 ([A + 3 * SIZE, A], [A + SIZE, A + 3 * SIZE - 16])])
def test_moves_refuse_caches_that_overlap(k, v):
    """Each cache is moved by blocks of its own, in any order: moved twice, its
    rows would be read after they were written over."""
    assert _compact(k, v) == pk.PA_ERR_INVALID_ARG
    assert "overlap" in pk.pa_last_error_string()


def test_one_call_steps_refuse_addresses_of_new_rows():
    """How many rows lie there cannot be checked."""
    q, tables, ctx = torch.zeros(3, 2, 64), torch.zeros(3, 4), torch.zeros(3)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="k_new"):
        pk.pa_decode_step_attention(q, q, A, q, slots, q, q, tables, ctx, 0.1, DESC)
    with pytest.raises(ValueError, match="slot_mapping"):
        pk.pa_decode_step_attention(q, q, q, q, A, q, q, tables, ctx, 0.1, DESC)
    with pytest.raises(ValueError, match="v_new"):
        pk.pa_prefill_step_attention(q, q, q, A, q, q, tables, ctx, ctx, 0.1, DESC, max_q_len=3)


class Fake:
    """What the bindings ask of a tensor; the calls here end before its address
    is used (scale is NaN, which the library refuses, where nothing else is)."""

    def __init__(self, shape, dtype=torch.float16, device=0, contiguous=True):
        self.shape, self.dtype, self.contiguous = shape, dtype, contiguous
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")
        self.is_cuda, self.index = device >= 0, device

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def data_ptr(self):
        return A


def _i32(*shape, **kw):
    return Fake(shape, torch.int32, **kw)


def _tree(**changed):
    a = dict(out=Fake((4, 2, 64)), q=Fake((4, 2, 64)), k_cache=Fake((8, 2, 16, 64)),
             v_cache=Fake((8, 2, 16, 64)), block_tables=_i32(2, 4), ctx_lens=_i32(2),
             q_starts=_i32(3), parents=_i32(4), scale=float("nan"), desc=DESC, max_q_len=4,
             workspace=Fake((1 << 30,), torch.uint8), stream=0)
    pk.pa_tree_attention(**{**a, **changed})


def _weights(**changed):
    a = dict(out=Fake((2, 2, 64)), weights_out=Fake((2, 2, 64), torch.float32), weights_in=None,
             q=Fake((2, 2, 64)), k_cache=Fake((8, 2, 16, 64)), v_cache=Fake((8, 2, 16, 64)),
             block_tables=_i32(2, 4), ctx_lens=_i32(2), scale=float("nan"), desc=DESC,
             workspace=Fake((1 << 30,), torch.uint8), stream=0)
    pk.pa_decode_attention_weights(**{**a, **changed})


@pytest.fixture
def one_gpu(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


@pytest.mark.parametrize("call", [_tree, _weights])
def test_workspaces_are_checked(call, one_gpu):
    with pytest.raises(pk.PagedKVError, match="scale"):      # nothing else is wrong
        call()
    for bad in (A, Fake((1 << 20,), torch.uint8, device=-1), Fake((1 << 20,), contiguous=False)):
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=bad)
    # any type will do; none is refused by the library
    with pytest.raises(pk.PagedKVError, match="scale"):
        call(workspace=Fake((1 << 20,), torch.float32))
    with pytest.raises(pk.PagedKVError, match="workspace"):
        call(workspace=None, scale=0.1)


def _verify(**changed):
    p = Fake((6, 50), torch.float32)
    a = dict(path=_i32(2, 0), path_lens=_i32(2), next_tokens=_i32(2), target_probs=p, draft_probs=p,
             draft_tokens=_i32(6), parents=_i32(6), q_starts=_i32(3), u_accept=Fake((6,), torch.float32),
             u_sample=Fake((2,), torch.float32), stream=0)      # (max_q_len 0)
    pk.pa_verify_draft(**{**a, **changed})


def _select(**changed):
    w = Fake((2, 2, 64), torch.float32)
    a = dict(keep=_i32(2, 2, 8), keep_lens=_i32(2), weights_out=w, weights_in=w, ctx_lens=_i32(2),
             budget=8, recent=9, stream=0)
    pk.pa_evict_select(**{**a, **changed})


def _move(**changed):
    c = Fake((8, 2, 16, 64))
    a = dict(k_caches=[c], v_caches=[c], src_tables=_i32(2, 4), dst_tables=_i32(2, 4),
             src_lens=_i32(2), keep=_i32(2, 8), keep_lens=_i32(2), desc=DESC, first=_i32(2), stream=0)
    pk.pa_compact_kv(**{**a, **changed})


@pytest.mark.parametrize("call,tensors,refusal", [
    (_tree, {"out": Fake((4, 2, 64), device=1), "q": Fake((4, 2, 64), device=1),
             "k_cache": Fake((8, 2, 16, 64), device=1), "v_cache": Fake((8, 2, 16, 64), device=1),
             "block_tables": _i32(2, 4, device=1), "ctx_lens": _i32(2, device=1),
             "q_starts": _i32(3, device=1), "parents": _i32(4, device=1),
             "workspace": Fake((1 << 30,), torch.uint8, device=1), "status": _i32(1, device=1)}, "scale"),
    (_weights, {"out": Fake((2, 2, 64), device=1), "weights_out": Fake((2, 2, 64), torch.float32, device=1),
                "weights_in": Fake((2, 2, 64), torch.float32, device=1),
                "workspace": Fake((1 << 30,), torch.uint8, device=1)}, "scale"),
    (_verify, {"target_probs": Fake((6, 50), torch.float32, device=1), "u_sample": Fake((2,), torch.float32, device=1),
               "path": _i32(2, 0, device=1)}, "max_q_len"),
    (_select, {"keep": _i32(2, 2, 8, device=1), "ctx_lens": _i32(2, device=1)}, "recent"),
    (_move, {"k_caches": [Fake((8, 2, 16, 64), device=1)], "first": _i32(2, device=1),
             "dst_tables": _i32(2, 4, device=1)}, "overlap")])
def test_tensors_on_another_gpu_are_refused(call, tensors, refusal, one_gpu):
    """Kernels run on the current GPU, which all tensors have to be on."""
    with pytest.raises(pk.PagedKVError, match=refusal):      # nothing else is wrong
        call()
    for name, t in tensors.items():
        with pytest.raises(ValueError, match=name):
            call(**{name: t})
