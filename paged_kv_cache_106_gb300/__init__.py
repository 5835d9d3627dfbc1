"""GB300 paged KV cache decode step: thin Python binding of libpagedkv.so.

Every function here has the name of the C entry point it calls
(``include/pagedkv.h``) and only marshals arguments: host arrays go in as
numpy arrays, device buffers as CUDA torch tensors (or raw device addresses),
streams as torch streams (default: torch's current stream).  All the work --
block management on the host, slot write, block copy and decode attention on
the GPU -- runs in the library.  There is no fallback: if the library is
missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# always the library that the package's own build step writes next to it
_LIB_PATH = os.path.join(_PKG, "libpagedkv.so")

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_OUT_OF_BLOCKS = 2
PA_ERR_NO_SEQ = 3
PA_ERR_CUDA = 4
PA_ERR_TIMEOUT = 5
PA_ERR_BAD_BLOCK = 6
PA_DTYPE_F16 = 0
PA_DTYPE_F32 = 1
PA_DTYPE_BF16 = 2
PA_DTYPE_I8 = 3
PA_DTYPE_I4 = 4
PA_TREE_MAX_NODES = 64
PA_TREE_MAX_SEQS = 4096
PA_POOL_PREFIX_CACHING = 1
PA_DEFAULT_PARTITION_TOKENS = 512
PA_NOALLOC_SCRATCH_BYTES = 32 << 20

_ERR_NAMES = {1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_OUT_OF_BLOCKS", 3: "PA_ERR_NO_SEQ",
              4: "PA_ERR_CUDA", 5: "PA_ERR_TIMEOUT", 6: "PA_ERR_BAD_BLOCK"}


class PagedKVError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_ERR_NAMES.get(code, code)}: {msg}")
        self.code = code


class OutOfBlocks(PagedKVError):
    pass


class pa_pool_desc(ctypes.Structure):
    _fields_ = [
        ("num_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_layers", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("partition_tokens", ctypes.c_int32),
        ("flags", ctypes.c_int32),
        ("free_order", ctypes.POINTER(ctypes.c_int32)),
    ]


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` "
            "(or python paged_kv_cache_106_gb300/_build.py)")
    lib = ctypes.CDLL(_LIB_PATH)
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER
    sig = {
        "pa_last_error_string": (ctypes.c_char_p, []),
        "pa_pool_create": (i32, [P(pa_pool_desc), P(vp)]),
        "pa_pool_destroy": (i32, [vp]),
        "pa_seq_add": (i32, [vp, i32, i32, vp]),
        "pa_seq_add_tokens": (i32, [vp, i32, i32, vp, i64, vp, P(i32)]),
        "pa_pool_cached_blocks": (i32, [vp, P(i32)]),
        "pa_swap_out": (i32, [vp, vp, i32, vp, vp, i32, P(i32)]),
        "pa_swap_in": (i32, [vp, vp, i32, vp, vp, i32, P(i32)]),
        "pa_swap_blocks": (i32, [vp, vp, i32, vp, vp, i32, i32, vp, i32, P(pa_pool_desc), vp, vp]),
        "pa_seq_fork": (i32, [vp, i32, i32]),
        "pa_seq_fork_batch": (i32, [vp, i32, vp, vp]),
        "pa_seq_free_batch": (i32, [vp, i32, vp]),
        "pa_seq_free": (i32, [vp, i32]),
        "pa_beam_prune": (i32, [vp, i32, i32, vp, vp, P(i32)]),
        "pa_alloc_slots": (i32, [vp, i32, vp, vp, vp, i32, P(i32)]),
        "pa_alloc_slots_n": (i32, [vp, i32, vp, vp, vp, vp, i32, P(i32)]),
        "pa_get_block_tables": (i32, [vp, i32, vp, i32, vp, vp]),
        "pa_decode_step_prepare": (i32, [vp, i32, vp, i32, vp, vp, vp, vp, i32, P(i32)]),
        "pa_decode_step_prepare_rows": (i32, [vp, i32, vp, i32, vp, vp, vp, vp, vp, i32, P(i32)]),
        "pa_seq_info": (i32, [vp, i32, P(i32), P(i32)]),
        "pa_pool_num_free": (i32, [vp, P(i32)]),
        "pa_pool_free_queue": (i32, [vp, vp, i32, P(i32)]),
        "pa_pool_refcounts": (i32, [vp, vp]),
        "pa_write_kv": (i32, [vp, vp, vp, i32, vp, vp, P(pa_pool_desc), vp, vp]),
        "pa_copy_blocks": (i32, [vp, vp, i32, vp, i32, P(pa_pool_desc), vp, vp]),
        "pa_decode_workspace_bytes": (sz, [i32, i32, P(pa_pool_desc)]),
        "pa_decode_attention": (i32, [vp, vp, vp, vp, vp, vp, i32, i32, ctypes.c_float, vp, sz,
                                      vp, P(pa_pool_desc), vp]),
        "pa_decode_step_attention": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32,
                                           ctypes.c_float, vp, sz, vp, P(pa_pool_desc), vp]),
        "pa_decode_attention_noalloc": (i32, [vp, vp, vp, vp, vp, vp, i32, i32, ctypes.c_float,
                                              vp, P(pa_pool_desc), vp]),
        "pa_prefill_attention": (i32, [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                       ctypes.c_float, vp, P(pa_pool_desc), vp]),
        "pa_prefill_step_attention": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32,
                                            i32, ctypes.c_float, vp, P(pa_pool_desc), vp]),
        "pa_seq_truncate": (i32, [vp, i32, vp, vp]),
        "pa_seq_compact": (i32, [vp, i32, vp, vp, i32, vp, vp, vp]),
        "pa_tree_workspace_bytes": (sz, [i32, i32, i32, P(pa_pool_desc)]),
        "pa_tree_attention": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                    ctypes.c_float, vp, sz, vp, P(pa_pool_desc), vp]),
        "pa_verify_draft": (i32, [vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                  vp, vp]),
        "pa_decode_weights_workspace_bytes": (sz, [i32, i32, P(pa_pool_desc)]),
        "pa_decode_attention_weights": (i32, [vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, i32,
                                              ctypes.c_float, vp, sz, vp, P(pa_pool_desc), vp]),
        "pa_evict_select": (i32, [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, vp, vp]),
        "pa_compact_kv": (i32, [vp, vp, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                P(pa_pool_desc), vp, vp]),
        "pa_kv_block_bytes": (sz, [P(pa_pool_desc)]),
        "pa_write_kv_quant": (i32, [vp, vp, i32, i64, i64, vp, i32, vp, vp, P(pa_pool_desc), vp, vp]),
        "pa_read_kv_quant": (i32, [vp, vp, i32, vp, vp, i32, i32, vp, vp, P(pa_pool_desc), vp, vp]),
        "pa_decode_quant_workspace_bytes": (sz, [i32, i32, P(pa_pool_desc)]),
        "pa_decode_attention_quant": (i32, [vp, vp, i32, i32, vp, vp, vp, vp, i32, i32,
                                            ctypes.c_float, vp, sz, vp, P(pa_pool_desc), vp]),
        "pa_norm_rope": (i32, [vp, vp, vp, vp, i32, i64, i64, vp, vp, ctypes.c_float, vp, i32, i32,
                               i32, vp, i32, i32, i32, i32, vp, vp]),
        "pa_norm_rope_write_kv": (i32, [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, ctypes.c_float,
                                        vp, i32, i32, i32, vp, vp, i32, i32, vp, vp,
                                        P(pa_pool_desc), vp, vp]),
        "pa_selftest_bounded_wait": (i32, [vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
LIB_PATH = _LIB_PATH


def pa_last_error_string() -> str:
    return _lib.pa_last_error_string().decode()


def _check(rc: int):
    if rc != PA_OK:
        msg = pa_last_error_string()
        if rc == PA_ERR_OUT_OF_BLOCKS:
            raise OutOfBlocks(rc, msg)
        raise PagedKVError(rc, msg)


def _need_elems(n_elems: int, **tensors):
    """Refuses a tensor holding fewer elements than the call reads from it, and
    a raw address, whose length is not known (None is left to the library, which
    refuses a NULL it needs)."""
    for name, t in tensors.items():
        if isinstance(t, int):
            raise ValueError(f"{name} is an address, a tensor of {n_elems} elements is read")
        if t is not None and t.numel() < n_elems:
            raise ValueError(f"{name} holds {t.numel()} elements, the call reads {n_elems}")


def _host_i32(a):
    return np.ascontiguousarray(a, dtype=np.int32)


def _dev(x):
    """Device address of a CUDA tensor (or an int address / None)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return x.data_ptr()


def _addr(x):
    """Device-reachable address of a CUDA tensor or of a pinned host tensor."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if not (x.is_cuda or x.is_pinned()):
        raise ValueError("expected a CUDA tensor or a pinned host tensor")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class PoolDesc:
    """Holds a pa_pool_desc (and keeps its free_order array alive).  ``dtype`` is
    the cache's: PA_DTYPE_F16, or PA_DTYPE_I8 or PA_DTYPE_I4 for a quantised one."""

    def __init__(self, num_blocks, block_size, num_layers=1, num_heads=1, head_dim=8,
                 partition_tokens=0, free_order=None, flags=0, dtype=PA_DTYPE_F16):
        self._free = None if free_order is None else _host_i32(free_order)
        self.c = pa_pool_desc(int(num_blocks), int(block_size), int(num_layers), int(num_heads),
                              int(head_dim), int(dtype), int(partition_tokens), int(flags),
                              None if self._free is None else
                              self._free.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))

        self.ref = ctypes.byref(self.c)

    def __getattr__(self, name):
        return getattr(self.__dict__["c"], name)


# ---------------------------------------------------------------- host calls
def pa_pool_create(desc: PoolDesc):
    h = ctypes.c_void_p()
    _check(_lib.pa_pool_create(desc.ref, ctypes.byref(h)))
    return h


def pa_pool_destroy(pool) -> None:
    _check(_lib.pa_pool_destroy(pool))


def pa_seq_add(pool, seq_id: int, n_tokens: int, want_slots: bool = True):
    slots = np.empty(max(int(n_tokens), 0), np.int64) if want_slots else None
    _check(_lib.pa_seq_add(pool, int(seq_id), int(n_tokens),
                           None if slots is None else slots.ctypes.data))
    return slots


def pa_seq_add_tokens(pool, seq_id: int, token_ids, extra_key: int = 0, want_slots: bool = True):
    """Returns (slots int64[n] or None, n_cached_tokens)."""
    toks = _host_i32(token_ids)
    n = int(toks.shape[0])
    slots = np.empty(n, np.int64) if want_slots else None
    nc = ctypes.c_int32(0)
    _check(_lib.pa_seq_add_tokens(pool, int(seq_id), n, toks.ctypes.data if n else None,
                                  int(extra_key), None if slots is None else slots.ctypes.data,
                                  ctypes.byref(nc)))
    return slots, nc.value


def pa_pool_cached_blocks(pool) -> int:
    n = ctypes.c_int32()
    _check(_lib.pa_pool_cached_blocks(pool, ctypes.byref(n)))
    return n.value


def _group_move(fn, src_pool, dst_pool, seq_ids):
    ids = _host_i32(seq_ids)
    cap = 0
    # room for every distinct block: at most the sum of the tables' lengths
    for s in ids.tolist():
        cap += pa_seq_info(src_pool, s)[1]
    pairs = np.empty((max(cap, 1), 2), np.int32)
    n = ctypes.c_int32(0)
    _check(fn(src_pool, dst_pool, ids.shape[0], ids.ctypes.data, pairs.ctypes.data, cap,
              ctypes.byref(n)))
    return pairs[: n.value]


def pa_swap_out(gpu_pool, cpu_pool, seq_ids):
    """Move a sequence group to the CPU pool; returns the (gpu, cpu) block pairs."""
    return _group_move(_lib.pa_swap_out, gpu_pool, cpu_pool, seq_ids)


def pa_swap_in(cpu_pool, gpu_pool, seq_ids):
    """Move a sequence group back to the GPU pool; returns the (cpu, gpu) block pairs."""
    return _group_move(_lib.pa_swap_in, cpu_pool, gpu_pool, seq_ids)


def pa_swap_blocks(src_k, src_v, src_num_blocks, dst_k, dst_v, dst_num_blocks, pairs,
                   desc: PoolDesc, status=None, stream=None, n_pairs: int | None = None) -> None:
    L = len(src_k)
    arr = lambda xs: (ctypes.c_void_p * L)(*[_addr(x) for x in xs])
    n = int(pairs.shape[0]) if n_pairs is None else int(n_pairs)
    _check(_lib.pa_swap_blocks(arr(src_k), arr(src_v), int(src_num_blocks), arr(dst_k),
                               arr(dst_v), int(dst_num_blocks), L, _addr(pairs), n, desc.ref,
                               _dev(status), _stream(stream)))


def pa_seq_fork(pool, parent: int, child: int) -> None:
    _check(_lib.pa_seq_fork(pool, int(parent), int(child)))


def pa_seq_fork_batch(pool, parents, children) -> None:
    p, c = _host_i32(parents), _host_i32(children)
    if p.shape != c.shape:
        raise ValueError("parents and children differ in length")
    _check(_lib.pa_seq_fork_batch(pool, p.shape[0], p.ctypes.data, c.ctypes.data))


def pa_seq_free_batch(pool, seq_ids) -> None:
    ids = _host_i32(seq_ids)
    _check(_lib.pa_seq_free_batch(pool, ids.shape[0], ids.ctypes.data))


def pa_beam_prune(pool, beams, counts, next_id: int) -> int:
    """beams: int32 [groups, width] (contiguous, updated in place); counts:
    int32 [groups, width], each row summing to width.  Returns the new next_id."""
    if beams.dtype != np.int32 or not beams.flags.c_contiguous or beams.ndim != 2:
        raise ValueError("beams must be a contiguous int32 [groups, width] array")
    cnt = _host_i32(counts)
    if cnt.shape != beams.shape:
        raise ValueError("counts and beams differ in shape")
    nid = ctypes.c_int32(int(next_id))
    _check(_lib.pa_beam_prune(pool, beams.shape[0], beams.shape[1], beams.ctypes.data,
                              cnt.ctypes.data, ctypes.byref(nid)))
    return nid.value


def pa_seq_free(pool, seq_id: int) -> None:
    _check(_lib.pa_seq_free(pool, int(seq_id)))


def pa_alloc_slots(pool, seq_ids, copies_cap: int | None = None, slot_out=None, copies_out=None):
    """Returns (slot_mapping int64[n], copies int32[n_copies, 2])."""
    ids = _host_i32(seq_ids)
    n = ids.shape[0]
    cap = n if copies_cap is None else int(copies_cap)
    slots = np.empty(n, np.int64) if slot_out is None else slot_out
    copies = np.empty((max(cap, 1), 2), np.int32) if copies_out is None else copies_out
    nc = ctypes.c_int32(0)
    _check(_lib.pa_alloc_slots(pool, n, ids.ctypes.data, slots.ctypes.data, copies.ctypes.data,
                               cap, ctypes.byref(nc)))
    return slots, copies[: nc.value]


def pa_alloc_slots_n(pool, seq_ids, counts, copies_cap: int | None = None):
    """counts[i] new tokens for seq_ids[i]; returns (slot_mapping int64[sum], copies)."""
    ids, cnt = _host_i32(seq_ids), _host_i32(counts)
    if ids.shape != cnt.shape:
        raise ValueError("seq_ids and counts differ in length")
    n = ids.shape[0]
    cap = n if copies_cap is None else int(copies_cap)
    slots = np.empty(max(int(cnt.sum()), 1), np.int64)
    copies = np.empty((max(cap, 1), 2), np.int32)
    nc = ctypes.c_int32(0)
    _check(_lib.pa_alloc_slots_n(pool, n, ids.ctypes.data, cnt.ctypes.data, slots.ctypes.data,
                                 copies.ctypes.data, cap, ctypes.byref(nc)))
    return slots[: int(cnt.sum())], copies[: nc.value]


def pa_get_block_tables(pool, seq_ids, max_blocks: int, tables_out=None, ctx_out=None):
    """Returns (tables int32[n, max_blocks] padded with -1, ctx_lens int32[n])."""
    ids = _host_i32(seq_ids)
    n = ids.shape[0]
    tables = np.empty((n, max_blocks), np.int32) if tables_out is None else tables_out
    ctx = np.empty(n, np.int32) if ctx_out is None else ctx_out
    _check(_lib.pa_get_block_tables(pool, n, ids.ctypes.data, int(max_blocks),
                                    tables.ctypes.data, ctx.ctypes.data))
    return tables, ctx


def pa_decode_step_prepare(pool, seq_ids, max_blocks: int, slot_out=None, ctx_out=None,
                           tables_out=None, copies_out=None, copies_cap: int | None = None):
    """One token appended to every sequence, then the batch's tables.
    Returns (slot_mapping int64[n], ctx_lens int32[n], tables int32[n, max_blocks],
    copies int32[n_copies, 2]); the *_out arrays (e.g. views of a pinned
    staging buffer) are written in place when given."""
    ids = _host_i32(seq_ids)
    n = ids.shape[0]
    cap = n if copies_cap is None else int(copies_cap)
    slots = np.empty(n, np.int64) if slot_out is None else slot_out
    ctx = np.empty(n, np.int32) if ctx_out is None else ctx_out
    tables = np.empty((n, max_blocks), np.int32) if tables_out is None else tables_out
    copies = np.empty((max(cap, 1), 2), np.int32) if copies_out is None else copies_out
    nc = ctypes.c_int32(0)
    _check(_lib.pa_decode_step_prepare(pool, n, ids.ctypes.data, int(max_blocks),
                                       slots.ctypes.data, ctx.ctypes.data, tables.ctypes.data,
                                       copies.ctypes.data, cap, ctypes.byref(nc)))
    return slots, ctx, tables, copies[: nc.value]


def pa_decode_step_prepare_rows(pool, seq_ids, max_blocks: int, tables, row_versions,
                                slot_out=None, ctx_out=None, copies_out=None,
                                copies_cap: int | None = None):
    """pa_decode_step_prepare into a ``tables`` array (int32[n, max_blocks])
    that the caller keeps from step to step, with its ``row_versions``
    (uint64[n], zeros at first): only rows whose sequence's table changed are
    rewritten.  Returns (slot_mapping, ctx_lens, tables, copies)."""
    ids = _host_i32(seq_ids)
    n = ids.shape[0]
    if tables.dtype != np.int32 or tables.shape != (n, max_blocks) or not tables.flags.c_contiguous:
        raise ValueError("tables must be a contiguous int32 array of shape (n, max_blocks)")
    if row_versions.dtype != np.uint64 or row_versions.shape != (n,) or \
            not row_versions.flags.c_contiguous:
        raise ValueError("row_versions must be a contiguous uint64 array of length n")
    cap = n if copies_cap is None else int(copies_cap)
    slots = np.empty(n, np.int64) if slot_out is None else slot_out
    ctx = np.empty(n, np.int32) if ctx_out is None else ctx_out
    copies = np.empty((max(cap, 1), 2), np.int32) if copies_out is None else copies_out
    nc = ctypes.c_int32(0)
    _check(_lib.pa_decode_step_prepare_rows(pool, n, ids.ctypes.data, int(max_blocks),
                                            slots.ctypes.data, ctx.ctypes.data, tables.ctypes.data,
                                            row_versions.ctypes.data, copies.ctypes.data, cap,
                                            ctypes.byref(nc)))
    return slots, ctx, tables, copies[: nc.value]


def pa_decode_step_prepare_into(pool, n_seqs: int, ids_addr: int, max_blocks: int,
                                slots_addr: int, ctx_addr: int, tables_addr: int,
                                copies_addr: int, copies_cap: int, n_copies) -> int:
    """pa_decode_step_prepare on raw host addresses (a serving loop's
    preallocated staging buffers); ``n_copies`` is a ctypes.c_int32 that
    receives the copy count.  Returns it."""
    _check(_lib.pa_decode_step_prepare(pool, n_seqs, ids_addr, max_blocks, slots_addr, ctx_addr,
                                       tables_addr, copies_addr, copies_cap, ctypes.byref(n_copies)))
    return n_copies.value


def pa_decode_step_prepare_rows_into(pool, n_seqs: int, ids_addr: int, max_blocks: int,
                                     slots_addr: int, ctx_addr: int, tables_addr: int,
                                     versions_addr: int, copies_addr: int, copies_cap: int,
                                     n_copies) -> int:
    """pa_decode_step_prepare_rows on raw host addresses: table rows whose
    sequence's table is unchanged since this call last wrote them (per the
    caller's ``versions_addr`` array, one uint64 per row) are left as they
    are.  ``n_copies`` is a ctypes.c_int32 that receives the copy count."""
    _check(_lib.pa_decode_step_prepare_rows(pool, n_seqs, ids_addr, max_blocks, slots_addr,
                                            ctx_addr, tables_addr, versions_addr, copies_addr,
                                            copies_cap, ctypes.byref(n_copies)))
    return n_copies.value


def pa_seq_info(pool, seq_id: int):
    nt, nb = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.pa_seq_info(pool, int(seq_id), ctypes.byref(nt), ctypes.byref(nb)))
    return nt.value, nb.value


def pa_pool_num_free(pool) -> int:
    n = ctypes.c_int32()
    _check(_lib.pa_pool_num_free(pool, ctypes.byref(n)))
    return n.value


def pa_pool_free_queue(pool, num_blocks: int):
    out = np.empty(max(int(num_blocks), 1), np.int32)
    n = ctypes.c_int32()
    _check(_lib.pa_pool_free_queue(pool, out.ctypes.data, int(num_blocks), ctypes.byref(n)))
    return out[: n.value]


def pa_pool_refcounts(pool, num_blocks: int):
    out = np.empty(max(int(num_blocks), 1), np.int32)
    _check(_lib.pa_pool_refcounts(pool, out.ctypes.data))
    return out[: int(num_blocks)]


def pa_seq_truncate(pool, seq_ids, new_lens) -> None:
    """Each sequence keeps its first new_lens[i] tokens; blocks past them are released."""
    ids, lens = _host_i32(seq_ids), _host_i32(new_lens)
    if ids.shape != lens.shape:
        raise ValueError("seq_ids and new_lens differ in length")
    _check(_lib.pa_seq_truncate(pool, ids.shape[0], ids.ctypes.data, lens.ctypes.data))


def pa_seq_compact(pool, seq_ids, new_lens, max_blocks: int):
    """Shrinks the sequences to new_lens tokens whose rows pa_compact_kv moves to
    their front.  Returns (src_tables int32[n, max_blocks], src_lens int32[n],
    dst_tables int32[n, max_blocks]), tables padded with -1."""
    ids, lens = _host_i32(seq_ids), _host_i32(new_lens)
    if ids.shape != lens.shape:
        raise ValueError("seq_ids and new_lens differ in length")
    n = ids.shape[0]
    src, dst = np.empty((n, max_blocks), np.int32), np.empty((n, max_blocks), np.int32)
    src_lens = np.empty(n, np.int32)
    _check(_lib.pa_seq_compact(pool, n, ids.ctypes.data, lens.ctypes.data, int(max_blocks),
                               src.ctypes.data, src_lens.ctypes.data, dst.ctypes.data))
    return src, src_lens, dst


# -------------------------------------------------------------- device calls
def pa_write_kv(k, v, slot_mapping, k_cache, v_cache, desc: PoolDesc, status=None,
                stream=None, n_tokens: int | None = None) -> None:
    n = int(slot_mapping.shape[0]) if n_tokens is None else int(n_tokens)
    _check(_lib.pa_write_kv(_dev(k), _dev(v), _dev(slot_mapping), n, _dev(k_cache),
                            _dev(v_cache), desc.ref, _dev(status), _stream(stream)))


def pa_copy_blocks(k_caches, v_caches, pairs, desc: PoolDesc, status=None, stream=None,
                   n_pairs: int | None = None) -> None:
    L = len(k_caches)
    kp = (ctypes.c_void_p * L)(*[_dev(x) for x in k_caches])
    vp = (ctypes.c_void_p * L)(*[_dev(x) for x in v_caches])
    n = int(pairs.shape[0]) if n_pairs is None else int(n_pairs)
    _check(_lib.pa_copy_blocks(kp, vp, L, _dev(pairs), n, desc.ref, _dev(status),
                               _stream(stream)))


def pa_decode_workspace_bytes(n_seqs: int, max_blocks: int, desc: PoolDesc) -> int:
    return int(_lib.pa_decode_workspace_bytes(int(n_seqs), int(max_blocks), desc.ref))


def pa_decode_attention(out, q, k_cache, v_cache, block_tables, ctx_lens, scale: float,
                        desc: PoolDesc, workspace=None, status=None, stream=None,
                        n_seqs: int | None = None, max_blocks: int | None = None) -> None:
    n = int(q.shape[0]) if n_seqs is None else int(n_seqs)
    mb = int(block_tables.shape[1]) if max_blocks is None else int(max_blocks)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.pa_decode_attention(_dev(out), _dev(q), _dev(k_cache), _dev(v_cache),
                                    _dev(block_tables), _dev(ctx_lens), n, mb,
                                    ctypes.c_float(scale), _dev(workspace), ws_bytes,
                                    _dev(status), desc.ref, _stream(stream)))


def pa_decode_step_attention(out, q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables,
                             ctx_lens, scale: float, desc: PoolDesc, workspace=None, status=None,
                             stream=None, n_seqs: int | None = None,
                             max_blocks: int | None = None) -> None:
    """The step's slot write (one new token per sequence, at slot_mapping[s])
    and decode attention in one call."""
    n = int(q.shape[0]) if n_seqs is None else int(n_seqs)
    mb = int(block_tables.shape[1]) if max_blocks is None else int(max_blocks)
    _need_elems(n * desc.num_heads * desc.head_dim, k_new=k_new, v_new=v_new)
    _need_elems(n, slot_mapping=slot_mapping)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.pa_decode_step_attention(_dev(out), _dev(q), _dev(k_new), _dev(v_new),
                                         _dev(slot_mapping), _dev(k_cache), _dev(v_cache),
                                         _dev(block_tables), _dev(ctx_lens), n, mb,
                                         ctypes.c_float(scale), _dev(workspace), ws_bytes,
                                         _dev(status), desc.ref, _stream(stream)))


def pa_prefill_attention(out, q, k_cache, v_cache, block_tables, ctx_lens, q_starts,
                         scale: float, desc: PoolDesc, max_q_len: int, status=None, stream=None,
                         n_seqs: int | None = None, max_blocks: int | None = None,
                         q_rows: int | None = None) -> None:
    """Causal paged prefill: rows q_starts[s]..q_starts[s+1]-1 of q are the last
    positions of sequence s's context of ctx_lens[s] tokens.  ``max_q_len``
    (host int) bounds every q_len; ``q_rows`` defaults to the rows of q and out."""
    n = int(ctx_lens.shape[0]) if n_seqs is None else int(n_seqs)
    mb = int(block_tables.shape[1]) if max_blocks is None else int(max_blocks)
    rows = min(int(q.shape[0]), int(out.shape[0])) if q_rows is None else int(q_rows)
    _check(_lib.pa_prefill_attention(_dev(out), _dev(q), _dev(k_cache), _dev(v_cache),
                                     _dev(block_tables), _dev(ctx_lens), _dev(q_starts), n, mb,
                                     int(max_q_len), rows, ctypes.c_float(scale), _dev(status),
                                     desc.ref, _stream(stream)))


def pa_prefill_step_attention(out, q, k_new, v_new, k_cache, v_cache, block_tables, ctx_lens,
                              q_starts, scale: float, desc: PoolDesc, max_q_len: int, status=None,
                              stream=None, n_seqs: int | None = None, max_blocks: int | None = None,
                              q_rows: int | None = None) -> None:
    """Whole prompts: their keys and values (k_new, v_new, rows as q) stored
    into their blocks and causal prefill attention over them, one call."""
    n = int(ctx_lens.shape[0]) if n_seqs is None else int(n_seqs)
    mb = int(block_tables.shape[1]) if max_blocks is None else int(max_blocks)
    rows = min(int(q.shape[0]), int(out.shape[0])) if q_rows is None else int(q_rows)
    # the new rows are read as [rows][num_heads][head_dim] tensors, like q
    _need_elems(rows * desc.num_heads * desc.head_dim, k_new=k_new, v_new=v_new)
    _check(_lib.pa_prefill_step_attention(_dev(out), _dev(q), _dev(k_new), _dev(v_new),
                                          _dev(k_cache), _dev(v_cache), _dev(block_tables),
                                          _dev(ctx_lens), _dev(q_starts), n, mb, int(max_q_len),
                                          rows, ctypes.c_float(scale), _dev(status), desc.ref,
                                          _stream(stream)))


# The calls below take microseconds on the GPU, so their arguments are checked
# with as few Python operations as will do.
_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _here(torch):
    """Index of the current GPU, where the calls' kernels run (before CUDA is in
    use: -2, no tensor's)."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2


def _arg(name, t, dtype, n, here):
    """Device address of a contiguous tensor of dtype on the current GPU with n
    elements or more (a raw address or None as it is)."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is not dtype or t.get_device() != here or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name}: a contiguous tensor of {n} or more {dtype} on the current GPU "
                         f"is read, not {tuple(t.shape)} {t.dtype} on {t.device}"
                         f"{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


def _raw_stream(torch, stream, here=None):
    """Address of a stream; None is the current one (of the current GPU, ``here``)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if here is None else here)
    return stream if stream.__class__ is int else stream.cuda_stream


def _workspace(ws, here):
    """Device address and bytes of a contiguous tensor of any type on the current
    GPU (None is left to the library, which refuses it)."""
    if ws is None:
        return None, 0
    if ws.__class__ is int:
        raise ValueError("workspace: an address, whose size is not known")
    if ws.get_device() != here or not ws.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on the current GPU is used, not "
                         f"{tuple(ws.shape)} on {ws.device}"
                         f"{'' if ws.is_contiguous() else ', not contiguous'}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def pa_tree_workspace_bytes(n_seqs: int, max_blocks: int, max_q_len: int, desc: PoolDesc) -> int:
    return int(_lib.pa_tree_workspace_bytes(int(n_seqs), int(max_blocks), int(max_q_len), desc.ref))


def pa_tree_attention(out, q, k_cache, v_cache, block_tables, ctx_lens, q_starts, parents,
                      scale: float, desc: PoolDesc, max_q_len: int, workspace=None, status=None,
                      stream=None, n_seqs: int | None = None, max_blocks: int | None = None,
                      q_rows: int | None = None) -> None:
    """Attention of drafted nodes: rows q_starts[s]..q_starts[s+1]-1 of q are
    the last positions of sequence s, each seeing the positions before the
    nodes, itself and its ancestors by ``parents`` (None: a chain)."""
    torch = _torch or _load_torch()
    here = _here(torch)
    f16, i32 = torch.float16, torch.int32
    n = ctx_lens.shape[0] if n_seqs is None else int(n_seqs)
    mb = block_tables.shape[1] if max_blocks is None else int(max_blocks)
    rows = min(q.shape[0], out.shape[0]) if q_rows is None else int(q_rows)
    c = desc.c
    width = c.num_heads * c.head_dim
    cache = c.num_blocks * c.block_size * width
    _check(_lib.pa_tree_attention(
        _arg("out", out, f16, rows * width, here), _arg("q", q, f16, rows * width, here),
        _arg("k_cache", k_cache, f16, cache, here), _arg("v_cache", v_cache, f16, cache, here),
        _arg("block_tables", block_tables, i32, n * mb, here),
        _arg("ctx_lens", ctx_lens, i32, n, here), _arg("q_starts", q_starts, i32, n + 1, here),
        _arg("parents", parents, i32, rows, here), n, mb, max_q_len, rows, scale,
        *_workspace(workspace, here), _arg("status", status, i32, 1, here), desc.ref,
        _raw_stream(torch, stream)))


def pa_verify_draft(path, path_lens, next_tokens, target_probs, draft_probs, draft_tokens,
                    parents, q_starts, u_accept, u_sample, max_q_len: int | None = None,
                    status=None, stream=None, n_seqs: int | None = None) -> None:
    """Accepted path, its length and the next token of every sequence from the
    target's and the drafter's probabilities ([rows, vocab] float32, float16 or
    bfloat16; draft_probs None: tokens picked outright) and given uniform
    numbers.  ``path`` is int32 [n_seqs, max_q_len]."""
    torch = _torch or _load_torch()
    here = _here(torch)
    f32, i32 = torch.float32, torch.int32
    n = u_sample.shape[0] if n_seqs is None else int(n_seqs)
    mq = path.shape[1] if max_q_len is None else int(max_q_len)
    rows, vocab = target_probs.shape
    kind = target_probs.dtype
    code = (PA_DTYPE_F32 if kind is f32 else PA_DTYPE_F16 if kind is torch.float16 else
            PA_DTYPE_BF16 if kind is torch.bfloat16 else -1)
    if code < 0:
        raise ValueError(f"target_probs is {kind}: float32, float16 or bfloat16 expected")
    if draft_probs is not None and draft_probs.shape[1] != vocab:
        raise ValueError("target_probs and draft_probs differ in width")
    if path.shape[1] != mq:
        raise ValueError(f"path is {path.shape[1]} wide, max_q_len {mq}")
    _check(_lib.pa_verify_draft(
        _arg("path", path, i32, n * mq, here), _arg("path_lens", path_lens, i32, n, here),
        _arg("next_tokens", next_tokens, i32, n, here),
        _arg("target_probs", target_probs, kind, 0, here),
        _arg("draft_probs", draft_probs, kind, rows * vocab, here), code,
        _arg("draft_tokens", draft_tokens, i32, rows, here),
        _arg("parents", parents, i32, rows, here), _arg("q_starts", q_starts, i32, n + 1, here),
        _arg("u_accept", u_accept, f32, rows, here), _arg("u_sample", u_sample, f32, n, here), n,
        mq, rows, vocab, _arg("status", status, i32, 1, here), _raw_stream(torch, stream)))


def pa_decode_weights_workspace_bytes(n_seqs: int, max_blocks: int, desc: PoolDesc) -> int:
    return int(_lib.pa_decode_weights_workspace_bytes(int(n_seqs), int(max_blocks), desc.ref))


def pa_decode_attention_weights(out, weights_out, weights_in, q, k_cache, v_cache, block_tables,
                                ctx_lens, scale: float, desc: PoolDesc, workspace=None,
                                status=None, stream=None, n_seqs: int | None = None,
                                max_blocks: int | None = None) -> None:
    """pa_decode_attention that adds each position's weight to weights_in
    (float32 [n_seqs, num_heads, weight_len], None: zeros) into weights_out,
    which may be the same tensor."""
    torch = _torch or _load_torch()
    here = _here(torch)
    f16, f32, i32 = torch.float16, torch.float32, torch.int32
    n = q.shape[0] if n_seqs is None else int(n_seqs)
    mb = block_tables.shape[1] if max_blocks is None else int(max_blocks)
    wl = weights_out.shape[-1]
    if weights_in is not None and weights_in.shape[-1] != wl:
        raise ValueError("weights_in and weights_out differ in length")
    c = desc.c
    if weights_out.shape[-2] != c.num_heads:
        raise ValueError(f"weights_out has {weights_out.shape[-2]} heads, the cache {c.num_heads}")
    width = c.num_heads * c.head_dim
    cache, sums = c.num_blocks * c.block_size * width, n * c.num_heads * wl
    _check(_lib.pa_decode_attention_weights(
        _arg("out", out, f16, n * width, here), _arg("weights_out", weights_out, f32, sums, here),
        _arg("weights_in", weights_in, f32, sums, here), wl, _arg("q", q, f16, n * width, here),
        _arg("k_cache", k_cache, f16, cache, here), _arg("v_cache", v_cache, f16, cache, here),
        _arg("block_tables", block_tables, i32, n * mb, here),
        _arg("ctx_lens", ctx_lens, i32, n, here), n, mb, scale, *_workspace(workspace, here),
        _arg("status", status, i32, 1, here), desc.ref, _raw_stream(torch, stream)))


def pa_evict_select(keep, keep_lens, weights_out, weights_in, ctx_lens, budget: int, recent: int,
                    status=None, stream=None, n_seqs: int | None = None) -> None:
    """Positions that stay, per (sequence, head): the last ``recent`` and those
    with the largest weights_in, ``budget`` in all, into keep (int32
    [n_seqs, num_heads, budget], ascending, padded with -1); their weights into
    weights_out, which may be weights_in."""
    torch = _torch or _load_torch()
    here = _here(torch)
    f32, i32 = torch.float32, torch.int32
    n = ctx_lens.shape[0] if n_seqs is None else int(n_seqs)
    _, heads, wl = weights_in.shape
    if weights_out.shape[1:] != weights_in.shape[1:]:
        raise ValueError("weights_in and weights_out differ in shape")
    if keep.shape[-1] != budget or keep.shape[-2] != heads:
        raise ValueError(f"keep is {tuple(keep.shape)}: {heads} heads, {budget} entries expected")
    sums = n * heads * wl
    _check(_lib.pa_evict_select(
        _arg("keep", keep, i32, n * heads * budget, here),
        _arg("keep_lens", keep_lens, i32, n, here),
        _arg("weights_out", weights_out, f32, sums, here),
        _arg("weights_in", weights_in, f32, sums, here), wl,
        _arg("ctx_lens", ctx_lens, i32, n, here), n, heads, budget, recent,
        _arg("status", status, i32, 1, here), _raw_stream(torch, stream)))


def pa_compact_kv(k_caches, v_caches, src_tables, dst_tables, src_lens, keep, keep_lens,
                  desc: PoolDesc, first=None, status=None, stream=None,
                  n_seqs: int | None = None) -> None:
    """Every layer's K/V rows at positions first + keep[s, h, j] (src_tables)
    move to first + j (dst_tables).  keep: int32 [n_seqs, 1 or num_heads, n]
    or [n_seqs, n] (one list for all heads)."""
    torch = _torch or _load_torch()
    here = _here(torch)
    f16, i32 = torch.float16, torch.int32
    L = len(k_caches)
    n = keep_lens.shape[0] if n_seqs is None else int(n_seqs)
    mb = src_tables.shape[1]
    heads = keep.shape[1] if keep.dim() == 3 else 1
    stride = keep.shape[-1]
    if len(v_caches) != L:
        raise ValueError("k_caches and v_caches differ in length")
    if dst_tables.shape[1] != mb:
        raise ValueError("src_tables and dst_tables differ in width")
    c = desc.c
    cache = c.num_blocks * c.block_size * c.num_heads * c.head_dim
    kp = (ctypes.c_void_p * L)(*[_arg("k_caches", x, f16, cache, here) for x in k_caches])
    vp = (ctypes.c_void_p * L)(*[_arg("v_caches", x, f16, cache, here) for x in v_caches])
    _check(_lib.pa_compact_kv(
        kp, vp, L, _arg("src_tables", src_tables, i32, n * mb, here),
        _arg("dst_tables", dst_tables, i32, n * mb, here), _arg("src_lens", src_lens, i32, n, here),
        _arg("first", first, i32, n, here), _arg("keep", keep, i32, n * heads * stride, here),
        _arg("keep_lens", keep_lens, i32, n, here), heads, stride, n, mb, desc.ref,
        _arg("status", status, i32, 1, here), _raw_stream(torch, stream)))


def pa_kv_block_bytes(desc: PoolDesc) -> int:
    """Bytes of one block of one layer's K (or V) cache, of any type (0: refused)."""
    return int(_lib.pa_kv_block_bytes(desc.ref))


def _kind(torch, name, t):
    """PA_DTYPE_F16 or PA_DTYPE_BF16 of a tensor of rows."""
    if t.dtype is torch.float16:
        return PA_DTYPE_F16
    if t.dtype is torch.bfloat16:
        return PA_DTYPE_BF16
    raise ValueError(f"{name} is {t.dtype}: float16 or bfloat16 expected")


def _cache_bytes(c):
    """Bytes of a layer's K (or V) cache of the pool that c (a pa_pool_desc) describes."""
    kind, dim = c.dtype, c.head_dim
    row = dim * 2 if kind == PA_DTYPE_F16 else (dim if kind == PA_DTYPE_I8 else dim // 2) + dim // 16
    return c.num_blocks * c.num_heads * c.block_size * row


def _rows(name, t, dtype, n, heads, dim, here):
    """Device address and row stride of [tokens, heads, dim] rows whose heads are
    contiguous (a slice of a packed projection, say)."""
    shape, strides = t.shape, t.stride()
    if t.dtype is not dtype or t.get_device() != here or len(shape) != 3 or shape[0] < n or \
            shape[1] != heads or shape[2] != dim or \
            ((strides[2] != 1 or strides[1] != dim and heads > 1) and n and heads):
        raise ValueError(f"{name}: {n} rows of {heads} heads of {dim} {dtype} on the current GPU are "
                         f"read, a token's next to one another, not {tuple(shape)} {t.dtype} with "
                         f"strides {strides} on {t.device}")
    return t.data_ptr(), strides[0] if n > 1 else heads * dim


def pa_write_kv_quant(k, v, slot_mapping, k_cache, v_cache, desc: PoolDesc, status=None, stream=None,
                      n_tokens: int | None = None) -> None:
    """pa_write_kv into a quantised cache (uint8, pa_kv_block_bytes(desc) a block);
    k and v: float16 or bfloat16 [tokens, heads, dim], a token's heads contiguous."""
    torch = _torch or _load_torch()
    here = _here(torch)
    n = slot_mapping.shape[0] if n_tokens is None else int(n_tokens)
    c, u8 = desc.c, torch.uint8
    cache = _cache_bytes(c)
    kind = _kind(torch, "k", k)
    kp, ks = _rows("k", k, k.dtype, n, c.num_heads, c.head_dim, here)
    vp, vs = _rows("v", v, k.dtype, n, c.num_heads, c.head_dim, here)
    _check(_lib.pa_write_kv_quant(
        kp, vp, kind, ks, vs, _arg("slot_mapping", slot_mapping, torch.int64, n, here), n,
        _arg("k_cache", k_cache, u8, cache, here), _arg("v_cache", v_cache, u8, cache, here), desc.ref,
        _arg("status", status, torch.int32, 1, here), _raw_stream(torch, stream, here)))


def pa_read_kv_quant(k, v, slot_mapping, k_cache, v_cache, desc: PoolDesc, out_slots=None, status=None,
                     stream=None, n_tokens: int | None = None) -> None:
    """Rows of a quantised cache read back into k and v: float16 or bfloat16 rows
    [tokens, heads, dim], or, with out_slots, float16 caches [blocks, heads, B, dim]."""
    torch = _torch or _load_torch()
    here = _here(torch)
    n = slot_mapping.shape[0] if n_tokens is None else int(n_tokens)
    c, u8, i64 = desc.c, torch.uint8, torch.int64
    width = c.num_heads * c.head_dim
    cache = _cache_bytes(c)
    kind = _kind(torch, "k", k)
    blocks, rows = 0, n
    if out_slots is not None:
        if tuple(k.shape[1:]) != (c.num_heads, c.block_size, c.head_dim):
            raise ValueError(f"k is {tuple(k.shape)}: blocks of {c.num_heads} heads, {c.block_size} "
                             f"tokens of {c.head_dim} expected")
        blocks = k.shape[0]
        rows = blocks * c.block_size
    elif tuple(k.shape[1:]) != (c.num_heads, c.head_dim):
        raise ValueError(f"k is {tuple(k.shape)}: rows of {c.num_heads} heads of {c.head_dim} expected")
    if v is not None and v.__class__ is not int and (v.shape[1:] != k.shape[1:] or v.shape[0] < blocks):
        raise ValueError(f"v is {tuple(v.shape)}: like k, {tuple(k.shape)}, expected")
    _check(_lib.pa_read_kv_quant(
        _arg("k", k, k.dtype, rows * width, here), _arg("v", v, k.dtype, rows * width, here), kind,
        _arg("slot_mapping", slot_mapping, i64, n, here), _arg("out_slots", out_slots, i64, n, here),
        blocks, n, _arg("k_cache", k_cache, u8, cache, here), _arg("v_cache", v_cache, u8, cache, here),
        desc.ref, _arg("status", status, torch.int32, 1, here), _raw_stream(torch, stream, here)))


def pa_decode_quant_workspace_bytes(n_seqs: int, q_heads: int, desc: PoolDesc) -> int:
    return int(_lib.pa_decode_quant_workspace_bytes(int(n_seqs), int(q_heads), desc.ref))


def pa_decode_attention_quant(out, q, k_cache, v_cache, block_tables, ctx_lens, scale: float,
                              desc: PoolDesc, workspace=None, status=None, stream=None,
                              n_seqs: int | None = None, max_blocks: int | None = None) -> None:
    """Decode attention over a quantised cache.  q and out: float16 or bfloat16
    [n_seqs, query heads, dim], the query heads a multiple of desc.num_heads."""
    torch = _torch or _load_torch()
    here = _here(torch)
    u8, i32 = torch.uint8, torch.int32
    n = q.shape[0] if n_seqs is None else int(n_seqs)
    mb = block_tables.shape[1] if max_blocks is None else int(max_blocks)
    c = desc.c
    shape = q.shape
    if len(shape) != 3 or shape[2] != c.head_dim:
        raise ValueError(f"q is {tuple(shape)}: [n_seqs, query heads, {c.head_dim}] expected")
    heads = shape[1]
    rows, cache = n * heads * c.head_dim, _cache_bytes(c)
    kind = _kind(torch, "q", q)
    _check(_lib.pa_decode_attention_quant(
        _arg("out", out, q.dtype, rows, here), _arg("q", q, q.dtype, rows, here), kind, heads,
        _arg("k_cache", k_cache, u8, cache, here), _arg("v_cache", v_cache, u8, cache, here),
        _arg("block_tables", block_tables, i32, n * mb, here),
        _arg("ctx_lens", ctx_lens, i32, n, here), n, mb, scale, *_workspace(workspace, here),
        _arg("status", status, i32, 1, here), desc.ref, _raw_stream(torch, stream, here)))


def _rotation(torch, here, dtype, dim, q_weight, k_weight, cos_sin, positions, n, rot_dim):
    """Addresses of the weights, the table and the positions, and the table's rows."""
    rows = 0
    if rot_dim and cos_sin is not None:
        shape = cos_sin.shape
        if len(shape) != 2 or shape[1] != rot_dim:
            raise ValueError(f"cos_sin is {tuple(shape)}: [positions, {rot_dim}] expected")
        rows = shape[0]
    return (_arg("q_weight", q_weight, dtype, dim, here), _arg("k_weight", k_weight, dtype, dim, here),
            _arg("cos_sin", cos_sin, torch.float32, 0, here), rows,
            _arg("positions", positions, torch.int32, n if rot_dim else 0, here))


def pa_norm_rope(q_out, k_out, q, k, q_weight, k_weight, eps: float, cos_sin, positions,
                 rot_dim: int | None = None, interleaved: bool = False, status=None, stream=None,
                 n_tokens: int | None = None) -> None:
    """Norm of every query and key head (weights None: none) and its rotation by
    position, rows [tokens, heads, dim] of float16 or bfloat16 in (a token's heads
    contiguous) and out.  cos_sin: float32 [positions, rot_dim], cosines then sines."""
    torch = _torch or _load_torch()
    here = _here(torch)
    n, hq, dim = q.shape
    if n_tokens is not None:
        n = int(n_tokens)
    hk = k.shape[1]
    rot = (0 if cos_sin is None else cos_sin.shape[1]) if rot_dim is None else int(rot_dim)
    kind = _kind(torch, "q", q)
    qp, qs = _rows("q", q, q.dtype, n, hq, dim, here)
    kp, ks = _rows("k", k, q.dtype, n, hk, dim, here)
    qw, kw, table, rows, pos = _rotation(torch, here, q.dtype, dim, q_weight, k_weight, cos_sin,
                                         positions, n, rot)
    _check(_lib.pa_norm_rope(
        _arg("q_out", q_out, q.dtype, n * hq * dim, here),
        _arg("k_out", k_out, q.dtype, n * hk * dim, here), qp, kp, kind, qs, ks, qw, kw, eps, table,
        rows, rot, int(interleaved), pos, n, hq, hk, dim, _arg("status", status, torch.int32, 1, here),
        _raw_stream(torch, stream, here)))


def pa_norm_rope_write_kv(q_out, q, k, v, q_weight, k_weight, eps: float, cos_sin, positions,
                          slot_mapping, k_cache, v_cache, desc: PoolDesc, rot_dim: int | None = None,
                          interleaved: bool = False, status=None, stream=None,
                          n_tokens: int | None = None) -> None:
    """pa_norm_rope with the keys and the values v written into their slots of the
    cache (float16, or uint8 where desc is a quantised one's)."""
    torch = _torch or _load_torch()
    here = _here(torch)
    n = slot_mapping.shape[0] if n_tokens is None else int(n_tokens)
    c = desc.c
    hq, hk, dim = q.shape[1], c.num_heads, c.head_dim
    rot = (0 if cos_sin is None else cos_sin.shape[1]) if rot_dim is None else int(rot_dim)
    kind = _kind(torch, "q", q)
    qp, qs = _rows("q", q, q.dtype, n, hq, dim, here)
    kp, ks = _rows("k", k, q.dtype, n, hk, dim, here)
    vp, vs = _rows("v", v, q.dtype, n, hk, dim, here)
    qw, kw, table, rows, pos = _rotation(torch, here, q.dtype, dim, q_weight, k_weight, cos_sin,
                                         positions, n, rot)
    plain = c.dtype == PA_DTYPE_F16
    cache = _cache_bytes(c) // (2 if plain else 1)
    t = torch.float16 if plain else torch.uint8
    _check(_lib.pa_norm_rope_write_kv(
        _arg("q_out", q_out, q.dtype, n * hq * dim, here), qp, kp, vp, kind, qs, ks, vs, qw, kw, eps,
        table, rows, rot, int(interleaved), pos,
        _arg("slot_mapping", slot_mapping, torch.int64, n, here), n, hq,
        _arg("k_cache", k_cache, t, cache, here), _arg("v_cache", v_cache, t, cache, here), desc.ref,
        _arg("status", status, torch.int32, 1, here), _raw_stream(torch, stream, here)))


def pa_selftest_bounded_wait(status, stream=None) -> None:
    """One thread waits, with the kernels' bounded wait, for an mbarrier phase
    that nothing completes; after the limit it writes PA_ERR_TIMEOUT into
    status (device int32)."""
    _check(_lib.pa_selftest_bounded_wait(_dev(status), _stream(stream)))


def pa_decode_attention_noalloc(out, q, k_cache, v_cache, block_tables, ctx_lens, scale: float,
                                desc: PoolDesc, status=None, stream=None,
                                n_seqs: int | None = None, max_blocks: int | None = None) -> None:
    """pa_decode_attention without a workspace argument, for callers that cannot
    allocate device memory when they run attention: the library's fixed
    scratch (PA_NOALLOC_SCRATCH_BYTES, shared by all calls) stands in for it.
    Calls that overlap on the GPU race on that scratch."""
    n = int(q.shape[0]) if n_seqs is None else int(n_seqs)
    mb = int(block_tables.shape[1]) if max_blocks is None else int(max_blocks)
    _check(_lib.pa_decode_attention_noalloc(_dev(out), _dev(q), _dev(k_cache), _dev(v_cache),
                                            _dev(block_tables), _dev(ctx_lens), n, mb,
                                            ctypes.c_float(scale), _dev(status), desc.ref,
                                            _stream(stream)))
