"""Paged KV cache and PagedAttention decode step for NVIDIA GB300 (sm_103a).

Thin Python binding over the C ABI of ``libpagedkv.so`` (include/pagedkv.h).
It only marshals arguments: the block ledger runs in the library's C++ code and
every device step runs in its CUDA kernels.  PyTorch supplies device memory and
streams.  If the library is not built, every call raises.

Typical decode step (the flow of "LLM 추론 배칭 전략 정리", section 5):

    pool = KVPool(num_blocks, num_kv_heads=8, head_dim=128, dtype="bf16", device="cuda")
    slots = pool.append_slots(seq_lens, num_new, tables)      # host: on-demand blocks
    d_tables.copy_(torch.from_numpy(tables)); d_slots.copy_(...)  # H2D hand-off
    cache_write(pool, k_new, v_new, d_slots, status)          # device: write new K/V
    paged_decode_attention(pool, q, d_tables, d_lens, scale, ws, status, out=out)
    pool.free(finished_blocks)                                # host: release

A model that rotates K and its queries by position, and attends to a window:

    table = rope_table(max_positions, rotary_dim, device="cuda")
    q = cache_write_rope(pool, k_new, v_new, d_positions, table, d_slots, status, q=q)
    paged_decode_attention_window(pool, q, d_tables, d_lens, scale, window, sinks, status)
"""
from __future__ import annotations

import ctypes

import numpy as np

from . import _native
from ._native import (DEV_BAD_BLOCK, DEV_BAD_LEN, DEV_BAD_POS, DEV_BAD_SLOT, DEV_TIMEOUT,
                      PKV_B8_BF16, PKV_B8_F16, PKV_BF16, PKV_F16, PKV_Q8_BF16, PKV_Q8_F16,
                      PagedKVError, check, lib)

__all__ = ["KVPool", "PagedKVError", "cache_write", "block_copy", "gather_blocks",
           "scatter_blocks", "paged_decode_attention", "CapturedDecode",
           "paged_decode_attention_noalloc", "paged_prefill_attention",
           "decode_plan", "decode_plan_bytes", "paged_decode_attention_planned",
           "cache_write_q8", "paged_decode_attention_q8",
           "cache_write_rope", "rope_table", "cache_write_b8", "dequantize_blocks",
           "paged_decode_attention_b8", "paged_decode_attention_window",
           "paged_prefill_attention_window",
           "prefill_workspace_bytes",
           "decode_workspace_bytes", "status_check", "kv_bytes_per_token",
           "kv_blocks_for_tokens", "kv_pool_bytes", "default_split", "lib",
           "DEV_BAD_SLOT", "DEV_BAD_BLOCK", "DEV_BAD_LEN", "DEV_TIMEOUT", "DEV_BAD_POS"]

_DTYPES = {"f16": PKV_F16, "fp16": PKV_F16, "float16": PKV_F16,
           "bf16": PKV_BF16, "bfloat16": PKV_BF16,
           "q8_bf16": PKV_Q8_BF16, "q8_f16": PKV_Q8_F16,
           "b8_bf16": PKV_B8_BF16, "b8_f16": PKV_B8_F16}
_NAMES = {PKV_F16: "f16", PKV_BF16: "bf16", PKV_Q8_BF16: "q8_bf16", PKV_Q8_F16: "q8_f16",
          PKV_B8_BF16: "b8_bf16", PKV_B8_F16: "b8_f16"}


def _np_ptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def _t_ptr(t):
    return ctypes.c_void_p(t.data_ptr() if t is not None else None)


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check_layout(contiguous: dict, int32: dict | None = None, int64: dict | None = None):
    """Tensors the C ABI reads as plain row-major arrays must be contiguous, and
    its index arrays of the stated integer type (a raise here launches nothing)."""
    import torch
    for name, t in contiguous.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for want, group in ((torch.int32, int32 or {}), (torch.int64, int64 or {})):
        for name, t in group.items():
            if t.dtype != want:
                raise TypeError(f"{name} must be {str(want).replace('torch.', '')}")


def _check_rows(name: str, t, rows, heads, head_dim: int, dtype, device) -> None:
    """``t`` must be a [rows][heads][head_dim] tensor of ``dtype`` on ``device``
    (``rows`` or ``heads`` None: any).  The library sizes every read and write of
    such an array from the pool's geometry and the counts it is given, so a
    tensor of another shape, type or device would be read or written past its
    end; a raise here launches nothing."""
    shape = tuple(t.shape)
    if (len(shape) != 3 or (rows is not None and shape[0] != rows)
            or (heads is not None and shape[1] != heads) or shape[2] != head_dim):
        want = f"[{'n' if rows is None else rows}][{'h' if heads is None else heads}][{head_dim}]"
        raise ValueError(f"{name} must be {want}, got {list(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}, got "
                        f"{str(t.dtype).replace('torch.', '')}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's rows are on {device}")


def _check_vector(name: str, t, n: int | None, device, ndim: int = 1) -> None:
    """An index array with ``n`` rows (None: any) on ``device``."""
    if t.dim() != ndim or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must have {ndim} dimension(s) and {n} rows, got "
                         f"{list(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's rows are on {device}")


def _check_device_call(q, status, workspace=None, pools=()) -> None:
    """Last check before a launch: every buffer the kernels touch sits on the
    same CUDA device (host tensors would hand the kernels host addresses)."""
    if q.device.type != "cuda":
        raise ValueError(f"the call's tensors must be CUDA tensors, got {q.device}")
    if status.dtype != _torch_int32() or status.numel() < 1:
        raise TypeError("status must be an int32 tensor of at least one element")
    for name, t in (("status", status), ("workspace", workspace)) + tuple(pools):
        if t is not None and t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, the call's rows are on {q.device}")


def _torch_int32():
    import torch
    return torch.int32


def _check_pool_tensor(name: str, t, pool: "KVPool") -> None:
    """A caller-supplied pool tensor must hold the pool's whole geometry."""
    if pool.record_bytes:
        want, dt = pool.num_blocks * pool.num_kv_heads * pool.record_bytes, None
    else:
        want = pool.num_blocks * pool.num_kv_heads * pool.block_size * pool.head_dim
        dt = _torch_dtype(pool.dtype_code)
    if t.numel() != want or (dt is not None and t.dtype != dt):
        raise ValueError(f"{name} does not match the pool's geometry and type")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_decode_args(pool: "KVPool", q, out, block_tables, context_lens, status,
                       workspace=None, k_pool=None, v_pool=None) -> None:
    """Shapes, types and devices of a decode call: q and out [S][Hq][D] in the
    pool's row type, block_tables [S][max_blocks], context_lens [S]."""
    import torch
    _check_layout({"q": q, "out": out, "block_tables": block_tables,
                   "context_lens": context_lens, "workspace": workspace},
                  int32={"block_tables": block_tables, "context_lens": context_lens})
    dt = _torch_dtype(pool.dtype_code)
    _check_rows("q", q, None, None, pool.head_dim, dt, None)
    S, hq = int(q.shape[0]), int(q.shape[1])
    if hq % pool.num_kv_heads:
        raise ValueError(f"q has {hq} heads, not a multiple of the pool's "
                         f"{pool.num_kv_heads} kv heads")
    _check_rows("out", out, S, hq, pool.head_dim, dt, q.device)
    _check_vector("block_tables", block_tables, S, q.device, ndim=2)
    _check_vector("context_lens", context_lens, S, q.device)
    if workspace is not None and workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    pools = []
    for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
        if t is not None:
            _check_pool_tensor(name, t, pool)
            pools.append((name, t))
    _check_device_call(q, status, workspace, pools)


def _torch_dtype(code: int):
    """Element type of K/V rows and queries for a pool type (8-bit pools take
    bf16 / fp16 rows and quantise them)."""
    import torch
    return torch.bfloat16 if code in (PKV_BF16, PKV_Q8_BF16, PKV_B8_BF16) else torch.float16


# ------------------------------------------------------------------ sizing
def kv_bytes_per_token(layers: int, kv_heads: int, head_dim: int, elem_bytes: int) -> int:
    return lib().kv_bytes_per_token(layers, kv_heads, head_dim, elem_bytes)


def kv_blocks_for_tokens(num_tokens: int, block_size: int = 16) -> int:
    return lib().kv_blocks_for_tokens(num_tokens, block_size)


def kv_pool_bytes(num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int,
                  dtype: str) -> int:
    return lib().kv_pool_bytes(num_blocks, block_size, num_kv_heads, head_dim, _DTYPES[dtype])


def default_split() -> int:
    return lib().paged_decode_default_split()


# ------------------------------------------------------------------ ledger
class KVPool:
    """A block pool: the library's host ledger plus (optionally) the device K/V pools.

    ``device=None`` creates the ledger only.  Otherwise ``k_pool``/``v_pool`` are
    torch tensors [num_blocks][num_kv_heads][block_size][head_dim] on that device
    (contents uninitialised, as a pool reserved up front).

    With ``dtype="q8_bf16"`` or ``"q8_f16"`` (8-bit cache, one fp16 scale per 32
    values; head_dim 128, block_size 16) the device pool is ``kv`` uint8
    [num_blocks][num_kv_heads][4352]: one record per slab holding K codes, V codes
    and both scale runs (layout in include/pagedkv.h).

    With ``dtype="b8_bf16"`` or ``"b8_f16"`` (8-bit cache, one fp32 scale per block,
    kv head and K or V; head_dim 64 or 128, block_size 16) ``kv`` is uint8
    [num_blocks][num_kv_heads][32 * head_dim + 32], one record per (block, kv head).
    """

    def __init__(self, num_blocks: int, num_kv_heads: int, head_dim: int, dtype: str = "bf16",
                 block_size: int = 16, free_order=None, device=None):
        self.num_blocks, self.num_kv_heads, self.head_dim = num_blocks, num_kv_heads, head_dim
        self.block_size = block_size
        self.dtype_code = _DTYPES[dtype]
        self.dtype = _NAMES[self.dtype_code]
        self.is_q8 = self.dtype_code in (PKV_Q8_BF16, PKV_Q8_F16)
        self.is_b8 = self.dtype_code in (PKV_B8_BF16, PKV_B8_F16)
        # bytes of one (block, kv head) record; 0: separate 16-bit K and V pools
        self.record_bytes = (_native.PKV_Q8_SLAB_BYTES if self.is_q8 else
                             32 * head_dim + 32 if self.is_b8 else 0)
        order = None
        if free_order is not None:
            order = np.ascontiguousarray(free_order, dtype=np.int32)
            if order.shape != (num_blocks,):
                raise ValueError("free_order must have num_blocks entries")
        h = ctypes.c_void_p()
        check(lib().kv_pool_create(num_blocks, block_size, num_kv_heads, head_dim,
                                   self.dtype_code, _np_ptr(order) if order is not None else None,
                                   ctypes.byref(h)), "kv_pool_create")
        self._h = h
        # what the compiled call checks need to know of the pool (see _load_torch)
        self._meta = (h.value, num_blocks, num_kv_heads, block_size, head_dim,
                      int(self.dtype_code in (PKV_BF16, PKV_B8_BF16)),
                      32 * head_dim + 32 if self.dtype_code in (PKV_B8_BF16, PKV_B8_F16) else 0)
        self.k_pool = self.v_pool = self.kv = self._rows = None
        if device is not None:
            import torch
            if self.record_bytes:
                self.kv = torch.empty((num_blocks, num_kv_heads, self.record_bytes),
                                      dtype=torch.uint8, device=device)
            else:
                shape = (num_blocks, num_kv_heads, block_size, head_dim)
                self.k_pool = torch.empty(shape, dtype=_torch_dtype(self.dtype_code), device=device)
                self.v_pool = torch.empty(shape, dtype=_torch_dtype(self.dtype_code), device=device)

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("pool is closed")
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None:
            lib().kv_pool_destroy(self._h)
            self._h = self._meta = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc(self, n: int) -> np.ndarray:
        out = np.empty(n, dtype=np.int32)
        check(lib().kv_block_alloc(self.handle, n, _np_ptr(out)), "kv_block_alloc")
        return out

    def ref(self, ids) -> None:
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        check(lib().kv_block_ref(self.handle, len(ids), _np_ptr(ids)), "kv_block_ref")

    def free(self, ids) -> None:
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        check(lib().kv_block_free(self.handle, len(ids), _np_ptr(ids)), "kv_block_free")

    def refcount(self, block_id: int) -> int:
        out = ctypes.c_int32()
        check(lib().kv_block_refcount(self.handle, block_id, ctypes.byref(out)), "kv_block_refcount")
        return out.value

    def num_shared(self) -> int:
        """Blocks referenced by two or more sequences."""
        out = ctypes.c_int64()
        check(lib().kv_pool_num_shared(self.handle, ctypes.byref(out)), "kv_pool_num_shared")
        return out.value

    def num_free(self) -> int:
        out = ctypes.c_int32()
        check(lib().kv_pool_num_free(self.handle, ctypes.byref(out)), "kv_pool_num_free")
        return out.value

    def append_slots(self, seq_lens, num_new, block_tables: np.ndarray) -> np.ndarray:
        """Grow sequences by ``num_new`` tokens; updates ``block_tables`` (int32
        [S][max_blocks], C-contiguous numpy, in place) and returns the int64 slots."""
        lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
        new = np.ascontiguousarray(num_new, dtype=np.int32)
        if not (isinstance(block_tables, np.ndarray) and block_tables.dtype == np.int32
                and block_tables.flags.c_contiguous and block_tables.ndim == 2):
            raise TypeError("block_tables must be a C-contiguous int32 numpy array [S][max_blocks]")
        if block_tables.shape[0] != len(lens) or len(new) != len(lens):
            raise ValueError("length mismatch")
        slots = np.empty(int(new.sum()), dtype=np.int64)
        check(lib().kv_append_slots(self.handle, len(lens), _np_ptr(lens), _np_ptr(new),
                                    _np_ptr(block_tables), block_tables.shape[1],
                                    _np_ptr(slots)), "kv_append_slots")
        return slots


    def fork(self, parent_row: np.ndarray, parent_len: int, child_row: np.ndarray) -> None:
        """The child sequence's table row shares every block of the parent's."""
        for r in (parent_row, child_row):
            if not (r.dtype == np.int32 and r.flags.c_contiguous):
                raise TypeError("table rows must be C-contiguous int32")
        check(lib().kv_seq_fork(self.handle, _np_ptr(parent_row), int(parent_len),
                                _np_ptr(child_row), child_row.shape[0]), "kv_seq_fork")

    def append_slots_cow(self, seq_lens, num_new, block_tables: np.ndarray):
        """append_slots with copy-on-write of shared tail blocks.
        Returns (slots int64, copies int32 [n][2] as (shared, fresh))."""
        lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
        new = np.ascontiguousarray(num_new, dtype=np.int32)
        if not (isinstance(block_tables, np.ndarray) and block_tables.dtype == np.int32
                and block_tables.flags.c_contiguous and block_tables.ndim == 2):
            raise TypeError("block_tables must be a C-contiguous int32 numpy array [S][max_blocks]")
        S = len(lens)
        slots = np.empty(int(new.sum()), dtype=np.int64)
        src = np.empty(max(S, 1), dtype=np.int32)
        dst = np.empty(max(S, 1), dtype=np.int32)
        n = ctypes.c_int32()
        check(lib().kv_append_slots_cow(self.handle, S, _np_ptr(lens), _np_ptr(new),
                                        _np_ptr(block_tables), block_tables.shape[1],
                                        _np_ptr(slots), _np_ptr(src), _np_ptr(dst),
                                        ctypes.byref(n)), "kv_append_slots_cow")
        return slots, np.stack([src[:n.value], dst[:n.value]], axis=1)


# ------------------------------------------------------------------ device ops
def _pools(pool: KVPool, k_pool, v_pool):
    """Device pools of a call: (K, V), or (records, None) for an 8-bit pool."""
    if pool.record_bytes:
        return (pool.kv if k_pool is None else k_pool), None
    return (pool.k_pool if k_pool is None else k_pool), (pool.v_pool if v_pool is None else v_pool)


def block_copy(pool: KVPool, src_ids, dst_ids, status, k_pool=None, v_pool=None,
               stream=None) -> None:
    """Launch the block-copy kernel (int32 device tensors of block ids)."""
    _check_layout({"src_ids": src_ids, "dst_ids": dst_ids},
                  int32={"src_ids": src_ids, "dst_ids": dst_ids})
    k_pool, v_pool = _pools(pool, k_pool, v_pool)
    _check_vector("src_ids", src_ids, None, None)
    n = int(src_ids.shape[0])
    _check_vector("dst_ids", dst_ids, n, src_ids.device)
    _check_block_pools(pool, src_ids, status, k_pool, v_pool)
    check(lib().kv_block_copy(pool.handle, _t_ptr(src_ids), _t_ptr(dst_ids), n, _t_ptr(k_pool),
                              _t_ptr(v_pool), _t_ptr(status), _stream(stream)), "kv_block_copy")


def _check_write_args(pool: KVPool, k_new, v_new, slot_mapping, status, pools) -> None:
    """Rows [T][Hkv][D] in the pool's row type for T int64 slots."""
    _check_layout({"k_new": k_new, "v_new": v_new, "slot_mapping": slot_mapping},
                  int64={"slot_mapping": slot_mapping})
    _check_vector("slot_mapping", slot_mapping, None, None)
    T = int(slot_mapping.shape[0])
    dt = _torch_dtype(pool.dtype_code)
    _check_rows("k_new", k_new, T, pool.num_kv_heads, pool.head_dim, dt, None)
    _check_rows("v_new", v_new, T, pool.num_kv_heads, pool.head_dim, dt, k_new.device)
    _check_vector("slot_mapping", slot_mapping, T, k_new.device)
    checked = []
    for name, t in pools:
        if t is not None:
            _check_pool_tensor(name, t, pool)
            checked.append((name, t))
    _check_device_call(k_new, status, None, checked)


def cache_write(pool: KVPool, k_new, v_new, slot_mapping, status, k_pool=None, v_pool=None,
                stream=None) -> None:
    """Launch the cache-write kernel: rows of ``k_new``/``v_new`` [T][Hkv][D] (device)
    go to their slots (int64 device tensor [T]) in the pools."""
    k_pool = pool.k_pool if k_pool is None else k_pool
    v_pool = pool.v_pool if v_pool is None else v_pool
    _check_write_args(pool, k_new, v_new, slot_mapping, status,
                      (("k_pool", k_pool), ("v_pool", v_pool)))
    T = int(slot_mapping.shape[0])
    check(lib().kv_cache_write(pool.handle, _t_ptr(k_new), _t_ptr(v_new), _t_ptr(slot_mapping), T,
                               _t_ptr(k_pool), _t_ptr(v_pool), _t_ptr(status), _stream(stream)),
          "kv_cache_write")


def _check_block_pools(pool: KVPool, ids, status, k_pool, v_pool, staging=None) -> None:
    """Pool tensors of a block-movement call hold the pool's geometry; a staging
    buffer holds every listed block; all on the ids' device."""
    pools = []
    for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
        if t is not None:
            _check_pool_tensor(name, t, pool)
            pools.append((name, t))
    if staging is not None:
        _check_vector("ids", ids, None, None)
        per_block = (pool.num_kv_heads * pool.record_bytes if pool.record_bytes else
                     2 * pool.num_kv_heads * pool.block_size * pool.head_dim * 2)
        if staging.numel() * staging.element_size() < int(ids.shape[0]) * per_block:
            raise ValueError(f"staging holds fewer than {int(ids.shape[0])} blocks of "
                             f"{per_block} bytes")
        pools.append(("staging", staging))
    _check_device_call(ids, status, None, pools)


def gather_blocks(pool: KVPool, ids, staging, status, k_pool=None, v_pool=None, stream=None):
    """Pack blocks ``ids`` (int32 device tensor) into ``staging`` (device,
    [n][2][Hkv][16][D] in the pool dtype; 8-bit pools [n][Hkv][record bytes]) for
    one host copy (swap out)."""
    _check_layout({"ids": ids, "staging": staging}, int32={"ids": ids})
    k_pool, v_pool = _pools(pool, k_pool, v_pool)
    _check_block_pools(pool, ids, status, k_pool, v_pool, staging)
    check(lib().kv_gather_blocks(pool.handle, _t_ptr(ids), int(ids.shape[0]), _t_ptr(k_pool),
                                 _t_ptr(v_pool), _t_ptr(staging), _t_ptr(status),
                                 _stream(stream)), "kv_gather_blocks")


def scatter_blocks(pool: KVPool, ids, staging, status, k_pool=None, v_pool=None, stream=None):
    """Unpack ``staging`` into blocks ``ids`` (swap in)."""
    _check_layout({"ids": ids, "staging": staging}, int32={"ids": ids})
    k_pool, v_pool = _pools(pool, k_pool, v_pool)
    _check_block_pools(pool, ids, status, k_pool, v_pool, staging)
    check(lib().kv_scatter_blocks(pool.handle, _t_ptr(ids), int(ids.shape[0]), _t_ptr(staging),
                                  _t_ptr(k_pool), _t_ptr(v_pool), _t_ptr(status),
                                  _stream(stream)), "kv_scatter_blocks")


def decode_plan_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                      max_blocks_per_seq: int) -> int:
    """Bytes of the host-built work plan (the start of the decode workspace)."""
    return lib().paged_decode_plan_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                         max_blocks_per_seq)


def _host_ptr_bytes(buf):
    """(pointer, bytes) of a host buffer: a numpy array or a CPU torch tensor."""
    if isinstance(buf, np.ndarray):
        if not buf.flags.c_contiguous:
            raise ValueError("plan must be contiguous")
        return buf.ctypes.data_as(ctypes.c_void_p), buf.nbytes
    if buf.device.type != "cpu" or not buf.is_contiguous():
        raise ValueError("plan must be a contiguous host tensor")
    return ctypes.c_void_p(buf.data_ptr()), buf.numel() * buf.element_size()


def decode_plan(pool: KVPool, context_lens: np.ndarray, block_tables, num_q_heads: int,
                plan, max_blocks_per_seq: int | None = None) -> int:
    """Build the decode work plan on the host (paged_decode_plan) from host
    int32 ``context_lens`` [S] and ``block_tables`` [S][max_blocks] into
    ``plan`` (a host buffer of ``decode_plan_bytes(...)`` bytes, pinned for an
    asynchronous copy).  With ``block_tables=None`` no shared-prefix runs are
    looked for and ``max_blocks_per_seq`` gives the table width.  Returns the
    number of shared-prefix work items."""
    lens = np.ascontiguousarray(context_lens, dtype=np.int32)
    S = len(lens)
    if block_tables is not None:
        if not (isinstance(block_tables, np.ndarray) and block_tables.dtype == np.int32 and
                block_tables.flags.c_contiguous and block_tables.ndim == 2 and
                block_tables.shape[0] == S):
            raise TypeError("block_tables must be a C-contiguous int32 numpy array [S][max_blocks]")
        maxb, tptr = block_tables.shape[1], _np_ptr(block_tables)
    else:
        if max_blocks_per_seq is None:
            raise ValueError("without block_tables, max_blocks_per_seq gives the table width")
        maxb, tptr = int(max_blocks_per_seq), None
    ptr, nbytes = _host_ptr_bytes(plan)
    n = ctypes.c_int32()
    check(lib().paged_decode_plan(pool.handle, _np_ptr(lens), tptr, maxb, S, num_q_heads, ptr,
                                  nbytes, ctypes.byref(n)), "paged_decode_plan")
    return n.value


def paged_decode_attention_planned(pool: KVPool, q, block_tables, context_lens, scale: float,
                                   shared_prefix_items: int, workspace, status, out=None,
                                   stream=None):
    """paged_decode_attention whose ``workspace`` already begins with a plan
    from ``decode_plan`` for the same lengths and tables."""
    import torch
    if out is None:
        out = torch.empty_like(q)
    _check_decode_args(pool, q, out, block_tables, context_lens, status, workspace,
                       pool.k_pool, pool.v_pool)
    S, hq, d = q.shape
    nbytes = workspace.numel() * workspace.element_size()
    check(lib().paged_decode_attention_planned(pool.handle, _t_ptr(out), _t_ptr(q),
                                               _t_ptr(pool.k_pool), _t_ptr(pool.v_pool),
                                               _t_ptr(block_tables), int(block_tables.shape[1]),
                                               _t_ptr(context_lens), S, hq, float(scale),
                                               int(shared_prefix_items), _t_ptr(workspace), nbytes,
                                               _t_ptr(status), _stream(stream)),
          "paged_decode_attention_planned")
    return out


def decode_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                           max_blocks_per_seq: int, blocks_per_split: int | None = None) -> int:
    if blocks_per_split is None:
        return lib().paged_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                  max_blocks_per_seq)
    return lib().paged_decode_workspace_bytes_split(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                    max_blocks_per_seq, blocks_per_split)


def paged_decode_attention(pool: KVPool, q, block_tables, context_lens, scale: float, workspace,
                           status, out=None, k_pool=None, v_pool=None,
                           blocks_per_split: int | None = None, stream=None):
    """Launch paged decode attention.  ``q`` [S][Hq][D] device tensor in the pool dtype;
    ``block_tables`` int32 device [S][max_blocks]; ``context_lens`` int32 device [S];
    ``workspace`` a uint8 device tensor of ``decode_workspace_bytes(...)`` bytes.
    Returns ``out`` [S][Hq][D]."""
    import torch
    k_pool = pool.k_pool if k_pool is None else k_pool
    v_pool = pool.v_pool if v_pool is None else v_pool
    if out is None:
        out = torch.empty_like(q)
    _check_decode_args(pool, q, out, block_tables, context_lens, status, workspace,
                       k_pool, v_pool)
    S, hq, d = q.shape
    maxb = int(block_tables.shape[1])
    nbytes = workspace.numel() * workspace.element_size()
    if blocks_per_split is None:
        rc = lib().paged_decode_attention(pool.handle, _t_ptr(out), _t_ptr(q), _t_ptr(k_pool),
                                          _t_ptr(v_pool), _t_ptr(block_tables), maxb,
                                          _t_ptr(context_lens), S, hq, float(scale),
                                          _t_ptr(workspace), nbytes, _t_ptr(status),
                                          _stream(stream))
    else:
        rc = lib().paged_decode_attention_split(pool.handle, _t_ptr(out), _t_ptr(q),
                                                _t_ptr(k_pool), _t_ptr(v_pool),
                                                _t_ptr(block_tables), maxb, _t_ptr(context_lens),
                                                S, hq, float(scale), int(blocks_per_split),
                                                _t_ptr(workspace), nbytes, _t_ptr(status),
                                                _stream(stream))
    check(rc, "paged_decode_attention")
    return out


class CapturedDecode:
    """One paged decode attention call (16-bit or 8-bit pool) captured into a
    CUDA graph on fixed device buffers: ``replay()`` runs the prep, attention
    and merge kernels with a single graph launch instead of a Python call and
    three kernel launches, so a serving loop whose steps are short does not
    leave the GPU waiting on the host.  Each replay reads the buffers' current
    contents (q, tables, lengths) and writes ``out``, the workspace and the
    status word; the partition size is chosen on the device as in a direct
    call.  At capture time the buffers must hold a valid batch (zero lengths
    will do): one untimed call on a side stream sets the kernels up first."""

    def __init__(self, pool: KVPool, q, block_tables, context_lens, scale: float, workspace,
                 status, out, planned_prefix_items: int | None = None,
                 window: int | None = None, sinks: int = 0):
        """``window``/``sinks``: capture the windowed call (16-bit and block-scaled
        pools; ``workspace`` is then not used and may be None, as for every
        block-scaled pool).  ``planned_prefix_items`` not None: capture the planned call
        (``paged_decode_attention_planned``, 16-bit pools): every replay then
        expects the workspace to begin with a host plan with that many
        shared-prefix items (the capture itself needs a valid plan there)."""
        import torch
        self.torch = torch

        def call():
            if pool.is_b8:
                paged_decode_attention_b8(pool, q, block_tables, context_lens, scale, status,
                                          window=window, sinks=sinks, out=out)
            elif window is not None:
                paged_decode_attention_window(pool, q, block_tables, context_lens, scale, window,
                                              sinks, status, out=out)
            elif pool.is_q8:
                paged_decode_attention_q8(pool, q, block_tables, context_lens, scale, workspace,
                                          status, out=out)
            elif planned_prefix_items is not None:
                paged_decode_attention_planned(pool, q, block_tables, context_lens, scale,
                                               planned_prefix_items, workspace, status, out=out)
            else:
                paged_decode_attention(pool, q, block_tables, context_lens, scale, workspace,
                                       status, out=out)

        side = torch.cuda.Stream(device=q.device)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            call()
        self.out = out

    def replay(self):
        """Enqueue the captured call on the current stream."""
        self.graph.replay()
        return self.out


def paged_decode_attention_noalloc(pool: KVPool, q, block_tables, context_lens, scale: float,
                                   status, out, k_pool=None, v_pool=None, stream=None):
    """Paged decode attention with the library's fixed scratch instead of a
    caller workspace; the library allocates nothing (for callers that cannot
    allocate device memory at decode time).  ``out`` must be given.  Calls on one
    device share the scratch: do not overlap them on the GPU."""
    k_pool = pool.k_pool if k_pool is None else k_pool
    v_pool = pool.v_pool if v_pool is None else v_pool
    _check_decode_args(pool, q, out, block_tables, context_lens, status, None, k_pool, v_pool)
    S, hq, d = q.shape
    rc = lib().paged_decode_attention_noalloc(pool.handle, _t_ptr(out), _t_ptr(q),
                                              _t_ptr(k_pool), _t_ptr(v_pool),
                                              _t_ptr(block_tables), int(block_tables.shape[1]),
                                              _t_ptr(context_lens), S, hq, float(scale),
                                              _t_ptr(status), _stream(stream))
    check(rc, "paged_decode_attention_noalloc")
    return out


def prefill_workspace_bytes(num_seqs: int, num_tokens: int, num_q_heads: int,
                            num_kv_heads: int, head_dim: int | None = None,
                            max_blocks_per_seq: int | None = None) -> int:
    """Workspace bytes of ``paged_prefill_attention``; with ``head_dim`` and
    ``max_blocks_per_seq`` also room for the fp16 copy of V that a bf16 pool
    then uses (one fp16 part of P in P V instead of two bf16 parts)."""
    if head_dim is None and max_blocks_per_seq is None:
        return lib().paged_prefill_workspace_bytes(num_seqs, num_tokens, num_q_heads, num_kv_heads)
    if head_dim is None or max_blocks_per_seq is None:
        raise ValueError("head_dim and max_blocks_per_seq go together")
    return lib().paged_prefill_workspace_bytes_staged(num_seqs, num_tokens, num_q_heads,
                                                      num_kv_heads, head_dim, max_blocks_per_seq)


def paged_prefill_attention(pool: KVPool, q, block_tables, query_start, context_lens,
                            scale: float, workspace, status, out=None, k_pool=None, v_pool=None,
                            stream=None):
    """Chunked-prefill attention: ``q`` [T][Hq][D] device rows of all chunks,
    ``query_start`` int32 device [S+1], ``context_lens`` int32 device [S]."""
    import torch
    _check_layout({"q": q, "out": out, "block_tables": block_tables, "query_start": query_start,
                   "context_lens": context_lens, "workspace": workspace},
                  int32={"block_tables": block_tables, "query_start": query_start,
                         "context_lens": context_lens})
    k_pool = pool.k_pool if k_pool is None else k_pool
    v_pool = pool.v_pool if v_pool is None else v_pool
    if out is None:
        out = torch.empty_like(q)
    dt = _torch_dtype(pool.dtype_code)
    _check_rows("q", q, None, None, pool.head_dim, dt, None)
    T, hq, d = q.shape
    if hq % pool.num_kv_heads:
        raise ValueError(f"q has {hq} heads, not a multiple of the pool's "
                         f"{pool.num_kv_heads} kv heads")
    _check_rows("out", out, T, hq, pool.head_dim, dt, q.device)
    _check_vector("context_lens", context_lens, None, q.device)
    S = int(context_lens.shape[0])
    _check_vector("block_tables", block_tables, S, q.device, ndim=2)
    _check_vector("query_start", query_start, S + 1, q.device)
    if workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    pools = []
    for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
        if t is not None:
            _check_pool_tensor(name, t, pool)
            pools.append((name, t))
    _check_device_call(q, status, workspace, pools)
    nbytes = workspace.numel() * workspace.element_size()
    check(lib().paged_prefill_attention(pool.handle, _t_ptr(out), _t_ptr(q), _t_ptr(k_pool),
                                        _t_ptr(v_pool), _t_ptr(block_tables),
                                        int(block_tables.shape[1]), _t_ptr(query_start),
                                        _t_ptr(context_lens), S, T, hq, float(scale),
                                        _t_ptr(workspace), nbytes, _t_ptr(status),
                                        _stream(stream)), "paged_prefill_attention")
    return out


def cache_write_q8(pool: KVPool, k_new, v_new, slot_mapping, status, stream=None) -> None:
    """Quantising cache write into an 8-bit pool: rows of ``k_new``/``v_new``
    [T][Hkv][128] (bf16 for q8_bf16, fp16 for q8_f16) go to their slots as codes
    and fp16 scales."""
    _check_write_args(pool, k_new, v_new, slot_mapping, status, (("kv", pool.kv),))
    T = int(slot_mapping.shape[0])
    check(lib().kv_cache_write_q8(pool.handle, _t_ptr(k_new), _t_ptr(v_new), _t_ptr(slot_mapping),
                                  T, _t_ptr(pool.kv), _t_ptr(status), _stream(stream)),
          "kv_cache_write_q8")


def paged_decode_attention_q8(pool: KVPool, q, block_tables, context_lens, scale: float,
                              workspace, status, out=None, stream=None):
    """Paged decode attention over an 8-bit pool (head_dim 128, G <= 8); ``q`` and
    the result in bf16 (q8_bf16) or fp16 (q8_f16); workspace as for
    ``decode_workspace_bytes``."""
    import torch
    if out is None:
        out = torch.empty_like(q)
    _check_decode_args(pool, q, out, block_tables, context_lens, status, workspace,
                       pool.kv if pool.kv is not None else None)
    S, hq, d = q.shape
    nbytes = workspace.numel() * workspace.element_size()
    check(lib().paged_decode_attention_q8(pool.handle, _t_ptr(out), _t_ptr(q), _t_ptr(pool.kv),
                                          _t_ptr(block_tables), int(block_tables.shape[1]),
                                          _t_ptr(context_lens), S, hq, float(scale),
                                          _t_ptr(workspace), nbytes, _t_ptr(status),
                                          _stream(stream)), "paged_decode_attention_q8")
    return out


# --------------------------------------- rotated append, 8-bit blocks, windows
# The calls below are also made for a few rows at a time, where the host side is
# most of their time.  Their argument checks exist twice: compiled (_fastcall,
# csrc/fastcall.cpp), which calls the library when every check holds, and here,
# which says what is wrong when one does not (and makes the call where the
# compiled form does not: a library built without torch's headers, tensors on
# another device than the current one).
_torch = _fast = None


def _load_fastcall(torch):
    """The module of compiled checks, or None: not built, or built for another torch, another
    Python or another interface of the library."""
    import sys
    from .build import interface_hash
    try:
        from . import _fastcall
        made_for = (_fastcall.torch_version, _fastcall.python_version, _fastcall.interface)
        here = (torch.__version__.split("+")[0], sys.version_info[0] * 100 + sys.version_info[1],
                interface_hash())
    except (ImportError, AttributeError, OSError):
        return None
    return _fastcall if made_for == here else None


def _load_torch():
    global _torch, _fast
    import torch
    _fastcall = _load_fastcall(torch)
    if _fastcall is not None:
        _fastcall.bind(*(ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value for name in (
            "paged_decode_attention_window", "paged_decode_attention_b8", "kv_cache_write_rope",
            "kv_dequantize_blocks", "paged_prefill_attention_window")))
    _torch, _fast = torch, _fastcall
    return torch


def _raw(stream):
    """A call's ``stream`` argument as the compiled checks take it."""
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _refuse(name: str, t, shape: tuple, dtype, index: int, contiguous: bool):
    """Raise for a tensor that failed its check."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}, got "
                        f"{str(t.dtype).replace('torch.', '')}")
    if t.get_device() != index:
        where = "the CPU" if index < 0 else f"cuda:{index}"
        raise ValueError(f"{name} is on {t.device}, the call's rows are on {where}")
    if contiguous:
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} was refused")


def _want(name: str, t, shape: tuple, dtype, index: int) -> int:
    """Check a contiguous tensor of the call; its address."""
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != index
            or not t.is_contiguous()):
        _refuse(name, t, shape, dtype, index, True)
    return t.data_ptr()


def _want_rows(name: str, t, shape: tuple, dtype, index: int):
    """Check rows [T][H][D] whose tokens may lie apart (slices of a fused
    projection); their address and token stride in elements."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        _refuse(name, t, shape, dtype, index, False)
    T, H, D = shape
    s, sh, sd = t.stride()
    if T > 0 and H > 0 and (sd != 1 or (sh != D and H > 1)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if T <= 1:
        s = H * D
    elif s < H * D or s % 8:
        raise ValueError(f"{name}: the token stride must be a multiple of 8 and at least "
                         f"{H * D}, got {s}")
    return t.data_ptr(), s


def _want_status(status, index: int) -> int:
    if status.dtype is not _torch.int32 or status.numel() < 1:
        raise TypeError("status must be an int32 tensor of at least one element")
    if status.get_device() != index:
        raise ValueError(f"status is on {status.device}, the call's rows are not")
    return status.data_ptr()


def _want_pools(pool: KVPool, index: int, k_pool=None, v_pool=None, kv=None):
    """Addresses of the call's device pools: (K, V), or (records, 0)."""
    if pool.record_bytes:
        if not pool.is_b8:
            raise ValueError("the call takes 16-bit and block-scaled 8-bit pools")
        kv = pool.kv if kv is None else kv
        if kv is None:
            raise ValueError("the pool has no device memory")
        return _want("kv", kv, (pool.num_blocks, pool.num_kv_heads, pool.record_bytes),
                     _torch.uint8, index), 0
    k_pool = pool.k_pool if k_pool is None else k_pool
    v_pool = pool.v_pool if v_pool is None else v_pool
    if k_pool is None or v_pool is None:
        raise ValueError("the pool has no device memory")
    shape = (pool.num_blocks, pool.num_kv_heads, pool.block_size, pool.head_dim)
    dt = _row_dtype(pool)
    return _want("k_pool", k_pool, shape, dt, index), _want("v_pool", v_pool, shape, dt, index)


def _row_dtype(pool: KVPool):
    """Element type of the pool's rows (looked up once per pool)."""
    dt = pool._rows
    if dt is None:
        if _torch is None:
            _load_torch()
        dt = pool._rows = _torch_dtype(pool.dtype_code)
    return dt


def _launch(name: str, index: int, stream, *args) -> None:
    """Call the library's ``name`` with ``args`` and, last, ``stream`` or the current
    stream of device ``index``, which is made current for the call if it is not."""
    if index < 0:
        raise ValueError("the call's tensors must be CUDA tensors, got cpu")
    torch = _torch
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    fn = getattr(lib(), name)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc:
        check(rc, name)


def rope_table(max_positions: int, rotary_dim: int, base: float = 10000.0, device=None):
    """cos/sin table of ``cache_write_rope``: fp32 [max_positions][rotary_dim], row p
    = the cosines, then the sines, of p * base^(-2 i / rotary_dim), i <
    rotary_dim / 2, computed in fp64."""
    import torch
    if max_positions < 1 or rotary_dim < 16 or rotary_dim % 16:
        raise ValueError("max_positions >= 1 and rotary_dim a multiple of 16")
    half = rotary_dim // 2
    freq = float(base) ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(max_positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).to(device)


def cache_write_rope(pool: KVPool, k_new, v_new, positions, cos_sin, slot_mapping, status, q=None,
                     q_out=None, interleaved: bool = False, k_pool=None, v_pool=None, kv=None,
                     stream=None):
    """Append tokens with their K (and queries) rotated by position, one launch.

    ``k_new``/``v_new`` [T][Hkv][D] and ``q`` [T][Hq][D] device rows in the pool's
    row type, tokens any stride apart (slices of a fused projection); ``positions``
    int32 [T]; ``cos_sin`` fp32 [max_positions][rotary_dim] (``rope_table``);
    ``slot_mapping`` int64 [T], negative = no token.  K and V go to their slots of a
    16-bit pool or a block-scaled 8-bit pool; the rotated queries to ``q_out``
    (default: a new tensor; ``q`` itself: in place), which is returned.  Rows of
    skipped tokens in ``q_out`` are left as they were.  ``interleaved``: pairs of
    neighbouring dimensions instead of the halves' (i, i + rotary_dim / 2)."""
    dt = pool._rows or _row_dtype(pool)
    torch = _torch
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if _fast is not None:
        a, b = ((pool.kv if kv is None else kv, None) if pool.record_bytes else
                (pool.k_pool if k_pool is None else k_pool, pool.v_pool if v_pool is None else v_pool))
        rc = None if pool.is_q8 else _fast.rope(
            pool._meta, k_new, v_new, positions, cos_sin, slot_mapping, status, q, q_out,
            1 if interleaved else 0, a, b, _raw(stream))
        if rc is not None:
            if rc:
                check(rc, "kv_cache_write_rope")
            return q_out
    dev, D, Hkv = k_new.get_device(), pool.head_dim, pool.num_kv_heads
    T = slot_mapping.shape[0] if slot_mapping.dim() == 1 else -1
    slots = _want("slot_mapping", slot_mapping, (T,), torch.int64, dev)
    pos = _want("positions", positions, (T,), torch.int32, dev)
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_positions][rotary_dim]")
    rows, rot = cos_sin.shape
    table = _want("cos_sin", cos_sin, (rows, rot), torch.float32, dev)
    k, ks = _want_rows("k_new", k_new, (T, Hkv, D), dt, dev)
    v, vs = _want_rows("v_new", v_new, (T, Hkv, D), dt, dev)
    qp = qs = qo = qos = hq = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must be [{T}][h][{D}], got {list(q.shape)}")
        hq = q.shape[1]
        qp, qs = _want_rows("q", q, (T, hq, D), dt, dev)
        qo, qos = (qp, qs) if q_out is q else _want_rows("q_out", q_out, (T, hq, D), dt, dev)
        if qp == qo and qs != qos:
            raise ValueError("q_out over q needs the same token stride")
    elif q_out is not None:
        raise ValueError("q_out without q")
    kp, vp = _want_pools(pool, dev, k_pool, v_pool, kv)
    _launch("kv_cache_write_rope", dev, stream, pool.handle, qo, qos, qp, qs, hq, k, ks, v, vs,
            pos, table, rows, rot, 1 if interleaved else 0, slots, T, kp, vp,
            _want_status(status, dev))
    return q_out


def cache_write_b8(pool: KVPool, k_new, v_new, slot_mapping, status, kv=None, stream=None) -> None:
    """Quantising append into a block-scaled 8-bit pool: contiguous rows
    ``k_new``/``v_new`` [T][Hkv][D] go to their slots; a block's scale covers the
    largest value written to it since its first token, and the codes before the new
    tokens are rounded to it when it grows.  The tokens of one block are neighbours
    in ``slot_mapping``, slots rising by one (as the ledger hands them out)."""
    torch = _torch or _load_torch()
    dev = k_new.get_device()
    if not pool.is_b8:
        raise ValueError("cache_write_b8 takes a block-scaled 8-bit pool")
    dt, shape = _row_dtype(pool), (pool.num_kv_heads, pool.head_dim)
    T = slot_mapping.shape[0] if slot_mapping.dim() == 1 else -1
    slots = _want("slot_mapping", slot_mapping, (T,), torch.int64, dev)
    k = _want("k_new", k_new, (T, *shape), dt, dev)
    v = _want("v_new", v_new, (T, *shape), dt, dev)
    rec, _ = _want_pools(pool, dev, kv=kv)
    _launch("kv_cache_write_b8", dev, stream, pool.handle, k, v, slots, T, rec,
            _want_status(status, dev))


def dequantize_blocks(pool: KVPool, ids, k_out, v_out, status, kv=None, stream=None):
    """Blocks ``ids`` (int32 device [n]) of a block-scaled 8-bit pool as 16-bit rows:
    ``k_out``/``v_out`` [n][Hkv][16][D] in the pool's row type (the layout of a 16-bit
    pool of n blocks).  Returns (k_out, v_out)."""
    torch = _torch or _load_torch()
    if not pool.is_b8:
        raise ValueError("dequantize_blocks takes a block-scaled 8-bit pool")
    if _fast is not None:
        rc = _fast.dequantize(pool._meta, ids, k_out, v_out, status, pool.kv if kv is None else kv,
                              _raw(stream))
        if rc is not None:
            if rc:
                check(rc, "kv_dequantize_blocks")
            return k_out, v_out
    dev = ids.get_device()
    n = ids.shape[0] if ids.dim() == 1 else -1
    i = _want("ids", ids, (n,), torch.int32, dev)
    dt, shape = _row_dtype(pool), (n, pool.num_kv_heads, 16, pool.head_dim)
    k = _want("k_out", k_out, shape, dt, dev)
    v = _want("v_out", v_out, shape, dt, dev)
    rec, _ = _want_pools(pool, dev, kv=kv)
    _launch("kv_dequantize_blocks", dev, stream, pool.handle, i, n, rec, k, v,
            _want_status(status, dev))
    return k_out, v_out


def _decode_call(name: str, pool: KVPool, q, out, block_tables, context_lens, scale, window, sinks,
                 status, k_pool, v_pool, kv, stream):
    """Checks and launch of the windowed decode calls."""
    dt = pool._rows or _row_dtype(pool)
    torch = _torch
    if out is None:
        out = torch.empty_like(q)
    if _fast is not None:
        a, b = ((pool.kv if kv is None else kv, None) if pool.is_b8 else
                (pool.k_pool if k_pool is None else k_pool, pool.v_pool if v_pool is None else v_pool))
        rc = _fast.decode(pool._meta, q, out, block_tables, context_lens, float(scale), window, sinks,
                          status, a, b, _raw(stream))
        if rc is not None:
            if rc:
                check(rc, name)
            return out
    dev, D = q.get_device(), pool.head_dim
    if q.dim() != 3 or q.shape[2] != D:
        raise ValueError(f"q must be [n][h][{D}], got {list(q.shape)}")
    S, hq, _ = shape = tuple(q.shape)
    if hq % pool.num_kv_heads:
        raise ValueError(f"q has {hq} heads, not a multiple of the pool's "
                         f"{pool.num_kv_heads} kv heads")
    qp = _want("q", q, shape, dt, dev)
    op = _want("out", out, shape, dt, dev)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must have 2 dimensions")
    maxb = block_tables.shape[1]
    tp = _want("block_tables", block_tables, (S, maxb), torch.int32, dev)
    lp = _want("context_lens", context_lens, (S,), torch.int32, dev)
    pools = _want_pools(pool, dev, k_pool, v_pool, kv)
    if pool.is_b8:
        pools = pools[:1]
    _launch(name, dev, stream, pool.handle, op, qp, *pools, tp, maxb, lp, S, hq, float(scale),
            window, sinks, _want_status(status, dev))
    return out


def _window(window, sinks):
    window, sinks = int(window), int(sinks)
    if window < 1 or sinks < 0 or window > 0x7fffffff or sinks > 0x7fffffff:
        raise ValueError(f"window >= 1 and sinks >= 0 (32 bits), got {window} and {sinks}")
    return window, sinks


def paged_decode_attention_window(pool: KVPool, q, block_tables, context_lens, scale: float,
                                  window: int, sinks: int, status, out=None, k_pool=None,
                                  v_pool=None, stream=None):
    """Decode attention over each sequence's last ``window`` tokens and its first
    ``sinks`` tokens (16-bit pools; ``paged_decode_attention_b8`` has the same for
    block-scaled 8-bit pools).  Arguments as ``paged_decode_attention``, without a
    workspace; table entries of blocks without a visible token are not read."""
    if pool.record_bytes:
        raise ValueError("paged_decode_attention_window takes a 16-bit pool")
    window, sinks = _window(window, sinks)
    return _decode_call("paged_decode_attention_window", pool, q, out, block_tables, context_lens,
                        scale, window, sinks, status, k_pool, v_pool, None, stream)


def paged_decode_attention_b8(pool: KVPool, q, block_tables, context_lens, scale: float, status,
                              window: int | None = None, sinks: int = 0, out=None, kv=None,
                              stream=None):
    """Decode attention over a block-scaled 8-bit pool (head_dim 64 or 128, G <= 16),
    over the whole context or, with ``window``, over the last ``window`` and the first
    ``sinks`` tokens.  ``q`` and the result in bf16 (b8_bf16) or fp16 (b8_f16); no
    workspace."""
    if not pool.is_b8:
        raise ValueError("paged_decode_attention_b8 takes a block-scaled 8-bit pool")
    if window is None:
        if sinks:
            raise ValueError("sinks without a window")
        window = 0
    else:
        window, sinks = _window(window, sinks)
    return _decode_call("paged_decode_attention_b8", pool, q, out, block_tables, context_lens,
                        scale, window, sinks, status, None, None, kv, stream)


def paged_prefill_attention_window(pool: KVPool, q, block_tables, query_start, context_lens,
                                   scale: float, window: int, sinks: int, workspace, status,
                                   out=None, k_pool=None, v_pool=None, stream=None):
    """``paged_prefill_attention`` where a query at position p attends to tokens p -
    window + 1 .. p and to the first ``sinks`` tokens (16-bit pools).  Workspace of
    ``prefill_workspace_bytes(S, T, Hq, Hkv)`` bytes."""
    torch = _torch or _load_torch()
    if pool.record_bytes:
        raise ValueError("paged_prefill_attention_window takes a 16-bit pool")
    window, sinks = _window(window, sinks)
    if out is None:
        out = torch.empty_like(q)
    if _fast is not None:
        rc = _fast.prefill(pool._meta, q, out, block_tables, query_start, context_lens, float(scale),
                           window, sinks, workspace, status,
                           pool.k_pool if k_pool is None else k_pool,
                           pool.v_pool if v_pool is None else v_pool, _raw(stream))
        if rc is not None:
            if rc:
                check(rc, "paged_prefill_attention_window")
            return out
    dev, dt, D = q.get_device(), _row_dtype(pool), pool.head_dim
    if q.dim() != 3 or q.shape[2] != D:
        raise ValueError(f"q must be [n][h][{D}], got {list(q.shape)}")
    T, hq, _ = shape = tuple(q.shape)
    if hq % pool.num_kv_heads:
        raise ValueError(f"q has {hq} heads, not a multiple of the pool's "
                         f"{pool.num_kv_heads} kv heads")
    qp = _want("q", q, shape, dt, dev)
    op = _want("out", out, shape, dt, dev)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must have 2 dimensions")
    S, maxb = block_tables.shape
    tp = _want("block_tables", block_tables, (S, maxb), torch.int32, dev)
    lp = _want("context_lens", context_lens, (S,), torch.int32, dev)
    sp = _want("query_start", query_start, (S + 1,), torch.int32, dev)
    nbytes = workspace.numel()
    wp = _want("workspace", workspace, (nbytes,), torch.uint8, dev)
    kp, vp = _want_pools(pool, dev, k_pool, v_pool)
    _launch("paged_prefill_attention_window", dev, stream, pool.handle, op, qp, kp, vp, tp, maxb,
            sp, lp, S, T, hq, float(scale), window, sinks, wp, nbytes, _want_status(status, dev))
    return out


def status_check(status, stream=None):
    """Synchronise the stream, read and clear the device status word.
    Returns (pkv_status code, raw word)."""
    word = ctypes.c_int32()
    rc = lib().kv_status_check(_t_ptr(status), _stream(stream), ctypes.byref(word))
    return rc, word.value
