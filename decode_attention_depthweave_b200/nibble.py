"""The 4-bit key/value cache of libdwkv: every channel kept in 4 bits, an 8-bit scale per 16
channels.  Argument marshalling and allocations; the functions have the names of the C ABI in
``include/dwkv.h``, which documents the codec, the layout and each call.

``Nibble`` wraps one handle: ``tables`` (block tables and slot map of a step, on the GPU),
``append``, ``read`` and ``attention`` on tensors the caller owns.  ``NibbleCache`` keeps the
tensors too: a pool per layer, the tables and the lengths of a fixed set of request slots.

    cache = NibbleCache(num_layers=32, num_q_heads=32, num_kv_heads=8, head_dim=128,
                        num_pages=4096, max_seqs=8, max_context=32768)
    cache.step(n_new)                      # device int32 [max_seqs]: rows that each slot adds
    for layer in range(32):
        cache.append(layer, k, v)          # [rows][Hkv][d], in slot order
        out = cache.attention(layer, q, max_q=1)
"""
from __future__ import annotations

import contextlib
import ctypes as C

import torch

import decode_attention_depthweave_b200 as _dw

__all__ = [
    "dwkv_nibble_config", "nibble_config_from", "dwkv_nibble_config_check", "dwkv_nibble_page_bytes",
    "dwkv_nibble_pool_bytes", "dwkv_nibble_arena_bytes", "dwkv_nibble_create", "dwkv_nibble_destroy",
    "dwkv_nibble_tables", "dwkv_nibble_append", "dwkv_nibble_read", "dwkv_nibble_attention",
    "dwkv_nibble_sync_status", "Nibble", "NibbleCache",
]

DWKV_BF16, DWKV_FP16 = 0, 1
_DTYPES = {torch.bfloat16: DWKV_BF16, torch.float16: DWKV_FP16}


class dwkv_nibble_config(C.Structure):
    _fields_ = [("num_q_heads", C.c_int32), ("num_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("page_tokens", C.c_int32), ("num_pages", C.c_int32), ("max_seqs", C.c_int32),
                ("max_blocks", C.c_int32), ("dtype", C.c_int32), ("window", C.c_int32), ("softmax_scale", C.c_float)]


def signatures():
    """(argument types, result type) of the entry points, for the library's loader."""
    vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    cfgp = C.POINTER(dwkv_nibble_config)
    return {
        "dwkv_nibble_config_check": ([cfgp], C.c_int),
        "dwkv_nibble_page_bytes": ([cfgp], sz),
        "dwkv_nibble_pool_bytes": ([cfgp], sz),
        "dwkv_nibble_arena_bytes": ([cfgp], sz),
        "dwkv_nibble_create": ([cfgp, vp, sz, vp, C.POINTER(vp)], C.c_int),
        "dwkv_nibble_destroy": ([vp], C.c_int),
        "dwkv_nibble_tables": ([vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp], C.c_int),
        "dwkv_nibble_append": ([vp, i32, vp, i64, vp, i64, vp, vp, vp], C.c_int),
        "dwkv_nibble_read": ([vp, i32, vp, vp, vp, vp, vp], C.c_int),
        "dwkv_nibble_attention": ([vp, i32, i32, i32, vp, i64, vp, vp, vp, vp, vp, vp, vp], C.c_int),
        "dwkv_nibble_sync_status": ([vp, vp], C.c_int),
    }


def nibble_config_from(num_q_heads, num_kv_heads, head_dim, page_tokens, num_pages, max_seqs, max_blocks,
                       dtype=torch.bfloat16, window=0, softmax_scale=0.0) -> dwkv_nibble_config:
    """dtype: torch.bfloat16 or torch.float16, the type of keys, values, queries and outputs."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be torch.bfloat16 or torch.float16 (got {dtype})")
    return dwkv_nibble_config(num_q_heads, num_kv_heads, head_dim, page_tokens, num_pages, max_seqs, max_blocks,
                              _DTYPES[dtype], window, softmax_scale)


# ------------------------------------------------------------------------------ C ABI
def dwkv_nibble_config_check(cfg) -> int:
    return _dw.lib().dwkv_nibble_config_check(C.byref(cfg))


def dwkv_nibble_page_bytes(cfg) -> int:
    return _dw.lib().dwkv_nibble_page_bytes(C.byref(cfg))


def dwkv_nibble_pool_bytes(cfg) -> int:
    return _dw.lib().dwkv_nibble_pool_bytes(C.byref(cfg))


def dwkv_nibble_arena_bytes(cfg) -> int:
    return _dw.lib().dwkv_nibble_arena_bytes(C.byref(cfg))


def dwkv_nibble_create(cfg, arena: torch.Tensor, stream=None) -> C.c_void_p:
    h = C.c_void_p()
    _dw._check(_dw.lib().dwkv_nibble_create(C.byref(cfg), arena.data_ptr(), arena.numel() * arena.element_size(),
                                            _raw(stream, arena.device), C.byref(h)))
    return h


def dwkv_nibble_destroy(h):
    _dw._check(_dw.lib().dwkv_nibble_destroy(h))


def dwkv_nibble_tables(h, n_seqs, n_new, release, seq_lens, block_tables, free_list, free_count, seq_lens_out,
                       free_count_out, max_rows, cu_rows, positions, slots, stream):
    _dw._check(_dw.lib().dwkv_nibble_tables(
        h, n_seqs, _at(n_new), _at(release), _at(seq_lens), _at(block_tables), _at(free_list), _at(free_count),
        _at(seq_lens_out), _at(free_count_out), max_rows, _at(cu_rows), _at(positions), _at(slots), stream))


def dwkv_nibble_append(h, n_rows, k, k_stride, v, v_stride, slots, pool, stream):
    _dw._check(_dw.lib().dwkv_nibble_append(h, n_rows, _at(k), k_stride, _at(v), v_stride, _at(slots), _at(pool), stream))


def dwkv_nibble_read(h, n_rows, slots, pool, k_out, v_out, stream):
    _dw._check(_dw.lib().dwkv_nibble_read(h, n_rows, _at(slots), _at(pool), _at(k_out), _at(v_out), stream))


def dwkv_nibble_attention(h, n_seqs, n_rows, max_q, q, q_stride, cu_rows, seq_lens, block_tables, pool, out, lse, stream):
    _dw._check(_dw.lib().dwkv_nibble_attention(h, n_seqs, n_rows, max_q, _at(q), q_stride, _at(cu_rows), _at(seq_lens),
                                               _at(block_tables), _at(pool), _at(out), _at(lse), stream))


def dwkv_nibble_sync_status(h, stream):
    _dw._check(_dw.lib().dwkv_nibble_sync_status(h, stream))


# ------------------------------------------------------------------------------ plumbing
def _at(t):
    return None if t is None else t.data_ptr()


def _raw(stream, device) -> int:
    """The cudaStream_t of `stream` (a torch stream, an integer, or None: the device's current one)."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _under(stream, device):
    """A context in which torch allocates and works on `stream` (as in _raw; None: nothing changes)."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


# cudaStream_t of a device's current stream, without building a Stream object where torch allows it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


class Nibble:
    """One handle on tensors that the caller owns.  Allocates the handle's arena, nothing else
    (and outputs that are not passed in).  A call's `stream` (a torch stream or a cudaStream_t; None:
    the device's current one) is the one that the call works on: what it is given has to be ready there,
    and the arena and outputs that are allocated here are tensors of that stream.  Keep the handle until
    its calls, and graphs captured from it, have run: nothing waits for them when it goes."""

    def __init__(self, cfg: dwkv_nibble_config, device="cuda", stream=None):
        if not torch.cuda.is_available():
            raise RuntimeError("libdwkv needs a CUDA device")
        _dw._check(dwkv_nibble_config_check(cfg))
        self.cfg = cfg
        self.device = torch.device("cuda", torch.cuda.current_device()) if torch.device(device).index is None \
            else torch.device(device)
        self.dtype = torch.float16 if cfg.dtype == DWKV_FP16 else torch.bfloat16
        self.pool_bytes = dwkv_nibble_pool_bytes(cfg)
        self.index, self.max_blocks, self.head_dim = self.device.index, cfg.max_blocks, cfg.head_dim
        self.num_q_heads, self.num_kv_heads = cfg.num_q_heads, cfg.num_kv_heads
        with torch.cuda.device(self.device), _under(stream, self.device):
            self.arena = torch.empty(dwkv_nibble_arena_bytes(cfg), dtype=torch.uint8, device=self.device)
            self.h = dwkv_nibble_create(cfg, self.arena, stream)

    def close(self):
        if getattr(self, "h", None):
            dwkv_nibble_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- checks of what the C side cannot see: types, devices, extents
    def _ints(self, name, t, n, exact=False):
        have = t.numel()
        if t.dtype is not torch.int32 or t.get_device() != self.index or not t.is_contiguous() or \
                (have != n if exact else have < n):
            raise ValueError(f"{name} must be contiguous int32 on {self.device} with {n} entries "
                             f"(got {t.dtype} {tuple(t.shape)} on {t.device})")

    def _table(self, t, n):
        if t.dtype is not torch.int32 or t.get_device() != self.index or not t.is_contiguous() or t.dim() != 2 or \
                t.size(0) < n or t.size(1) != self.max_blocks:
            raise ValueError(f"block_tables must be contiguous int32 [>= {n}][{self.max_blocks}] on {self.device} "
                             f"(got {t.dtype} {tuple(t.shape)} on {t.device})")

    def _pool(self, t):
        if t.get_device() != self.index or not t.is_contiguous() or t.numel() * t.element_size() != self.pool_bytes:
            raise ValueError(f"pool must be {self.pool_bytes} contiguous bytes on {self.device}")

    def _rows(self, name, t, heads):
        """(rows, row stride) of a [rows][heads][head_dim] tensor whose rows are dense."""
        if t.dtype is not self.dtype or t.get_device() != self.index or t.dim() != 3:
            shape = ()
        else:
            shape = t.shape
        d = self.head_dim
        if len(shape) != 3 or shape[1] != heads or shape[2] != d:
            raise ValueError(f"{name} must be {self.dtype} [rows][{heads}][{d}] on {self.device} "
                             f"(got {t.dtype} {tuple(t.shape)} on {t.device})")
        row, head, one = t.stride()
        if one != 1 or (head != d and heads > 1):
            raise ValueError(f"{name}: each row's heads must be dense (strides {t.stride()})")
        return shape[0], row if shape[0] > 1 else heads * d

    def _stream(self, stream):
        return _current_stream(self.index) if stream is None else _raw(stream, self.device)

    def tables(self, n_new, seq_lens, block_tables, free_list, free_count, cu_rows, slots, positions=None, release=None,
               seq_lens_out=None, free_count_out=None, stream=None):
        """Block tables and slot map of a step (dwkv_nibble_tables); lengths and the free count are
        updated in place unless outputs of their own are given.  slots.numel() is max_rows."""
        n, rows = n_new.numel(), slots.numel()
        lens_out = seq_lens if seq_lens_out is None else seq_lens_out
        count_out = free_count if free_count_out is None else free_count_out
        self._ints("n_new", n_new, n)
        self._ints("seq_lens", seq_lens, n, True)
        self._ints("seq_lens_out", lens_out, n, True)
        self._ints("free_list", free_list, self.cfg.num_pages)
        self._ints("free_count", free_count, 1, True)
        self._ints("free_count_out", count_out, 1, True)
        self._ints("cu_rows", cu_rows, n + 1, True)
        self._ints("slots", slots, rows)
        if positions is not None:
            self._ints("positions", positions, rows, True)
        if release is not None:
            self._ints("release", release, n, True)
        self._table(block_tables, n)
        dwkv_nibble_tables(self.h, n, n_new, release, seq_lens, block_tables, free_list, free_count, lens_out, count_out,
                           rows, cu_rows, positions, slots, self._stream(stream))

    def append(self, k, v, slots, pool, stream=None):
        """k, v: [rows][Hkv][d] (rows may be strided views); slots int32 [rows], -1 skips a row."""
        n, ks = self._rows("k", k, self.num_kv_heads)
        nv, vs = self._rows("v", v, self.num_kv_heads)
        if nv != n:
            raise ValueError(f"k has {n} rows and v {nv}")
        self._ints("slots", slots, n, True)
        self._pool(pool)
        dwkv_nibble_append(self.h, n, k, ks, v, vs, slots, pool, self._stream(stream))

    def read(self, slots, pool, stream=None):
        """(k, v) [rows][Hkv][d]: the stored values of the given slots."""
        n = slots.numel()
        self._ints("slots", slots, n)
        self._pool(pool)
        with _under(stream, self.device):
            k = torch.empty(n, self.num_kv_heads, self.head_dim, dtype=self.dtype, device=self.device)
            v = torch.empty_like(k)
        dwkv_nibble_read(self.h, n, slots, pool, k, v, self._stream(stream))
        return k, v

    def attention(self, q, cu_rows, seq_lens, block_tables, pool, max_q, out=None, lse=None, want_lse=False, stream=None):
        """out [rows][Hq][d] (with want_lse or lse: (out, lse), lse fp32 [rows][Hq]).  In tensors that
        are allocated here, rows that no request has are not set."""
        hq, d = self.num_q_heads, self.head_dim
        (rows, qs), n = self._rows("q", q, hq), seq_lens.numel()
        self._ints("seq_lens", seq_lens, n)
        self._ints("cu_rows", cu_rows, n + 1, True)
        self._table(block_tables, n)
        self._pool(pool)
        if out is None:
            with _under(stream, self.device):
                out = torch.empty(rows, hq, d, dtype=self.dtype, device=self.device)
        elif self._rows("out", out, hq) != (rows, hq * d):
            raise ValueError("out must be contiguous and have q's rows")
        if lse is not None:
            if lse.dtype is not torch.float32 or lse.get_device() != self.index or not lse.is_contiguous() or \
                    lse.numel() != rows * hq:
                raise ValueError(f"lse must be contiguous float32 [{rows}][{hq}] on {self.device}")
        elif want_lse:
            with _under(stream, self.device):
                lse = torch.empty(rows, hq, dtype=torch.float32, device=self.device)
        dwkv_nibble_attention(self.h, n, rows, int(max_q), q, qs, cu_rows, seq_lens, block_tables, pool, out, lse,
                              self._stream(stream))
        return out if lse is None else (out, lse)

    def sync(self, stream=None):
        """Waits for the stream and raises DwkvError if a kernel recorded an error."""
        dwkv_nibble_sync_status(self.h, self._stream(stream))


class NibbleCache:
    """A 4-bit cache of `num_layers` layers for `max_seqs` request slots: the pools, the tables
    and a handle.  step() places the rows of a step; append() and attention() then take them
    layer by layer.  The tensors are made, and cleared, on the constructor's `stream`."""

    def __init__(self, num_layers, num_q_heads, num_kv_heads, head_dim, num_pages, max_seqs, max_context, page_tokens=64,
                 max_rows=None, dtype=torch.bfloat16, window=0, softmax_scale=0.0, device="cuda", stream=None):
        blocks = -(-max_context // page_tokens)
        self.ops = Nibble(nibble_config_from(num_q_heads, num_kv_heads, head_dim, page_tokens, num_pages, max_seqs, blocks,
                                             dtype, window, softmax_scale), device, stream)
        dev = self.device = self.ops.device
        self.num_layers, self.max_seqs = num_layers, max_seqs

        def ints(*shape):
            return torch.zeros(*shape, dtype=torch.int32, device=dev)
        rows = max_rows or max_seqs
        with _under(stream, dev):
            self.pools = torch.zeros(num_layers, self.ops.pool_bytes, dtype=torch.uint8, device=dev)
            self.seq_lens, self.block_tables = ints(max_seqs), ints(max_seqs, blocks)
            self.free_list = torch.arange(num_pages, dtype=torch.int32, device=dev)
            self.free_count = torch.full((1,), num_pages, dtype=torch.int32, device=dev)
            self.cu_rows = ints(max_seqs + 1)
            self.positions, self.slots = ints(rows), ints(rows)

    def close(self):
        self.ops.close()

    def step(self, n_new, release=None, stream=None):
        """Places n_new[b] new rows of each slot (device int32 [max_seqs]); slots with release[b]
        set give their pages back first.  Rows are numbered in slot order: `positions` (for
        rotary embeddings) and `slots`, -1 behind the last row."""
        if n_new.numel() != self.max_seqs:
            raise ValueError(f"n_new must have {self.max_seqs} entries")
        self.ops.tables(n_new, self.seq_lens, self.block_tables, self.free_list, self.free_count, self.cu_rows, self.slots,
                        self.positions, release, stream=stream)

    def append(self, layer, k, v, stream=None):
        """The step's keys and values of one layer; k.shape[0] rows, at most `max_rows`."""
        self.ops.append(k, v, self.slots[:k.shape[0]], self.pools[layer], stream)

    def attention(self, layer, q, max_q, out=None, lse=None, want_lse=False, stream=None):
        """Attention of the step's rows of one layer, after its append."""
        return self.ops.attention(q, self.cu_rows, self.seq_lens, self.block_tables, self.pools[layer], max_q, out, lse,
                                  want_lse, stream)

    def read(self, layer, seq, length, stream=None):
        """(k, v) [length][Hkv][d]: the first `length` tokens of a slot, as stored."""
        p = self.ops.cfg.page_tokens
        with _under(stream, self.device):                 # after the steps on that stream, and kept for it
            t = torch.arange(length, device=self.device)
            slots = (self.block_tables[seq, t // p] * p + (t % p).to(torch.int32)).to(torch.int32)
            return self.ops.read(slots, self.pools[layer], stream)

    def sync(self, stream=None):
        self.ops.sync(stream)
