"""Key/value cache held in 8 bits, in pages: torch tensors on the gpt_kv8_*
calls of libgpt.so (include/gpt.h defines each of them).

``KV8Cache`` owns or wraps the buffers, ``KV8Pool`` the record of which rows
hold which pages, ``KV8Batch`` says which sequences (and how many new tokens of
each) a call is about.  Calls enqueue on the current torch stream of the
tensors' device and never wait for it; bad ids found on the device are recorded
and reported by ``status()``.

    cache = KV8Cache.empty(n_layers=12, n_pages=2048, n_kv_heads=12, head_dim=64, n_rows=32, max_pages=64)
    cache.extend(prompt_lens)                          # pages for the prompts
    batch = cache.batch(start, rows)                   # rows of sequence b: start[b] .. start[b + 1] - 1
    cache.append(layer, k, v, batch)                   # [rows, heads, head_dim]
    cache.fork(src, dst)                               # further continuations of a prompt
    one = cache.batch()                                # one new token per row
    cache.extend(ones); cache.append(layer, k, v, one); out = cache.attention(layer, q, one)
    cache.free(rows)
"""
from __future__ import annotations

import ctypes

import torch

from . import gpt as G

_KINDS = {torch.int8: G.GPT_KV8_INT8, torch.float8_e4m3fn: G.GPT_KV8_E4M3}
_NAMES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_DTYPES = {torch.bfloat16: 1, torch.float16: 2}

# the current stream's handle without the Stream object (2 of the 10 us a call takes on the host)
_stream = torch._C._cuda_getCurrentRawStream
_new = torch.empty_strided   # 1.5 us where torch.empty takes 2.4


def _i32(t, name, device, dim=1):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != dim or t.device != device:
        raise ValueError(f"{name} must be an int32 tensor with {dim} dimension(s) on {device}")
    if t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t


class KV8Batch:
    """The sequences of a call: page table [B, max_pages], tokens [B] (the
    call's own included) and, for several new tokens each, their rows' starts
    [B + 1] with the number of rows.  Holds the tensors, not copies: later
    calls see what they hold then."""

    def __init__(self, table, lens, start=None, rows=None):
        dev = table.device
        self.table, self.lens = _i32(table, "table", dev, 2), _i32(lens, "lens", dev)
        self.start = None if start is None else _i32(start, "start", dev)
        B, max_pages = table.shape
        if lens.numel() != B or (start is not None and (start.numel() != B + 1 or rows is None)):
            raise ValueError("lens must have one entry per row of table, start one more, and start needs rows")
        self.rows = B if rows is None else int(rows)
        if start is None and self.rows != B:
            raise ValueError("without start every sequence has one row")
        ld = table.stride(0) if B > 1 else max_pages
        self.c = G.gpt_kv8_batch(start=None if start is None else start.data_ptr(), lens=lens.data_ptr(),
                                 table=table.data_ptr(), B=B, max_pages=max_pages, ld_table=ld, rows=self.rows)
        self.ref = ctypes.byref(self.c)
        self.work = {}


class _Calls:
    """The plumbing of a call: device, stream and the device error word."""

    def _setup(self, device):
        if device.type != "cuda":
            raise ValueError("the tensors must be on a GPU")
        self.lib, self.device, self._index = G.load_library(), device, device.index
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self._err = self.err.data_ptr()

    def _call(self, fn, *args):
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self._index):
                rc = fn(*args, self._err, _stream(self._index))
        else:
            rc = fn(*args, self._err, _stream(self._index))
        if rc != G.GPT_OK:
            raise G.GPTError(rc, self.lib.gpt_last_error(None).decode())

    def status(self) -> int:
        """The device error word (GPT_DEVERR_* bits of include/gpt.h), which is
        cleared.  Waits for the current stream."""
        bits = int(self.err.item())
        if bits:
            self.err.zero_()
        return bits


class KV8Pool(_Calls):
    """Which pages each row holds: table [rows, max_pages], lens [rows] and ref
    [pages], int32 on the GPU; `page` tokens a page."""

    def __init__(self, table, lens, ref, page):
        dev = table.device
        _i32(table, "table", dev, 2), _i32(lens, "lens", dev), _i32(ref, "ref", dev)
        if lens.numel() != table.shape[0]:
            raise ValueError("lens must have one entry per row of table")
        self._setup(dev)
        self.table, self.lens, self.ref, self.page, self.n_pages = table, lens, ref, page, ref.numel()
        ld = table.stride(0) if table.shape[0] > 1 else table.shape[1]
        self.c = G.gpt_kv8_pool(table=table.data_ptr(), lens=lens.data_ptr(), ref=ref.data_ptr(),
                                n_rows=table.shape[0], max_pages=table.shape[1], ld_table=ld, n_pages=ref.numel(),
                                page=page)
        self._c = ctypes.byref(self.c)

    def extend(self, add):
        """Grow row r by add[r] tokens: takes pages, adds to lens."""
        if _i32(add, "add", self.device).numel() != self.lens.numel():
            raise ValueError("add must have one entry per row")
        self._call(self.lib.gpt_kv8_extend, self._c, add.data_ptr())

    def free(self, rows):
        """Empty the given rows."""
        self._call(self.lib.gpt_kv8_free, self._c, _i32(rows, "rows", self.device).data_ptr(), rows.numel())


class KV8Cache(_Calls):
    """Codes k [layers, pages, heads, page, d] and v [layers, pages, heads,
    page / 16, d, 16] (int8 or float8_e4m3fn), scales [layers, pages, heads]
    (float32) and, for the calls that keep track of pages, table [rows,
    max_pages], lens [rows] and ref [pages] (int32)."""

    def __init__(self, k, v, k_scale, v_scale, table=None, lens=None, ref=None):
        dev = k.device
        if k.dtype not in _KINDS or v.dtype != k.dtype or k.dim() != 5:
            raise ValueError("k and v must be int8 or float8_e4m3fn, k with 5 dimensions")
        L, n, h, p, d = k.shape
        if tuple(v.shape) != (L, n, h, p // 16, d, 16) or tuple(k_scale.shape) != (L, n, h) or \
                tuple(v_scale.shape) != (L, n, h):
            raise ValueError("shapes of k, v and the scales do not belong together")
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if not t.is_contiguous() or t.device != dev or dev.type != "cuda":
                raise ValueError(f"{name} must be contiguous, on the GPU that holds k")
        if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
            raise ValueError("scales must be float32")
        self._setup(dev)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_kv_heads, self.head_dim, self.page, self.n_pages = h, d, p, n
        self._shape = (h, d, p)
        self.c = G.gpt_kv8_cache(kind=_KINDS[k.dtype], n_layers=L, n_pages=n, n_kv_heads=h, head_dim=d, page=p,
                                 k=k.data_ptr(), v=v.data_ptr(), k_scale=k_scale.data_ptr(),
                                 v_scale=v_scale.data_ptr())
        self._c = ctypes.byref(self.c)
        self.table, self.lens, self.ref, self._pool = table, lens, ref, None
        if ref is not None:
            if table is None or lens is None:
                raise ValueError("ref needs table and lens beside it")
            if _i32(ref, "ref", dev).numel() != n or table.device != dev:
                raise ValueError("ref must have one entry per page, on the GPU that holds k")
            self._pool = KV8Pool(table, lens, ref, p)
            self._pool.err, self._pool._err = self.err, self._err   # one error word for both

    @classmethod
    def empty(cls, n_layers, n_pages, n_kv_heads, head_dim, page=16, kind="int8", n_rows=1, max_pages=None,
              device="cuda"):
        """A cache with all pages free and all rows empty."""
        def make(shape, dtype, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device=device) if dtype == torch.int32 else \
                torch.zeros(shape, dtype=dtype, device=device)
        if kind not in _NAMES:
            raise ValueError("kind must be int8 or e4m3")
        code = _NAMES[kind]
        shape = (n_layers, n_pages, n_kv_heads)
        return cls(make((*shape, page, head_dim), torch.uint8).view(code),
                   make((*shape, page // 16, head_dim, 16), torch.uint8).view(code),
                   make(shape, torch.float32), make(shape, torch.float32),
                   make((n_rows, max_pages or n_pages), torch.int32, -1), make((n_rows,), torch.int32),
                   make((n_pages,), torch.int32))

    def batch(self, start=None, rows=None) -> KV8Batch:
        """All rows of the cache's own table."""
        if self.table is None or self.lens is None:
            raise ValueError("this cache was made without table and lens")
        return KV8Batch(self.table, self.lens, start, rows)

    # -- plumbing
    def _rows(self, x, name, rows, heads, dtype=None):
        """(pointer, row stride) of a matrix [rows, heads, d] or [rows, heads * d]."""
        d, st = self.head_dim, x.stride()
        if x.device != self.device or x.dtype not in _DTYPES or (dtype is not None and x.dtype != dtype):
            raise ValueError(f"{name} must be bfloat16 or float16 on {self.device}, like its companions")
        if not (x.shape == (rows, heads, d) and st[2] == 1 and (heads == 1 or st[1] == d)) and \
                not (x.shape == (rows, heads * d) and st[1] == 1):
            raise ValueError(f"{name} must be [{rows}, {heads}, {d}] with the heads of a row side by side")
        return x.data_ptr(), st[0] if rows > 1 else heads * d

    def _batch(self, batch):
        if batch is None:
            batch = self.batch()
        if batch.table.device != self.device:
            raise ValueError(f"the batch must be on {self.device}")
        return batch

    @property
    def pool(self) -> KV8Pool:
        if self._pool is None:
            raise ValueError("this cache was made without table, lens and ref")
        return self._pool

    # -- one layer
    def append(self, layer, k, v, batch=None):
        """Quantise new keys and values [rows, heads, head_dim] into the pages."""
        b = self._batch(batch)
        pk, ldk = self._rows(k, "k", b.rows, self.n_kv_heads)
        pv, ldv = self._rows(v, "v", b.rows, self.n_kv_heads, k.dtype)
        self._call(self.lib.gpt_kv8_append, self._c, layer, b.ref, pk, ldk, pv, ldv, _DTYPES[k.dtype])

    def read(self, layer, batch=None, dtype=torch.bfloat16):
        """(k, v) [rows, heads, head_dim]: what the cache holds of the batch's
        tokens.  Rows without a token in the cache are not written."""
        b = self._batch(batch)
        if dtype not in _DTYPES:
            raise ValueError("dtype must be bfloat16 or float16")
        h, d = self.n_kv_heads, self.head_dim
        ld = h * d
        k = _new((b.rows, h, d), (ld, d, 1), dtype=dtype, device=self.device)
        v = torch.empty_like(k)
        self._call(self.lib.gpt_kv8_read, self._c, layer, b.ref, k.data_ptr(), ld, v.data_ptr(), ld, _DTYPES[dtype])
        return k, v

    def attention(self, layer, q, batch=None, scale=None, out=None, return_lse=False):
        """Attention of the newest queries [rows, n_heads, head_dim] over the
        cache (scale: head_dim ** -0.5 unless given); with return_lse also the
        natural log of the softmax denominators [rows, n_heads]."""
        b = self._batch(batch)
        d, dev = self.head_dim, self.device
        if q.dim() not in (2, 3):
            raise ValueError("q must be [rows, n_heads, head_dim] or [rows, n_heads * head_dim]")
        H = q.shape[1] if q.dim() == 3 else q.shape[1] // d
        pq, ldq = self._rows(q, "q", b.rows, H)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            po, ldo = out.data_ptr(), H * d
        else:
            po, ldo = self._rows(out, "out", b.rows, H, q.dtype)
        lse = _new((b.rows, H), (H, 1), dtype=torch.float32, device=dev) if return_lse else None
        n = b.work.get((self._shape, H))
        if n is None:
            n = b.work[self._shape, H] = self._work(b, H)
        work = _new((n,), (1,), dtype=torch.uint8, device=dev) if n else None
        self._call(self.lib.gpt_kv8_attention, self._c, layer, b.ref, pq, ldq, H, _DTYPES[q.dtype],
                   d ** -0.5 if scale is None else scale, po, ldo, lse.data_ptr() if return_lse else None,
                   work.data_ptr() if n else None, n)
        return (out, lse) if return_lse else out

    def _work(self, b, H):
        need = ctypes.c_size_t()
        with torch.cuda.device(self._index):   # the scratch depends on the device's SMs
            rc = self.lib.gpt_kv8_attention_work(self._c, b.ref, H, ctypes.byref(need))
        if rc != G.GPT_OK:
            raise G.GPTError(rc, self.lib.gpt_last_error(None).decode())
        return need.value

    # -- pages
    def extend(self, add):
        """Grow row r by add[r] tokens: takes pages, adds to lens."""
        self.pool.extend(add)

    def free(self, rows):
        """Empty the given rows."""
        self.pool.free(rows)

    def fork(self, src, dst):
        """Rows dst (empty) become copies of rows src; returns int32 [n], 1
        where the fork was made."""
        n = _i32(src, "src", self.device).numel()
        if _i32(dst, "dst", self.device).numel() != n:
            raise ValueError("src and dst must have the same length")
        done = _new((n,), (1,), dtype=torch.int32, device=self.device)
        self._call(self.lib.gpt_kv8_fork, self.pool._c, self._c, src.data_ptr(), dst.data_ptr(), n, done.data_ptr())
        return done

    def compact(self):
        """Move the pages in use to the front; returns their number (a tensor)."""
        n = _new((), (), dtype=torch.int64, device=self.device)
        work = _new((2 * self.n_pages + 8,), (1,), dtype=torch.int32, device=self.device)
        self._call(self.lib.gpt_kv8_compact, self.pool._c, self._c, n.data_ptr(), work.data_ptr())
        return n
