"""Key/value cache held in 8 bits, in pages: torch tensors on the gpt_kv8_*
calls of libgpt.so (include/gpt.h defines each of them).

``KV8Cache`` owns or wraps the buffers, ``KV8Batch`` says which sequences (and
how many new tokens of each) a call is about.  Calls enqueue on the current
torch stream of the cache's device and never wait for it; bad ids found on the
device are recorded and reported by ``KV8Cache.status()``.

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


class KV8Cache:
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
        self.lib = G.load_library()
        self.device = dev
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_kv_heads, self.head_dim, self.page, self.n_pages = h, d, p, n
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.c = G.gpt_kv8_cache(kind=_KINDS[k.dtype], n_layers=L, n_pages=n, n_kv_heads=h, head_dim=d, page=p,
                                 k=k.data_ptr(), v=v.data_ptr(), k_scale=k_scale.data_ptr(),
                                 v_scale=v_scale.data_ptr())
        self._c, self._err = ctypes.byref(self.c), self.err.data_ptr()
        self.table, self.lens, self.ref, self._pool = table, lens, ref, None
        if ref is not None:
            _i32(table, "table", dev, 2), _i32(lens, "lens", dev), _i32(ref, "ref", dev)
            if lens.numel() != table.shape[0] or ref.numel() != n:
                raise ValueError("lens must have one entry per row of table, ref one per page")
            ld = table.stride(0) if table.shape[0] > 1 else table.shape[1]
            self.pool = G.gpt_kv8_pool(table=table.data_ptr(), lens=lens.data_ptr(), ref=ref.data_ptr(),
                                       n_rows=table.shape[0], max_pages=table.shape[1], ld_table=ld, n_pages=n, page=p)
            self._pool = ctypes.byref(self.pool)

    @classmethod
    def empty(cls, n_layers, n_pages, n_kv_heads, head_dim, page=16, kind="int8", n_rows=1, max_pages=None,
              device="cuda"):
        """A cache with all pages free and all rows empty."""
        def make(shape, dtype, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device=device) if dtype == torch.int32 else \
                torch.zeros(shape, dtype=dtype, device=device)
        code = _NAMES[kind]
        shape = (n_layers, n_pages, n_kv_heads)
        return cls(make((*shape, page, head_dim), torch.uint8).view(code),
                   make((*shape, page // 16, head_dim, 16), torch.uint8).view(code),
                   make(shape, torch.float32), make(shape, torch.float32),
                   make((n_rows, max_pages or n_pages), torch.int32, -1), make((n_rows,), torch.int32),
                   make((n_pages,), torch.int32))

    def batch(self, start=None, rows=None) -> KV8Batch:
        """All rows of the cache's own table."""
        return KV8Batch(self.table, self.lens, start, rows)

    # -- plumbing
    def _call(self, name, *args):
        dev = self.device
        fn = getattr(self.lib, name)
        if torch.cuda.current_device() != dev.index:
            with torch.cuda.device(dev):
                rc = fn(*args, self._err, torch.cuda.current_stream(dev).cuda_stream)
        else:
            rc = fn(*args, self._err, torch.cuda.current_stream(dev).cuda_stream)
        if rc != G.GPT_OK:
            raise G.GPTError(rc, self.lib.gpt_last_error(None).decode())

    def _rows(self, x, name, batch, heads, dtype=None):
        """(pointer, row stride) of a matrix [rows, heads, d] or [rows, heads * d]."""
        d = self.head_dim
        if x.device != self.device or x.dtype not in _DTYPES or (dtype is not None and x.dtype != dtype):
            raise ValueError(f"{name} must be bfloat16 or float16 on {self.device}, like its companions")
        if x.dim() == 3:
            ok = x.shape[1] == heads and x.shape[2] == d and x.stride(2) == 1 and (heads == 1 or x.stride(1) == d)
        else:
            ok = x.dim() == 2 and x.shape[1] == heads * d and x.stride(1) == 1
        if not ok or x.shape[0] != batch.rows:
            raise ValueError(f"{name} must be [{batch.rows}, {heads}, {d}] with the heads of a row side by side")
        return x.data_ptr(), x.stride(0) if batch.rows > 1 else heads * d

    def _batch(self, batch):
        if batch is None:
            batch = self.batch()
        if batch.table.device != self.device:
            raise ValueError(f"the batch must be on {self.device}")
        return batch

    def _needs_pool(self):
        if self._pool is None:
            raise ValueError("this cache was made without table, lens and ref")

    # -- one layer
    def append(self, layer, k, v, batch=None):
        """Quantise new keys and values [rows, heads, head_dim] into the pages."""
        b = self._batch(batch)
        pk, ldk = self._rows(k, "k", b, self.n_kv_heads)
        pv, ldv = self._rows(v, "v", b, self.n_kv_heads, k.dtype)
        self._call("gpt_kv8_append", self._c, layer, b.ref, pk, ldk, pv, ldv, _DTYPES[k.dtype])

    def read(self, layer, batch=None, dtype=torch.bfloat16):
        """(k, v) [rows, heads, head_dim]: what the cache holds of the batch's
        tokens.  Rows without a token in the cache are not written."""
        b = self._batch(batch)
        k = torch.empty(b.rows, self.n_kv_heads, self.head_dim, dtype=dtype, device=self.device)
        v = torch.empty_like(k)
        pk, ldk = self._rows(k, "k", b, self.n_kv_heads)
        pv, ldv = self._rows(v, "v", b, self.n_kv_heads)
        self._call("gpt_kv8_read", self._c, layer, b.ref, pk, ldk, pv, ldv, _DTYPES[dtype])
        return k, v

    def attention(self, layer, q, batch=None, scale=None, out=None, return_lse=False):
        """Attention of the newest queries [rows, n_heads, head_dim] over the
        cache (scale: head_dim ** -0.5 unless given); with return_lse also the
        natural log of the softmax denominators [rows, n_heads]."""
        b = self._batch(batch)
        H = q.shape[1] if q.dim() == 3 else q.shape[1] // self.head_dim
        if H < 1 or H % self.n_kv_heads:
            raise ValueError("the number of query heads must be a multiple of the cache's heads")
        pq, ldq = self._rows(q, "q", b, H)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        po, ldo = self._rows(out, "out", b, H, q.dtype)
        lse = torch.empty(b.rows, H, dtype=torch.float32, device=self.device) if return_lse else None
        key = (H, self.n_kv_heads, self.head_dim, self.page)
        n = b.work.get(key)
        if n is None:
            need = ctypes.c_size_t()
            if self.lib.gpt_kv8_attention_work(self._c, b.ref, H, ctypes.byref(need)) != G.GPT_OK:
                raise G.GPTError(G.GPT_ERR_ARG, self.lib.gpt_last_error(None).decode())
            n = b.work[key] = need.value
        work = torch.empty(n, dtype=torch.uint8, device=self.device) if n else None
        self._call("gpt_kv8_attention", self._c, layer, b.ref, pq, ldq, H, _DTYPES[q.dtype],
                   self.head_dim ** -0.5 if scale is None else scale, po, ldo,
                   None if lse is None else lse.data_ptr(), None if work is None else work.data_ptr(), n)
        return (out, lse) if return_lse else out

    # -- pages
    def extend(self, add):
        """Grow row r by add[r] tokens: takes pages, adds to lens."""
        self._needs_pool()
        if _i32(add, "add", self.device).numel() != self.lens.numel():
            raise ValueError("add must have one entry per row")
        self._call("gpt_kv8_extend", self._pool, add.data_ptr())

    def fork(self, src, dst):
        """Rows dst (empty) become copies of rows src; returns int32 [n], 1
        where the fork was made."""
        self._needs_pool()
        n = _i32(src, "src", self.device).numel()
        if _i32(dst, "dst", self.device).numel() != n:
            raise ValueError("src and dst must have the same length")
        done = torch.empty(n, dtype=torch.int32, device=self.device)
        self._call("gpt_kv8_fork", self._pool, self._c, src.data_ptr(), dst.data_ptr(), n, done.data_ptr())
        return done

    def free(self, rows):
        """Empty the given rows."""
        self._needs_pool()
        self._call("gpt_kv8_free", self._pool, _i32(rows, "rows", self.device).data_ptr(), rows.numel())

    def compact(self):
        """Move the pages in use to the front; returns their number (int32 [1])."""
        self._needs_pool()
        n = torch.empty(1, dtype=torch.int32, device=self.device)
        work = torch.empty(2 * self.n_pages + 8, dtype=torch.int32, device=self.device)
        self._call("gpt_kv8_compact", self._pool, self._c, n.data_ptr(), work.data_ptr())
        return n

    def status(self) -> int:
        """The device error word (GPT_DEVERR_* bits of include/gpt.h), which is
        cleared.  Waits for the current stream."""
        bits = int(self.err.item())
        if bits:
            self.err.zero_()
        return bits
