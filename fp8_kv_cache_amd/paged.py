"""The paged KV cache over torch tensors: append with norm and rotation,
attention, and gather and scatter between pages and the codec's contiguous
layer tensors (include/paged_kv.h).  torch allocates device buffers; the
library's kernels do the work.

    cache = PagedCache.empty(num_pages, 16, kv_heads=8, head_dim=128)        # BF16; or dtype=SZ_DTYPE_FP8_E5M2
    rope = Rope(rope_table(max_positions, 128))
    batch = PageBatch(page_table, cu_tokens, kv_lens, total_tokens, max_tokens, max_kv_len)
    q = append(cache, batch, k, v, q=q, rope=rope, q_norm=wq, k_norm=wk)     # keys and values into their pages
    out = attention(cache, batch, q)                                         # [tokens, q_heads, head_dim]
    k, v = gather(cache, batch)                                              # layer tensors for codec.compress
    scatter(cache, batch, k, v)

Every call is asynchronous on `stream` (default: torch's current stream of
the cache's device) and runs on the cache's device, whatever the current one
is.  Nothing here has a gradient: tensors that ask for one are refused.
`status`, an int32 tensor of one element on the same device that the caller
zeroed, becomes SZ_ERR_INVALID_ARGUMENT where a page, length or position in
device memory was out of bounds.
"""
import math

import torch

from . import (SZ_DTYPE_BF16, SZ_DTYPE_FP8_E5M2, SZ_ERR_INVALID_ARGUMENT, SzError, KvAppendArgs, KvAttentionArgs,
               KvBatch, KvCache, check, kv_append, kv_attention, kv_attention_workspace_bytes, kv_gather, kv_scatter)

_CACHE_DTYPES = {torch.bfloat16: SZ_DTYPE_BF16, torch.int16: SZ_DTYPE_BF16,
                 torch.float8_e5m2: SZ_DTYPE_FP8_E5M2, torch.uint8: SZ_DTYPE_FP8_E5M2}


def _refuse(what):
    raise SzError(SZ_ERR_INVALID_ARGUMENT, what)


class PagedCache:
    """One layer's key and value pools, each [pages, page_size, kv_heads,
    head_dim] with any strides that are multiples of 16 bytes (a transposed
    view is a head-major cache) and head_dim contiguous; BF16 or E5M2, or
    their raw words as int16 or uint8.  page_size is a power of two."""

    def __init__(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            _refuse("PagedCache: k and v want one shape [pages, page_size, kv_heads, head_dim], dtype and device")
        if k.dtype not in _CACHE_DTYPES:
            _refuse(f"PagedCache: dtype {k.dtype}")
        if k.device.type != "cuda" or k.requires_grad or v.requires_grad:
            _refuse("PagedCache: pools are device memory and have no gradient")
        strides = k.stride()
        for size, a, b in zip(k.shape, strides, v.stride()):
            if size > 1 and a != b:
                _refuse("PagedCache: k and v want the same strides")
        if k.numel() == 0 or (strides[3] != 1 and k.shape[3] > 1):
            _refuse("PagedCache: empty pools, or head_dim not contiguous")
        self.k, self.v, self.device = k, v, k.device
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.dtype = _CACHE_DTYPES[k.dtype]
        self.dtypes = tuple(t for t, d in _CACHE_DTYPES.items() if d == self.dtype)   # of its layer tensors
        # a dimension of one entry may have any stride in torch; the library looks at no offset through it
        page, token, head = (s if n > 1 else 0 for n, s in zip(k.shape[:3], strides))
        self.raw = KvCache(k.data_ptr(), v.data_ptr(), page, token, head, self.num_pages, self.page_size,
                           self.kv_heads, self.head_dim, self.dtype, 0)

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, dtype=SZ_DTYPE_BF16, device="cuda", head_major=False):
        """Pools allocated here, not initialised; head_major puts each head's
        tokens of a page together."""
        shape = (num_pages, kv_heads, page_size, head_dim) if head_major else (num_pages, page_size, kv_heads, head_dim)
        torch_dtype = torch.bfloat16 if dtype == SZ_DTYPE_BF16 else torch.float8_e5m2
        k, v = (torch.empty(shape, dtype=torch_dtype, device=device) for _ in range(2))
        return cls(k.transpose(1, 2), v.transpose(1, 2)) if head_major else cls(k, v)


class PageBatch:
    """A step's sequences: page_table int32 [seqs, pages] (rows contiguous),
    cu_tokens int32 [seqs + 1] (sequence s has the token rows cu[s] ..
    cu[s+1] - 1) and kv_lens int32 [seqs] (cached tokens, the new ones
    among them).  total_tokens is the row count of the step's tensors (rows
    from cu[-1] on are padding), max_tokens (1 or more) and max_kv_len bound
    what the device arrays hold; what is not given is read from them, which waits for
    the device.  The arrays may change between calls within those bounds."""

    def __init__(self, page_table, cu_tokens, kv_lens, total_tokens=None, max_tokens=None, max_kv_len=None):
        seqs = kv_lens.numel()
        for t in (page_table, cu_tokens, kv_lens):
            if t.dtype != torch.int32 or t.device != page_table.device or t.device.type != "cuda":
                _refuse("PageBatch: int32 tensors on one device")
        if page_table.dim() != 2 or page_table.shape[0] != seqs or cu_tokens.shape != (seqs + 1,) or kv_lens.dim() != 1:
            _refuse("PageBatch: page_table [seqs, pages], cu_tokens [seqs + 1], kv_lens [seqs]")
        if not cu_tokens.is_contiguous() or not kv_lens.is_contiguous() or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            _refuse("PageBatch: contiguous lengths and table rows")
        width = page_table.shape[1]
        if seqs > 1 and page_table.stride(0) < width:
            _refuse("PageBatch: overlapping table rows")
        if total_tokens is None:
            total_tokens = int(cu_tokens[-1])
        if max_tokens is None:
            max_tokens = max(1, int((cu_tokens[1:] - cu_tokens[:-1]).max())) if seqs else 0
        if max_kv_len is None:
            max_kv_len = int(kv_lens.max()) if seqs else 0
        for n in (total_tokens, max_tokens, max_kv_len):
            if not 0 <= n < 1 << 31:
                _refuse("PageBatch: lengths")
        self.device = page_table.device
        self.total_tokens = total_tokens
        self._keep = (page_table, cu_tokens, kv_lens)
        self.raw = KvBatch(page_table.data_ptr(), cu_tokens.data_ptr(), kv_lens.data_ptr(),
                           page_table.stride(0) if seqs > 1 else width, width, seqs, total_tokens, max_tokens,
                           max_kv_len, 0)


class Rope:
    """Rotation table: float32 [positions, rotary_dim], cos of the pairs'
    angles, then their sin (see rope_table).  Pairs are (i, i +
    rotary_dim/2), or (2i, 2i + 1) if interleaved."""

    def __init__(self, cos_sin, interleaved=False):
        if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous() or \
                cos_sin.device.type != "cuda" or cos_sin.numel() == 0 or cos_sin.requires_grad:
            _refuse("Rope: a contiguous float32 [positions, rotary_dim] table on the device")
        self.cos_sin, self.interleaved = cos_sin, bool(interleaved)
        self.positions, self.rotary_dim = cos_sin.shape
        self.raw = (cos_sin.data_ptr(), self.rotary_dim, self.positions, int(self.interleaved))


def rope_table(positions, rotary_dim, base=10000.0, device="cuda"):
    """cos and sin of p * base^(-2i / rotary_dim), computed in 64 bits (far
    positions' angles lose their last digits in 32) and rounded once."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * \
        torch.exp(i * (-2.0 * math.log(base) / rotary_dim))
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)


def _rows(name, x, tokens, heads, dim, dtypes, device):
    """Token stride of a [tokens, heads, head_dim] tensor whose heads are contiguous."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != tokens or shape[1] != heads or heads == 0 or shape[2] != dim or \
            x.dtype not in dtypes or x.device != device:
        _refuse(f"{name}: wants [{tokens}, {heads}, {dim}] of {dtypes[0]} on {device}")
    if x.requires_grad and torch.is_grad_enabled():
        _refuse(f"{name}: has no gradient here")
    t, h, d = x.stride()
    if d != 1 or (h != dim and heads > 1):
        _refuse(f"{name}: heads are not contiguous")
    return t if tokens > 1 else heads * dim


def _heads(q):
    return q.shape[1] if q.dim() == 3 else 0


def _check(cache, batch, status):
    if batch.device != cache.device:
        _refuse("the batch is on another device than the cache")
    if status is not None and (status.device != cache.device or status.dtype != torch.int32 or status.numel() < 1):
        _refuse("status: an int32 tensor on the cache's device")


# the current stream's handle on a device, without an object around it where torch has that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(call, cache, batch, stream, *args):
    """call(handle, ...) with the stream's handle.  Where the call's device is
    not the current one, or its stream is given, they are made torch's current
    ones meanwhile, so that what the call allocates belongs to them."""
    device = cache.device
    if stream is None and device.index == torch.cuda.current_device():
        return call(_raw_stream(device.index), cache, batch, *args)
    with torch.cuda.device(device):
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        elif stream.device != device:
            _refuse("the stream is on another device than the cache")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream, cache, batch, *args)


_BF16 = (torch.bfloat16, torch.int16)


def append(cache, batch, k, v, q=None, q_out=None, rope=None, q_norm=None, k_norm=None, eps=1e-6, status=None,
           stream=None):
    """Keys and values [tokens, kv_heads, head_dim] (BF16) of the batch's new
    tokens into their pages: keys normed with k_norm (BF16 [head_dim]) and
    rotated by `rope` where given, both rounded to the cache's dtype.  With q
    [tokens, q_heads, head_dim] the queries are normed with q_norm and rotated
    in the same pass, into q_out (allocated here unless given; q itself will
    do); rows of padding and of tokens that have no place are not written.
    Returns q_out, or None."""
    return _run(_append, cache, batch, stream, k, v, q, q_out, rope, q_norm, k_norm, eps, status)


def _append(stream, cache, batch, k, v, q, q_out, rope, q_norm, k_norm, eps, status):
    _check(cache, batch, status)
    n, dim, dev = batch.total_tokens, cache.head_dim, cache.device
    k_stride = _rows("k", k, n, cache.kv_heads, dim, _BF16, dev)
    v_stride = _rows("v", v, n, cache.kv_heads, dim, _BF16, dev)
    q_ptr = q_out_ptr = None
    q_stride = q_out_stride = q_heads = 0
    if q is not None:
        q_heads = _heads(q)
        q_stride = _rows("q", q, n, q_heads, dim, _BF16, dev)
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        q_out_stride = _rows("q_out", q_out, n, q_heads, dim, _BF16, dev)
        q_ptr, q_out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None or q_norm is not None:
        _refuse("append: q_out and q_norm go with q")
    for w in (q_norm, k_norm):
        if w is not None and (w.shape != (dim,) or w.dtype not in _BF16 or w.device != dev or not w.is_contiguous() or
                              (w.requires_grad and torch.is_grad_enabled())):
            _refuse(f"append: norm weights want BF16 [{dim}] on {dev}, without gradient")
    table, rotary_dim, positions, interleaved = None, 0, 0, 0
    if rope is not None:
        if rope.cos_sin.device != dev:
            _refuse("append: the rotation table is on another device")
        table, rotary_dim, positions, interleaved = rope.raw
    a = KvAppendArgs(k.data_ptr(), v.data_ptr(), q_ptr, q_out_ptr, k_stride, v_stride, q_stride, q_out_stride, table,
                     None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(), eps,
                     q_heads, rotary_dim, positions, interleaved, 0)
    check(kv_append(cache.raw, batch.raw, a, status, stream), "kv_append")
    return q_out


def attention(cache, batch, q, scale=None, causal=True, window=0, out=None, return_lse=False, workspace=None,
              status=None, stream=None):
    """Attention of the batch's new tokens (q [tokens, q_heads, head_dim],
    BF16, their keys and values appended before) over the cache.  scale
    defaults to head_dim ** -0.5.  window > 0: a token sees itself and the
    window - 1 positions before it.  Returns out (BF16, q's shape; allocated
    here unless given; q itself will do), with return_lse (out, lse float32 [tokens, q_heads]).
    Rows of padding are not written.  workspace: a uint8 tensor of
    workspace_bytes(...) that no overlapping call uses (allocated here unless
    given)."""
    return _run(_attention, cache, batch, stream, q, scale, causal, window, out, return_lse, workspace, status)


def _attention(stream, cache, batch, q, scale, causal, window, out, return_lse, workspace, status):
    _check(cache, batch, status)
    n, dim, dev, heads = batch.total_tokens, cache.head_dim, cache.device, _heads(q)
    q_stride = _rows("q", q, n, heads, dim, _BF16, dev)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    out_stride = _rows("out", out, n, heads, dim, _BF16, dev)
    if not isinstance(window, int) or not 0 <= window < 1 << 31:
        _refuse("attention: window")
    lse = torch.empty(n, heads, dtype=torch.float32, device=dev) if return_lse else None
    a = KvAttentionArgs(q.data_ptr(), out.data_ptr(), lse.data_ptr() if return_lse else None, q_stride, out_stride,
                        dim ** -0.5 if scale is None else scale, heads, bool(causal), window)
    if workspace is None:
        need = kv_attention_workspace_bytes(cache.raw, batch.raw, a)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        _refuse("attention: workspace wants contiguous uint8 on the cache's device")
    check(kv_attention(cache.raw, batch.raw, a, workspace, 0 if workspace is None else workspace.numel(), status, stream),
          "kv_attention")
    return (out, lse) if return_lse else out


def workspace_bytes(cache, batch, q_heads, window=0):
    """Bytes of workspace that attention() takes for this cache, batch and
    number of query heads (0: none)."""
    # any aligned address does for the tensors: the size query looks at shapes alone
    a = KvAttentionArgs(16, 16, None, q_heads * cache.head_dim, q_heads * cache.head_dim, 1.0, q_heads, 1, window)
    return kv_attention_workspace_bytes(cache.raw, batch.raw, a)


def gather(cache, batch, k=None, v=None, status=None, stream=None):
    """The batch's tokens out of the pages into contiguous layer tensors
    [tokens, kv_heads, head_dim] of the cache's dtype (allocated here unless
    given), the form the codec compresses; rows of padding are not written.
    Returns (k, v)."""
    return _run(_gather, cache, batch, stream, k, v, status)


def _gather(stream, cache, batch, k, v, status):
    _check(cache, batch, status)
    shape, dev, dtypes = (batch.total_tokens, cache.kv_heads, cache.head_dim), cache.device, cache.dtypes
    if k is None:
        k = torch.empty(shape, dtype=cache.k.dtype, device=dev)
    if v is None:
        v = torch.empty(shape, dtype=cache.k.dtype, device=dev)
    check(kv_gather(cache.raw, batch.raw, k, _rows("k", k, *shape, dtypes, dev), v, _rows("v", v, *shape, dtypes, dev),
                    status, stream), "kv_gather")
    return k, v


def scatter(cache, batch, k, v, status=None, stream=None):
    """Layer tensors [tokens, kv_heads, head_dim] of the cache's dtype (as
    gather made them, or the codec decoded them) into the batch's pages."""
    return _run(_scatter, cache, batch, stream, k, v, status)


def _scatter(stream, cache, batch, k, v, status):
    _check(cache, batch, status)
    shape, dev, dtypes = (batch.total_tokens, cache.kv_heads, cache.head_dim), cache.device, cache.dtypes
    check(kv_scatter(cache.raw, batch.raw, k, _rows("k", k, *shape, dtypes, dev), v, _rows("v", v, *shape, dtypes, dev),
                     status, stream), "kv_scatter")
