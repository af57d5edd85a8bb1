"""``KVCache`` and ``flash_attention_kvcache``: answering with a trained model.

The framework-level API on the C ABI's quantised, paged key/value cache, next
to ``attention.flash_attention`` for training: keys and values of the tokens so
far live in pages of 8-bit codes with one fp32 scale per token and head, and
the newest tokens attend to them there.  Forward only.  torch supplies memory
and streams; every step runs in the CUDA library.

    cache = KVCache(num_pages, num_kv_heads, head_dim, page_size=64, dtype=torch.int8)
    cache.append(k, v, block_table, lens)                     # one new token per sequence
    o = flash_attention_kvcache(q, cache, block_table, lens + 1)

Calls are asynchronous on the current stream (or ``stream``) of the cache's
device and may be captured into a CUDA graph: lengths, block tables and the
cache's contents are read on the device at replay.
"""
from __future__ import annotations

import torch

from . import binding


class KVCache:
    """Quantised, paged keys and values: codes ``k``, ``v`` [num_pages, num_kv_heads, page_size, head_dim] and fp32
    ``k_scale``, ``v_scale`` [num_pages, num_kv_heads, page_size].

    ``dtype`` is torch.int8 (code = rint(127 x / amax)) or torch.float8_e4m3fn (code = 448 x / amax); a code stands
    for code * scale, with one scale per token and head.  page_size is 16, 32, 64 or 128, head_dim 64 or 128.  Which
    page holds what is the caller's: sequence b's position p is slot p % page_size of page
    ``block_table[b, p // page_size]`` (int32 [B, max_pages] on the device).
    """

    def __init__(self, num_pages: int, num_kv_heads: int, head_dim: int, page_size: int = 64, dtype=torch.int8,
                 device="cuda"):
        if dtype not in binding.KV_FORMATS:
            raise ValueError("dtype is torch.int8 or torch.float8_e4m3fn")
        if page_size not in (16, 32, 64, 128):
            raise ValueError("page_size is 16, 32, 64 or 128")
        if head_dim not in (64, 128):
            raise ValueError("head_dim is 64 or 128")
        if num_pages < 1 or num_kv_heads < 1:
            raise ValueError("num_pages and num_kv_heads are at least 1")
        shape = (num_pages, num_kv_heads, page_size)
        k, v = (torch.zeros((*shape, head_dim), dtype=torch.int8, device=device).view(dtype) for _ in range(2))
        ks, vs = (torch.zeros(shape, dtype=torch.float32, device=device) for _ in range(2))
        self.buffers = binding.KvBuffers(k, v, ks, vs)

    @classmethod
    def from_tensors(cls, k, v, k_scale, v_scale) -> "KVCache":
        """A cache over existing buffers (one layer of a larger allocation, say), which it shares."""
        self = cls.__new__(cls)
        self.buffers = binding.KvBuffers(k, v, k_scale, v_scale)
        return self

    k = property(lambda self: self.buffers.tensors[0])
    v = property(lambda self: self.buffers.tensors[1])
    k_scale = property(lambda self: self.buffers.tensors[2])
    v_scale = property(lambda self: self.buffers.tensors[3])
    num_pages = property(lambda self: self.buffers.num_pages)
    num_kv_heads = property(lambda self: self.buffers.num_kv_heads)
    page_size = property(lambda self: self.buffers.page_size)
    head_dim = property(lambda self: self.buffers.d)
    dtype = property(lambda self: self.k.dtype)
    device = property(lambda self: self.buffers.device)

    def append(self, k, v, block_table, starts=None, cu_seqlens=None, stream=None) -> None:
        """Quantise new keys and values into the cache.

        k, v: bf16 [T, num_kv_heads, head_dim].  Without ``cu_seqlens`` there is one token per sequence (T = B); with
        it (int32 [B + 1]) sequence b's tokens are rows cu_seqlens[b] to cu_seqlens[b + 1].  They go to positions
        starts[b], starts[b] + 1, ... (int32 [B]; None: from 0).  Sequences may share pages, but not the slots written
        here.  No gradients: k and v that require one are refused, as q is in attention.
        """
        if (k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
            raise ValueError("KVCache.append has no backward: detach k and v or use torch.no_grad()")
        binding.kv_append(self.buffers, k, v, block_table, starts, cu_seqlens, stream)

    def read(self, block_table, cu_seqlens, total_tokens: int, starts=None, stream=None):
        """The cached keys and values as bf16 [total_tokens, num_kv_heads, head_dim]: row cu_seqlens[b] + i holds
        position starts[b] + i of sequence b (None: from 0).  Rows at or past cu_seqlens[B] are not written."""
        return binding.kv_read(self.buffers, block_table, total_tokens, starts, cu_seqlens, stream=stream)


def flash_attention_kvcache(q, cache: KVCache, block_table, seqlens, cu_seqlens_q=None, max_seqlen_q: int | None = None,
                            causal: bool = True, scale: float | None = None, prefix_len: int = 0,
                            return_lse: bool = False, workspace=None, stream=None):
    """Exact attention of each sequence's newest tokens over its cached keys and values.

    q: bf16, (batch, new tokens, query heads, head_dim), or token-major (T, query heads, head_dim) with
    ``cu_seqlens_q`` (int32 [B + 1]) and ``max_seqlen_q`` (at least the most queries of a sequence) for a ragged
    batch; a (batch, query heads, head_dim) q without ``cu_seqlens_q`` is one token per sequence.  Rows of no sequence,
    and those of a sequence past ``max_seqlen_q`` (an error in ``binding.device_error()``), are not written: what o and
    the logsumexp hold there is not defined.  The query heads are
    a multiple of the cache's heads; query head h reads key head h // (query heads / key heads).
    ``seqlens`` (int32 [B]) counts each sequence's keys, the new tokens' own included (append them first).  When
    ``causal``, query i of L sees keys j < seqlens[b] - L + i + 1.  A query that sees no key gets zeros.

    How the work is done follows from the longest sequence's rows, max_seqlen_q * query heads / key heads: a prompt's
    chunk among sequences of one token is faster as a call of its own beside theirs.

    ``prefix_len`` > 0 (a multiple of the page size) says that all sequences begin with the same prefix_len keys, in
    the pages of block_table's first row: they are then read once for the batch.  The result is the same.

    Returns o like q, and with ``return_lse`` the fp32 logsumexp [query heads, T] (-inf where no key is seen).
    ``workspace`` (a CUDA tensor of at least ``binding.fwd_kvcache_workspace_size`` bytes) is allocated if not given.
    No gradients.
    """
    ctx = binding._other_stream(cache.buffers, stream)
    if ctx is not None:
        with ctx:
            return flash_attention_kvcache(q, cache, block_table, seqlens, cu_seqlens_q, max_seqlen_q, causal, scale,
                                           prefix_len, return_lse, workspace)
    if q.requires_grad and torch.is_grad_enabled():
        raise ValueError("flash_attention_kvcache has no backward: detach q or use torch.no_grad()")
    dim = q.dim()
    if dim == 4:
        if cu_seqlens_q is not None:
            raise ValueError("q with cu_seqlens_q is token-major: [T, Hq, d]")
        if max_seqlen_q is not None and max_seqlen_q != q.shape[1]:
            raise ValueError("max_seqlen_q is q's second dimension")
        shape = q.shape
        max_seqlen_q = shape[1]
        q = q.flatten(0, 1)
    elif dim != 3:
        raise ValueError("q is (batch, new tokens, heads, head_dim) or (T, heads, head_dim)")
    elif max_seqlen_q is None:
        if cu_seqlens_q is not None:
            raise ValueError("cu_seqlens_q needs max_seqlen_q")
        max_seqlen_q = 1
    o, lse = binding.fwd_kvcache(q, cache.buffers, block_table, seqlens, int(max_seqlen_q),
                                 cu_seqlens_q=cu_seqlens_q, causal=causal, scale=scale, prefix_len=int(prefix_len),
                                 want_lse=return_lse, workspace=workspace)
    if dim == 4:
        o = o.view(shape)
    return (o, lse) if return_lse else o
