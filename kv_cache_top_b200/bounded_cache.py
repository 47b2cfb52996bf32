"""A decode cache of a bounded number of tokens, held in 4 bits.

DecodeCache keeps every token and searches the old ones; this one keeps a
quarter of the bf16 bytes of the tokens that attention has looked at, attends
all of them, and drops the others.  It is written on the library's C-ABI
(pk_quant_append, pk_quant_attend, pk_quant_evict): quantisation, attention
and eviction run in the library's kernels.

Every (sequence, KV head) pair holds between `budget` and `budget + update`
tokens: the first `sink`, the last `recent`, and between them those whose
accumulated attention weight (summed over the pair's query heads and over the
queries since they came in) is largest.  A step that finds `budget + update`
tokens evicts down to `budget` first, into a second buffer, and the buffers
swap; pairs choose their tokens separately.  The order of the tokens is kept.

The kernels record what they find wrong on the GPU (a length out of range, rows
that do not fit, a copy that did not arrive) in a status word; a step does not
wait for it, check() reads it.

A longer prompt comes in whole: until the first step its tokens are all there,
and observe() lets queries of the prompt's end add their weights without adding
a token, so that the first eviction has something to go by.
"""
from __future__ import annotations

import math

import torch

from . import (PK_BF16, PK_F32, PK_OK, PK_QUANT_BLOCK_BYTES, PK_QUANT_KEYS, PkError, pk_quant_append, pk_quant_attend,
               pk_quant_attend_workspace, pk_quant_evict, pk_quant_rows, pk_quant_view)


class BoundedCache:
    """K, V: the prompt [batch][H][T0][D], bf16 or fp32, on the GPU.  scale: the
    softmax scale (0: 1/sqrt(D))."""

    def __init__(self, K, V, *, group: int, budget: int, sink: int = 64, recent: int = 512, update: int = 512,
                 scale: float = 0.0):
        if K.dim() != 4 or K.shape != V.shape or K.shape[-1] != 128 or K.dtype != V.dtype:
            raise ValueError("K and V must be [batch][H][T0][128] of one type")
        if K.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("K and V must be bf16 or fp32")
        if sink < 0 or recent < 0 or sink + recent > budget or budget < 1 or update < 1 or not 1 <= group <= 8:
            raise ValueError("need 0 <= sink, recent; sink + recent <= budget; update >= 1; 1 <= group <= 8")
        if not 0 <= scale < math.inf:
            raise ValueError("scale must be 0 or a finite positive number")
        self.batch, self.H, T0, self.D = K.shape
        self.G, self.budget, self.sink, self.recent, self.update = group, budget, sink, recent, update
        self.scale, self.dtype, self.device = scale, K.dtype, K.device
        self.kind = PK_BF16 if K.dtype == torch.bfloat16 else PK_F32
        self.bh = self.batch * self.H
        self.limit = budget + update
        self.T = T0                                       # tokens seen
        self.n = T0                                       # tokens held per pair
        self.evictions = 0
        cap = max(T0, self.limit)
        self._status = torch.zeros(2, dtype=torch.int32, device=self.device)     # of both buffers, whichever is in use
        self._cache, self._pos = self._buffers(cap)
        self._other = None                                # the second buffer, made at the first eviction
        self.out = torch.empty(self.batch, self.H * group, self.D, dtype=torch.float32, device=self.device)
        self.lse = torch.empty(self.batch, self.H * group, dtype=torch.float32, device=self.device)
        self._work = self._workspace(self._cache)
        self._keep = torch.empty(self.bh, budget, dtype=torch.int32, device=self.device)
        if T0:
            pk_quant_append(self._cache, K.contiguous(), V.contiguous(), T0)
            self._pos[:, :T0] = torch.arange(T0, device=self.device)

    def _buffers(self, tokens):
        m = -(-tokens // PK_QUANT_KEYS)
        dev = self.device
        cache = pk_quant_view(torch.empty(self.bh, m, PK_QUANT_BLOCK_BYTES, dtype=torch.uint8, device=dev),
                              torch.zeros(self.bh, dtype=torch.int32, device=dev), self.kind,
                              acc=torch.zeros(self.bh, m * PK_QUANT_KEYS, device=dev),
                              status=self._status)
        return cache, torch.zeros(self.bh, m * PK_QUANT_KEYS, dtype=torch.int64, device=dev)

    def _workspace(self, cache):
        return torch.empty(pk_quant_attend_workspace(cache, self.G, True), dtype=torch.uint8, device=self.device)

    @property
    def positions(self):
        """[batch][H][n]: the positions of the tokens held, ascending."""
        return self._pos[:, :self.n].view(self.batch, self.H, self.n)

    @property
    def weights(self):
        """[batch][H][n]: their accumulated attention weights."""
        return self._cache.tensors[2][:, :self.n].view(self.batch, self.H, self.n)

    def rows(self):
        """The values of the tokens held: K, V [batch][H][n][D]."""
        k, v = (torch.empty(self.batch, self.H, self.n, self.D, dtype=self.dtype, device=self.device) for _ in range(2))
        if self.n:
            pk_quant_rows(self._cache, self.n, k, v)
        return k, v

    def check(self):
        """Wait for the calls so far on the current stream and raise PkError if
        one of them recorded a failure on the GPU: results since the last check
        may then be wrong.  The record is cleared."""
        status, pair = self._status.tolist()
        if status != PK_OK:
            self._status.zero_()
            raise PkError(status, "BoundedCache: pair %d" % pair)

    def _check(self, name, t, shape):
        if t.shape != shape or t.dtype != self.dtype or (t.device != self.device and not t.is_pinned()):
            raise ValueError("%s must be %s of the cache's type, on its device or in pinned memory" % (name, list(shape)))

    def evict(self):
        """Drop to `budget` tokens per pair (nothing if there are no more)."""
        if self.n <= self.budget:
            return
        if self._other is None:
            self._other = self._buffers(self.limit)
        dst, pos = self._other
        pk_quant_evict(self._cache, dst, self.budget, sink=self.sink, recent=self.recent, keep=self._keep)
        torch.gather(self._pos, 1, self._keep.long(), out=pos[:, :self.budget])
        small = self._cache.n_cap == dst.n_cap            # a longer prompt's buffer and workspace are not needed again
        if small:
            self._other = (self._cache, self._pos)
        else:
            self._other = None
            work, self._work = self._work, self._workspace(dst)
            for t in (*self._cache.tensors[:3], self._pos, work):     # the current stream may not be the one they were made on
                t.record_stream(torch.cuda.current_stream())
        self._cache, self._pos = dst, pos
        self.n = self.budget
        self.evictions += 1

    def observe(self, q):
        """Attend q [batch][H*G][D] over the tokens held and add the weights,
        without adding a token.  Returns the output [batch][H*G][D] fp32 (a
        buffer reused by the next call); lse holds the log-sums."""
        self._check("q", q, self.out.shape)
        pk_quant_attend(self._cache, q.contiguous(), self.G, self.out, self._work, lse=self.lse, accumulate=True, scale=self.scale)
        return self.out

    def step(self, q, k_new, v_new):
        """One decode step: evict if the buffer is full, add the token k_new,
        v_new [batch][H][1][D], and attend q over every token held.  Everything
        runs on torch's current stream, in order.  A step that is refused
        changes nothing."""
        self._check("q", q, self.out.shape)
        for name, t in (("k_new", k_new), ("v_new", v_new)):
            self._check(name, t, (self.batch, self.H, 1, self.D))
        if self.n >= self.limit:
            self.evict()
        pk_quant_append(self._cache, k_new.contiguous(), v_new.contiguous(), 1)
        self._pos[:, self.n] = self.T
        self.n += 1
        self.T += 1
        return self.observe(q)
