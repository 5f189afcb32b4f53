"""One attention layer's decode step over a paged cache that is kept to a budget.

A server that holds many sequences of unequal length keeps a layer's K/V cache in
pages, and bounds it: positions that gathered little attention leave it.  One
step for one new token per sequence is the library's paged decode path in order
(include/hs2.h, "paged decode path"):

  1. hs2_add_rmsnorm   the residual's addition, the norm, its output in E4M3
  2. hs2_fp8_gemm      the token's queries, and its K and V rows
  3. hs2_paged_append  the rows to their pages
  4. hs2_paged_attn    attention over the pages, weights accumulated
  5. hs2_paged_evict   every `interval` steps: down to topk + window positions

This module is the orchestration only: buffers, pages and the order of the calls.
All arithmetic runs in the library's kernels; the weights are packed once, with
torch, when a layer is made.
"""

from dataclasses import dataclass

import torch

from . import (HS2_KV_BF16, HS2_KV_FP8_E4M3, hs2_add_rmsnorm, hs2_fp8_gemm, hs2_paged_append,
               hs2_paged_attn, hs2_paged_attn_workspace, hs2_paged_evict, paged_cache)

E4M3 = torch.float8_e4m3fn


def pack_weight(w):
    """E4M3 codes of a weight [N, K] and their fp32 scales per block of 128 x 128."""
    N, K = w.shape
    x = torch.nn.functional.pad(w.float(), (0, -K % 128, 0, -N % 128))
    x = x.view(x.shape[0] // 128, 128, x.shape[1] // 128, 128)
    s = x.abs().amax((1, 3)) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    codes = (x / s[:, None, :, None]).to(E4M3).view(x.shape[0] * 128, x.shape[2] * 128)
    return codes[:N, :K].contiguous(), s.contiguous()


@dataclass
class PagedConfig:
    B: int                  # sequences
    hidden: int             # a multiple of 16
    H: int                  # query heads
    kv_heads: int
    D: int                  # 64 or 128
    fp8: bool = True        # an E4M3 cache
    page_size: int = 64     # a power of two
    topk: int = 1024        # heaviest positions kept outside the window
    window: int = 128       # most recent positions kept
    interval: int = 64      # steps between two evictions
    eps: float = 1e-6

    @property
    def pages_per_sequence(self) -> int:
        return -(-(self.topk + self.window + self.interval) // self.page_size)


class PagedLayer:
    """The layer's weights, pages and buffers on the current device.  step() may be
    captured into a CUDA graph (once for a step without eviction and once for one
    with it); lengths live on the device.  `steps` counts the calls of step(), not a
    graph's replays: whoever replays keeps the count, and replays the step with the
    eviction once `interval` steps have passed."""

    def __init__(self, cfg: PagedConfig, gamma, w_q, w_kv):
        """gamma [hidden], w_q [H * D, hidden], w_kv [2 * kv_heads * D, hidden] (K rows, then
        V rows), bf16 on the device."""
        c, dev = cfg, gamma.device
        self.cfg, self.gamma = cfg, gamma
        self.w_q, self.w_q_scale = pack_weight(w_q)
        self.w_kv, self.w_kv_scale = pack_weight(w_kv)
        n = c.B * c.pages_per_sequence
        pool = (n, c.page_size, c.kv_heads)
        kv_type = torch.uint8 if c.fp8 else torch.bfloat16
        self.k, self.v = (torch.zeros(*pool, c.D, dtype=kv_type, device=dev) for _ in range(2))
        self.k_scale, self.v_scale = ((torch.ones(pool, device=dev) if c.fp8 else None)
                                      for _ in range(2))
        self.weight = torch.zeros(pool[:2], device=dev)
        self.table = torch.arange(n, dtype=torch.int32, device=dev).view(c.B, -1)
        self.seq_len = torch.zeros(c.B, dtype=torch.int32, device=dev)
        self.cache = paged_cache(self.k, self.v, self.table, self.seq_len, self.k_scale,
                                 self.v_scale, self.weight)
        self.dt = HS2_KV_FP8_E4M3 if c.fp8 else HS2_KV_BF16
        bf16 = dict(dtype=torch.bfloat16, device=dev)
        self.codes = torch.empty(c.B, c.hidden, dtype=E4M3, device=dev)
        self.codes_scale = torch.empty(c.B, -(-c.hidden // 128), device=dev)
        self.q = torch.empty(c.B, c.H, c.D, **bf16)
        self.kv = torch.empty(c.B, 2, c.kv_heads * c.D, **bf16)
        self.out = torch.empty(c.B, c.H, c.D, **bf16)
        self.lse = torch.empty(c.B, c.H, device=dev)
        self.kept = torch.empty(c.B, c.topk + c.window, dtype=torch.int32, device=dev)
        self.ws = torch.empty(hs2_paged_attn_workspace(c.B, c.H, c.kv_heads, c.D),
                              dtype=torch.uint8, device=dev)
        self.steps = 0              # since the last eviction

    def step(self, x, residual):
        """x: the layer's input [B, hidden] bf16; residual [B, hidden] bf16, to which x is added
        in place.  Returns the attention's output [B, H, D] bf16 (the layer's own buffer)."""
        c = self.cfg
        if self.steps == c.interval:
            hs2_paged_evict(self.cache, c.B, c.kv_heads, c.D, self.dt, c.topk, c.window, None,
                            self.kept, self.seq_len)
            self.steps = 0
        self.seq_len += 1
        self.steps += 1
        hs2_add_rmsnorm(x, residual, self.gamma, c.B, c.hidden, c.eps, residual, None, self.codes,
                        self.codes_scale)
        hs2_fp8_gemm(self.codes, self.codes_scale, c.B, self.w_q, self.w_q_scale, c.H * c.D,
                     c.hidden, self.q)
        hs2_fp8_gemm(self.codes, self.codes_scale, c.B, self.w_kv, self.w_kv_scale,
                     2 * c.kv_heads * c.D, c.hidden, self.kv)
        hs2_paged_append(self.kv[:, 0], self.kv[:, 1], self.kv.stride(0), c.B, None, self.cache,
                         c.B, c.kv_heads, c.D, self.dt)
        hs2_paged_attn(self.q, self.cache, c.B, c.H, c.kv_heads, c.D, c.D ** -0.5, self.dt,
                       self.out, self.lse, True, self.ws, self.ws.numel())
        return self.out
