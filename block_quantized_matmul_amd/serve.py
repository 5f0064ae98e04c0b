"""The attention block of a decoder layer, served for a batch of conversations
behind one shared prompt, from the library's serving operators:

  e4m3 of the activations (lqmm_quant_f8b128) -> q, k, v in one product
  (lqmm_gemm_f8b128) -> rotation and append to the paged cache
  (lqmm_kv_append) -> attention, the shared prompt's keys read once for the
  whole batch (lqmm_attn_prefix) -> e4m3 -> output product.

Each half has a form in fewer bits: weight_bits=4 takes the products from
microscaled 4-bit floats (lqmm_quant_mxfp4, lqmm_gemm_mxfp4), kv_bits=8 keeps
the cache as e4m3 codes (lqmm_kv_append_norm, lqmm_attn_prefix_f8, and
lqmm_kv_read_f8 for what it holds); q_norm and k_norm normalize the heads of q
and k before the rotation (lqmm_kv_append_norm).

The caches, tables and lengths are device tensors made when the block is built,
and a step reads its lengths and pages from them, so that one captured HIP graph
serves every later step behind a prompt of the same length. What a step computes
(codes, scales, products, outputs, the attention's workspace) is allocated by
torch, in a captured step from the graph's own memory.

Usage: python -m block_quantized_matmul_amd.serve  (a small run on one GPU)
"""
from __future__ import annotations

import functools

import numpy as np


def quantize_weight_f8b128(w):
    """Float weights (N, K) to (codes, scales) with one scale for each 128 x 128
    block: load-time work, in torch, on the weights' device."""
    import torch
    n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    p = torch.nn.functional.pad(w.float(), (0, kb * 128 - k, 0, nb * 128 - n))
    p = p.view(nb, 128, kb, 128)
    scale = (p.abs().amax((1, 3)) / 448.0).clamp_min(2.0 ** -126)
    codes = (p / scale[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(nb * 128, kb * 128)[:n, :k].contiguous(), scale.contiguous()


class SharedPromptAttention:
    """wqkv: ((n_q_heads + 2 n_kv_heads) * head_dim, hidden) and wo: (hidden,
    n_q_heads * head_dim) float weights; `batch` conversations of at most
    `max_pages` pages each behind one prompt; fp16 activations. weight_bits: 8
    (e4m3, blocks of 128) or 4 (microscaled floats; hidden % 32 == 0); kv_bits:
    16 or 8; q_norm, k_norm: weights (head_dim,) of the norms of q's and k's
    heads with `eps`, None: no norm."""

    def __init__(self, wqkv, wo, n_q_heads, n_kv_heads, head_dim, batch, prompt_pages, max_pages,
                 page_size=16, rope_base=10000.0, weight_bits=8, kv_bits=16, q_norm=None, k_norm=None,
                 eps=1e-6):
        import torch

        import block_quantized_matmul_amd as bq
        if weight_bits not in (4, 8) or kv_bits not in (8, 16):
            raise ValueError("weight_bits is 4 or 8, kv_bits 8 or 16")
        self.torch, self.bq = torch, bq
        self.weight_bits, self.kv_bits, self.eps = weight_bits, kv_bits, eps
        self.hq, self.hkv, self.d, self.ps = n_q_heads, n_kv_heads, head_dim, page_size
        self.dev = wqkv.device
        self.q_norm, self.k_norm = (
            None if w is None else w.to(device=self.dev, dtype=torch.float32).contiguous()
            for w in (q_norm, k_norm))
        quantize = quantize_weight_f8b128 if weight_bits == 8 else self._quantize_weight_mxfp4
        self.wqkv, self.wqkv_scale = quantize(wqkv)
        self.wo, self.wo_scale = quantize(wo)
        # the cache: (k, v), in 8 bits (k, v, k_scales, v_scales)
        of, num_pages = dict(device=self.dev), prompt_pages + batch * max_pages
        if kv_bits == 8:
            of["dtype"] = torch.float8_e4m3fn
        self.cache = bq.kv_cache_empty(num_pages, n_kv_heads, page_size, head_dim, **of)
        self.k_cache, self.v_cache = self.cache
        if kv_bits == 8:
            self.cache += bq.kv_scales_empty(num_pages, n_kv_heads, page_size, device=self.dev)
        inv_freq = rope_base ** (-np.arange(0, head_dim, 2) / head_dim)
        self.turns = bq.lqmm_rope_turns(inv_freq, device=self.dev)
        i32 = dict(dtype=torch.int32, device=self.dev)
        self.prompt_pages = torch.arange(prompt_pages, **i32)
        self.pages = (prompt_pages + torch.arange(batch * max_pages, **i32)).view(batch, max_pages)
        # a conversation's slots in order, and behind the last the -1 that is not
        # appended (of the pages above, which stay as they are)
        self.slots = torch.full((batch, max_pages * page_size + 1), -1, device=self.dev)
        self.slots[:, :-1] = (self.pages.long()[:, :, None] * page_size
                              + torch.arange(page_size, device=self.dev)).view(batch, -1)
        self.lens = torch.zeros(batch, **i32)
        self.prompt_len = 0
        self.rows = torch.arange(batch, device=self.dev)

    def _quantize_weight_mxfp4(self, w):
        return self.bq.lqmm_quant_mxfp4(w.float().contiguous())

    def _product(self, w, scale, x):
        if self.weight_bits == 4:
            return self.bq.lqmm_gemm_mxfp4(w, scale, *self.bq.lqmm_quant_mxfp4(x))
        return self.bq.lqmm_gemm_f8b128(w, scale, *self.bq.lqmm_quant_f8b128(x))

    def _project(self, x):
        """x (T, hidden) -> views q, k, v of the product's rows."""
        y = self._product(self.wqkv, self.wqkv_scale, x).view(x.shape[0], self.hq + 2 * self.hkv, self.d)
        return y[:, :self.hq], y[:, self.hq:self.hq + self.hkv], y[:, self.hq + self.hkv:]

    def _append(self, q, k, v, positions, slots):
        """Norms, rotation and append; returns q as the attention reads it."""
        if self.kv_bits == 16 and self.q_norm is None and self.k_norm is None:
            return self.bq.lqmm_kv_append(q, k, v, positions, slots, *self.cache, self.turns)
        return self.bq.lqmm_kv_append_norm(q, k, v, positions, slots, *self.cache, q_norm=self.q_norm,
                                           k_norm=self.k_norm, eps=self.eps, rope_turns=self.turns)

    def _attend(self, q, pages, lens, **kw):
        call = self.bq.lqmm_attn_prefix if self.kv_bits == 16 else self.bq.lqmm_attn_prefix_f8
        return call(q, *self.cache, pages, lens, **kw)

    def _output(self, o):
        return self._product(self.wo, self.wo_scale, o.view(o.shape[0], -1))

    def prompt(self, x):
        """Computes the shared prompt x (T, hidden) into its pages; returns the
        block's output for it."""
        torch, n = self.torch, x.shape[0]
        if n > self.prompt_pages.numel() * self.ps:
            raise ValueError("the prompt does not fit its pages")
        q, k, v = self._project(x)
        at = torch.arange(n, device=self.dev)
        slots = self.prompt_pages.long()[at // self.ps] * self.ps + at % self.ps
        q = self._append(q, k, v, at.int(), slots)
        i32 = dict(dtype=torch.int32, device=self.dev)
        o = self._attend(q, self.prompt_pages[None], torch.tensor([n], **i32),
                         q_start=torch.tensor([0, n], **i32), max_q=n)
        self.prompt_len = n
        return self._output(o)

    def step(self, x):
        """One new token of every conversation, x (batch, hidden): the block's
        output. The conversations' lengths advance by one. A conversation that
        already fills its max_pages pages gets no token and keeps its length;
        its row of the output is NaN (lengths are known on the device only, so
        that neither an eager step nor a replayed one can raise)."""
        q, k, v = self._project(x)
        n = self.lens.clamp(0, self.slots.shape[1] - 1)
        full = n == self.slots.shape[1] - 1
        slots = self.slots[self.rows, n]
        q = self._append(q, k, v, self.lens + self.prompt_len, slots)
        self.torch.add(n, ~full, out=self.lens)
        o = self._attend(q, self.pages, self.lens, prefix_pages=self.prompt_pages,
                         prefix_len=self.prompt_len)
        return self._output(o).masked_fill_(full[:, None], float("nan"))

    def keys_values(self, dtype=None):
        """What an 8-bit cache holds, as dense rows: (k, v, starts), rows starts[0]
        .. starts[1] - 1 the shared prompt's and starts[1 + b] .. starts[2 + b] - 1
        conversation b's own, keys as they were rotated. Waits for the lengths."""
        if self.kv_bits != 8:
            raise ValueError("keys_values reads an 8-bit cache")
        torch = self.torch
        # (lengths as a step takes them)
        counts = [self.prompt_len] + self.lens.clamp(0, self.slots.shape[1] - 1).tolist()
        pages = torch.zeros(len(counts), max(self.prompt_pages.numel(), self.pages.shape[1]),
                            dtype=torch.int32, device=self.dev)
        pages[0, :self.prompt_pages.numel()] = self.prompt_pages
        pages[1:, :self.pages.shape[1]] = self.pages
        starts = np.concatenate(([0], np.cumsum(counts))).tolist()
        if starts[-1] == 0:  # nothing held yet
            k, v = torch.empty(2, 0, self.hkv, self.d, dtype=dtype or torch.float16, device=self.dev)
            return k, v, starts
        k, v = self.bq.lqmm_kv_read_f8(*self.cache, pages,
                                       torch.tensor(starts, dtype=torch.int32, device=self.dev),
                                       starts[-1], dtype=dtype)
        return k, v, starts

    def capture(self, x):
        """A HIP graph of one step that reads x; returns (graph, output). Steps
        taken before are kept; capturing takes none. The graph serves later
        steps behind a prompt of the present length: its replay() raises
        RuntimeError after a prompt() of another one."""
        torch = self.torch
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # a first step outside the graph loads the kernels
            kept = self.lens.clone()
            self.step(x)
            self.lens.copy_(kept)
        torch.cuda.current_stream().wait_stream(side)
        graph = _step_graph_class()()
        graph.layer, graph.prompt_len = self, self.prompt_len
        with torch.cuda.graph(graph, stream=side):
            out = self.step(x)
        return graph, out


@functools.cache
def _step_graph_class():
    import torch

    class StepGraph(torch.cuda.CUDAGraph):
        """A graph of a step of `layer`. The prompt's length is part of what is
        captured (it plans the attention's launches): the graph is good for that
        length only."""

        def replay(self):
            if self.layer.prompt_len != self.prompt_len:
                raise RuntimeError(f"the graph was captured behind a prompt of {self.prompt_len} tokens, "
                                   f"which now has {self.layer.prompt_len}: capture it again")
            super().replay()

    return StepGraph


def main():
    import time

    import torch
    hidden, hq, hkv, d, batch = 4096, 32, 8, 128, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    wqkv = torch.randn((hq + 2 * hkv) * d, hidden, device="cuda", generator=g) / hidden ** 0.5
    wo = torch.randn(hidden, hq * d, device="cuda", generator=g) / hidden ** 0.5
    xp = torch.randn(8000, hidden, device="cuda", generator=g).half()
    x = torch.randn(batch, hidden, device="cuda", generator=g).half()
    ones = torch.ones(d, device="cuda")
    for what, kw in (("e4m3 products, 16-bit cache", {}),
                     ("4-bit products, 8-bit cache, norms of q and k",
                      dict(weight_bits=4, kv_bits=8, q_norm=ones, k_norm=ones))):
        layer = SharedPromptAttention(wqkv, wo, hq, hkv, d, batch, prompt_pages=512, max_pages=8, **kw)
        layer.prompt(xp)
        graph, _ = layer.capture(x)
        graph.replay()
        torch.cuda.synchronize()
        t, n = time.perf_counter(), 100
        for _ in range(n):
            graph.replay()
        torch.cuda.synchronize()
        print(f"{batch} conversations behind 8000 tokens: {(time.perf_counter() - t) / n * 1e6:.1f} us "
              f"per decode step of one attention block ({hidden} hidden, {hq}/{hkv} heads of {d}; {what})")


if __name__ == "__main__":
    main()
