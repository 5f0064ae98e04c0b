"""The attention block of a decoder layer, served for a batch of conversations
behind one shared prompt, from the library's serving operators:

  e4m3 of the activations (lqmm_quant_f8b128) -> q, k, v in one product
  (lqmm_gemm_f8b128) -> rotation and append to the paged cache
  (lqmm_kv_append) -> attention, the shared prompt's keys read once for the
  whole batch (lqmm_attn_prefix) -> e4m3 -> output product.

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
    `max_pages` pages each behind one prompt; fp16 activations."""

    def __init__(self, wqkv, wo, n_q_heads, n_kv_heads, head_dim, batch, prompt_pages, max_pages,
                 page_size=16, rope_base=10000.0):
        import torch

        import block_quantized_matmul_amd as bq
        self.torch, self.bq = torch, bq
        self.hq, self.hkv, self.d, self.ps = n_q_heads, n_kv_heads, head_dim, page_size
        self.dev = wqkv.device
        self.wqkv, self.wqkv_scale = quantize_weight_f8b128(wqkv)
        self.wo, self.wo_scale = quantize_weight_f8b128(wo)
        self.k_cache, self.v_cache = bq.kv_cache_empty(prompt_pages + batch * max_pages, n_kv_heads,
                                                       page_size, head_dim, device=self.dev)
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

    def _project(self, x):
        """x (T, hidden) -> views q, k, v of the product's rows."""
        codes, scales = self.bq.lqmm_quant_f8b128(x)
        y = self.bq.lqmm_gemm_f8b128(self.wqkv, self.wqkv_scale, codes, scales)
        y = y.view(x.shape[0], self.hq + 2 * self.hkv, self.d)
        return y[:, :self.hq], y[:, self.hq:self.hq + self.hkv], y[:, self.hq + self.hkv:]

    def _output(self, o):
        codes, scales = self.bq.lqmm_quant_f8b128(o.view(o.shape[0], -1))
        return self.bq.lqmm_gemm_f8b128(self.wo, self.wo_scale, codes, scales)

    def prompt(self, x):
        """Computes the shared prompt x (T, hidden) into its pages; returns the
        block's output for it."""
        torch, n = self.torch, x.shape[0]
        if n > self.prompt_pages.numel() * self.ps:
            raise ValueError("the prompt does not fit its pages")
        q, k, v = self._project(x)
        at = torch.arange(n, device=self.dev)
        slots = self.prompt_pages.long()[at // self.ps] * self.ps + at % self.ps
        q = self.bq.lqmm_kv_append(q, k, v, at.int(), slots, self.k_cache, self.v_cache, self.turns)
        i32 = dict(dtype=torch.int32, device=self.dev)
        o = self.bq.lqmm_attn_prefix(q, self.k_cache, self.v_cache, self.prompt_pages[None],
                                     torch.tensor([n], **i32), q_start=torch.tensor([0, n], **i32),
                                     max_q=n)
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
        q = self.bq.lqmm_kv_append(q, k, v, self.lens + self.prompt_len, slots, self.k_cache,
                                   self.v_cache, self.turns)
        self.torch.add(n, ~full, out=self.lens)
        o = self.bq.lqmm_attn_prefix(q, self.k_cache, self.v_cache, self.pages, self.lens,
                                     prefix_pages=self.prompt_pages, prefix_len=self.prompt_len)
        return self._output(o).masked_fill_(full[:, None], float("nan"))

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
    layer = SharedPromptAttention(wqkv, wo, hq, hkv, d, batch, prompt_pages=512, max_pages=8)
    layer.prompt(torch.randn(8000, hidden, device="cuda", generator=g).half())
    x = torch.randn(batch, hidden, device="cuda", generator=g).half()
    graph, _ = layer.capture(x)
    graph.replay()
    torch.cuda.synchronize()
    t, n = time.perf_counter(), 100
    for _ in range(n):
        graph.replay()
    torch.cuda.synchronize()
    print(f"{batch} conversations behind 8000 tokens: {(time.perf_counter() - t) / n * 1e6:.1f} us "
          f"per decode step of one attention block ({hidden} hidden, {hq}/{hkv} heads of {d})")


if __name__ == "__main__":
    main()
