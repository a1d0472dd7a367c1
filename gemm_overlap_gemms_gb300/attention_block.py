"""The attention half of a transformer layer for serving, on one user buffer: tp virtual
shards of heads between the column-parallel QKV projection and the row-parallel output
projection.

    QKV (ag_gemm; the other shards' from the gathered buffer)
      -> rotation and append to the shard's paged cache (kv_append)
      -> attention: prompts or chunks of prompts (attn_prompt_paged), or one new token per
         sequence (attn_decode)
      -> output projection, summed over the shards (gemm_rs)

Nothing is read on the host between the calls, so a decoding step can be captured into a
CUDA graph and replayed with new lengths and page tables.

    python -m gemm_overlap_gemms_gb300.attention_block

runs packed prompts and some decoding steps with random weights and prints their times.
"""
from __future__ import annotations

import math

import torch

from . import synth, ub


class AttentionBlock:
    """Weights and caches of one layer's attention.

    buf: the user buffer (hidden, tp). Wqkv: tp weights [(heads + 2 kv_heads) * D, hidden], a
    shard's query, key and value rows in this order. Wo: tp weights [hidden, heads * D]. heads,
    kv_heads: of one shard. caches: tp pairs (k, v) [pages, kv_heads, page_size, D]. cos, sin:
    fp32 [positions, rot / 2]."""

    def __init__(self, buf: ub.UserBuffer, Wqkv, Wo, heads: int, kv_heads: int, caches, cos, sin,
                 interleaved: bool = False):
        self.buf, self.Wqkv, self.Wo, self.caches = buf, Wqkv, Wo, caches
        self.heads, self.kv_heads = heads, kv_heads
        self.head_dim = Wqkv[0].shape[0] // (heads + 2 * kv_heads)
        self.cos, self.sin, self.interleaved = cos, sin, interleaved

    def _run(self, shards, seq_starts, kv_lens, page_table, attention, stream):
        # Everything below allocates and clears on the current stream, so that has to be the
        # call's: a clearing elsewhere could land after the attention has written, and memory
        # dropped here could be reused while the call still reads it.
        with torch.cuda.stream(stream):
            return self._run_here(shards, seq_starts, kv_lens, page_table, attention, stream)

    def _run_here(self, shards, seq_starts, kv_lens, page_table, attention, stream):
        buf, H, G, D = self.buf, self.heads, self.kv_heads, self.head_dim
        T = buf.active_shape[0]
        A = []
        for j in range(buf.tp):
            y = (buf.ag_gemm(shards, self.Wqkv[j], stream=stream) if j == 0
                 else buf.ag_gemm_from_buffer(self.Wqkv[j], stream=stream)).view(T, H + 2 * G, D)
            q = y[:, :H]
            k_cache, v_cache = self.caches[j]
            buf.kv_append(q, y[:, H:H + G], y[:, H + G:], self.cos, self.sin, seq_starts, kv_lens, page_table,
                          k_cache, v_cache, q_out=q, interleaved=self.interleaved, stream=stream)
            # rows of no sequence (T rounded up to a multiple of tp) go on as zeros
            a = torch.zeros((T, H, D), dtype=torch.bfloat16, device=y.device)
            attention(q, k_cache, v_cache, a)
            A.append(a.view(T, H * D))
        return buf.gemm_rs(A, self.Wo, stream=stream)

    def prompt(self, shards, seq_starts, kv_lens, page_table, stream=None):
        """Output shards for the active tokens: whole prompts, or chunks of prompts whose
        beginnings are cached; seq_starts [n + 1], kv_lens [n] with these tokens, page_table
        [n, entries]. With `stream` everything runs there, the inputs have to be ready there, and
        the outputs belong to it."""
        return self._run(shards, seq_starts, kv_lens, page_table,
                         lambda q, k, v, a: self.buf.attn_prompt_paged(q, k, v, seq_starts, kv_lens, page_table, out=a,
                                                                       stream=stream), stream)

    def step(self, shards, seq_starts, kv_lens, page_table, stream=None):
        """The same for one new token per sequence (seq_starts = 0, 1, ... n)."""
        return self._run(shards, seq_starts, kv_lens, page_table,
                         lambda q, k, v, a: self.buf.attn_decode(q, k, v, kv_lens, page_table, out=a, stream=stream),
                         stream)


def rotation_tables(positions: int, rot: int, base: float = 10000.0, device="cuda"):
    """fp32 (cos, sin) [positions, rot / 2] of the angles position * base^(-2 j / rot)."""
    inv = torch.exp(torch.arange(0, rot, 2, device=device, dtype=torch.float32) * (-math.log(base) / rot))
    angle = torch.arange(positions, device=device, dtype=torch.float32)[:, None] * inv[None, :]
    return angle.cos(), angle.sin()


def main():
    tp, hidden, heads, kv_heads, D, page = 4, 4096, 8, 2, 128, 64
    lengths, steps = [3040, 2716, 875, 1406], 16
    dev = torch.device("cuda")
    gen = synth.generator(dev)
    n, longest = len(lengths), max(lengths) + steps
    width = -(-longest // page)
    table = torch.arange(n * width, dtype=torch.int32, device=dev).view(n, width)
    caches = [tuple(torch.zeros(n * width, kv_heads, page, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
              for _ in range(tp)]
    Wqkv = [synth.normal_bf16(((heads + 2 * kv_heads) * D, hidden), hidden ** -0.5, gen, dev) for _ in range(tp)]
    Wo = [synth.normal_bf16((hidden, heads * D), (tp * heads * D) ** -0.5, gen, dev) for _ in range(tp)]
    cos, sin = rotation_tables(longest, D)
    T = -(-sum(lengths) // tp) * tp
    with ub.UserBuffer([8192, hidden], tp) as buf:
        block = AttentionBlock(buf, Wqkv, Wo, heads, kv_heads, caches, cos, sin)

        def timed(what, fn):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            fn()
            a.record()
            fn()
            b.record()
            b.synchronize()
            if buf.query_status() != ub.UB_OK:
                raise RuntimeError("%s: device status %d" % (what, buf.query_status()))
            print("%s: %.1f us" % (what, a.elapsed_time(b) * 1e3))

        starts = torch.tensor([0] + lengths, device=dev).cumsum(0).to(torch.int32)
        lens = torch.tensor(lengths, dtype=torch.int32, device=dev)
        buf.set_active_shape([T, hidden])
        shards = [synth.normal_bf16((T // tp, hidden), 1.0, gen, dev) for _ in range(tp)]
        timed("prompts of %s tokens" % lengths, lambda: block.prompt(shards, starts, lens, table))

        buf.set_active_shape([n, hidden])
        tokens = [synth.normal_bf16((n // tp, hidden), 1.0, gen, dev) for _ in range(tp)]
        one = torch.arange(n + 1, dtype=torch.int32, device=dev)
        lens += 1
        timed("decoding step of %d sequences" % n, lambda: block.step(tokens, one, lens, table))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block.step(tokens, one, lens, table, stream=torch.cuda.current_stream())
            lens += 1
        timed("decoding step from a graph", graph.replay)


if __name__ == "__main__":
    main()
