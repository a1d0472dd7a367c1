"""Host side of the attention block that needs no GPU: everything that a call on a given
stream allocates, clears and launches has to belong to that stream."""
import contextlib

import pytest
import torch

from gemm_overlap_gemms_gb300 import attention_block as ab

TP, HIDDEN, HEADS, KV_HEADS, D, T = 2, 32, 2, 1, 8, 4


class Recorder:
    """Stands in for the user buffer: notes the current stream whenever something is
    allocated, cleared or launched."""

    def __init__(self, monkeypatch):
        self.current, self.seen = "default", []
        self.tp, self.active_shape = TP, (T, HIDDEN)

        @contextlib.contextmanager
        def use(stream):
            before, self.current = self.current, self.current if stream is None else stream
            yield
            self.current = before

        def zeros(*a, **kw):
            self.seen.append(("zeros", self.current))
            return real_zeros(*a, **kw)
        real_zeros = torch.zeros
        monkeypatch.setattr(torch.cuda, "stream", use)
        monkeypatch.setattr(torch, "zeros", zeros)

    def note(self, name, stream):
        self.seen += [(name + " memory", self.current), (name, self.current if stream is None else stream)]

    def ag_gemm(self, shards, Wt, Y=None, stream=None):
        self.note("ag_gemm", stream)
        return torch.ones(T, Wt.shape[0])

    def ag_gemm_from_buffer(self, Wt, Y=None, stream=None):
        return self.ag_gemm(None, Wt, stream=stream)

    def kv_append(self, q, *a, stream=None, **kw):
        self.note("kv_append", stream)

    def attn_prompt_paged(self, q, k, v, starts, lens, table, out=None, stream=None):
        self.note("attn_prompt_paged", stream)

    def attn_decode(self, q, k, v, lens, table, out=None, stream=None):
        self.note("attn_decode", stream)

    def gemm_rs(self, A, Bt, Y_shards=None, stream=None):
        self.note("gemm_rs", stream)
        return [torch.ones(T // TP, HIDDEN) for _ in range(TP)]


@pytest.mark.parametrize("call", ["prompt", "step"])
@pytest.mark.parametrize("stream", [None, "side"])
def test_all_memory_and_work_of_a_call_is_on_its_stream(monkeypatch, call, stream):
    buf = Recorder(monkeypatch)
    Wqkv = [torch.ones((HEADS + 2 * KV_HEADS) * D, HIDDEN) for _ in range(TP)]
    Wo = [torch.ones(HIDDEN, HEADS * D) for _ in range(TP)]
    block = ab.AttentionBlock(buf, Wqkv, Wo, HEADS, KV_HEADS, [(None, None)] * TP, None, None)
    getattr(block, call)([None] * TP, None, None, None, stream=stream)
    assert ("gemm_rs", stream or "default") in buf.seen
    assert {s for _, s in buf.seen} == {stream or "default"}, buf.seen
