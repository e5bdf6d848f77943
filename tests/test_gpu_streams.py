"""Calls given a stream but no workspace or output: what they allocate belongs to that stream.

The current stream is kept busy, and the memory that a workspace could get is
left dirty, so that a zero-fill or a buffer of the current stream would be seen."""
from __future__ import annotations

import pytest
import torch

import gemm_nvfp4_gb300 as g
from gemm_nvfp4_gb300 import inputs
from helpers import DEV
from test_gpu_attention import Batch

pytestmark = pytest.mark.gpu


def _busy():
    a = torch.ones(4096, 4096, dtype=torch.bfloat16, device=DEV)
    for _ in range(40):
        a = (a @ a).clamp_(max=1)
    return a


def _on_side_stream(call):
    """call(stream) on a side stream whose free memory is all ones, behind a busy current stream."""
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        dirty = [torch.full((1 << n,), 255, dtype=torch.uint8, device=DEV) for n in range(9, 26)]
    for d in dirty:
        d.record_stream(s)
    del dirty, d
    s.synchronize()
    busy = _busy()
    outs = [call(s) for _ in range(3)]
    s.synchronize()
    outs = [torch.stack([x.clone() for x in o]) if isinstance(o, tuple) else o.clone() for o in outs]
    torch.cuda.synchronize()
    assert torch.isfinite(busy).all()
    return outs


@pytest.mark.parametrize("q_len,kv", [(1, 9000), (5, 9000), (40, 3000), (150, 3000)])
def test_attention_without_a_workspace(q_len, kv):
    b = Batch(g.NVFP4_KV_E4M3, [q_len], [kv], 8, 2, 128, 64, seed=3)
    want = b.run()
    for got in _on_side_stream(lambda s: b.run(stream=s)):
        assert torch.equal(got, want)


def test_cache_rows_read_into_new_tensors():
    b = Batch(g.NVFP4_KV_NVFP4, [1], [5000], 8, 2, 128, 64, seed=4)
    slots = b.slots(0, 5000).to(DEV)
    want = torch.stack(g.nvfp4_kv_read(b.cache, slots))
    for got in _on_side_stream(lambda s: g.nvfp4_kv_read(b.cache, slots, stream=s)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("N", [1, 16, 512])
def test_products_without_a_workspace(N):
    """Skinny products keep split-K counters in the workspace, the prefill product partial tiles."""
    W = g.nvfp4_quantize(inputs.weights(2048, 4096, seed=5, device=DEV))
    x = inputs.activations(N, 4096, seed=N, device=DEV)
    call = g.nvfp4_gemv_skinny if N <= 16 else g.nvfp4_gemm_prefill
    want = call(x, W)
    for got in _on_side_stream(lambda s: call(x, W, stream=s)):
        assert torch.equal(got, want)


def test_weights_quantised_into_new_tensors():
    w = inputs.weights(512, 1024, seed=1, device=DEV)
    want = g.nvfp4_quantize(w).codes
    for got in _on_side_stream(lambda s: g.nvfp4_quantize(w, stream=s).codes):
        assert torch.equal(got, want)
