"""The operators of a decoder layer one after the other, as a model calls them: QKV product with bias, rotary positions,
cache append, attention over prompts (or, for the next tokens, over the cache), O product onto the residual stream, and an
MLP with bias, GELU and residual.  Each is held to its bound on the input that it got."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_nvfp4_gb300 as g
import oracle
from gemm_nvfp4_gb300 import inputs
from helpers import DEV, assert_close, to_np
from test_gpu_epilogue import reference as product_reference
from test_gpu_prompt_attention import Prompts
from test_gpu_rope import angles, check as check_turned, frequencies

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HIDDEN, HQ, HK, D, MLP, PAGE = 512, 6, 2, 64, 768, 16


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


class Layer:
    def __init__(self, mlp):
        rand = lambda m, k, seed: torch.randn(m, k, device=DEV, generator=gen(seed)) * k ** -0.5  # noqa: E731
        quantize = g.nvfp4_quantize if mlp == "nvfp4" else g.nvfp4_fp6_quantize
        self.mlp = mlp
        self.qkv, self.o = g.nvfp4_quantize(rand((HQ + 2 * HK) * D, HIDDEN, 1)), g.nvfp4_quantize(rand(HIDDEN, HQ * D, 2))
        self.up, self.down = quantize(rand(MLP, HIDDEN, 3)), quantize(rand(HIDDEN, MLP, 4))
        self.b_qkv = torch.randn((HQ + 2 * HK) * D, device=DEV, generator=gen(5)).to(BF)
        self.b_up = torch.randn(MLP, device=DEV, generator=gen(6))
        self.rope = g.RopeTable.make(frequencies(D // 2))

    def __call__(self, x, positions, attend):
        """Every stage's output; attend(q, k, v) -> attention output."""
        qkv = g.nvfp4_gemm_epilogue(x, self.qkv, bias=self.b_qkv, out_dtype=BF)
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split((HQ * D, HK * D, HK * D), 1))
        turned = g.nvfp4_rope(q, k, positions, self.rope)
        a = attend(*turned, v)
        h = g.nvfp4_gemm_epilogue(a.flatten(1), self.o, residual=x, out_dtype=BF)
        call = g.nvfp4_gemm_epilogue if self.mlp == "nvfp4" else g.nvfp4_fp6_gemm_epilogue
        u = call(h, self.up, bias=self.b_up, activation=g.NVFP4_ACT_GELU_TANH, out_dtype=BF)
        y = call(u, self.down, residual=h, out_dtype=torch.float32)
        return dict(x=x, positions=positions, q=q, k=k, v=v, turned=turned, a=a, h=h, u=u, y=y, qkv=qkv)

    def product(self, got, x, W, bias=None, act="none", residual=None):
        bits = inputs.bf16_bits(x.cpu())
        if isinstance(W, g.FP6Weight):
            s, A = oracle.fp6_gemv(bits, W.codes.cpu().numpy(), W.scales.cpu().numpy())
        else:
            s, A = oracle.gemv(bits, W.codes.cpu().numpy(), W.scales.cpu().numpy(), W.tensor_scale.cpu().numpy()[0])
        assert_close(to_np(got), *product_reference(s, A, bias, act, residual, got.dtype))

    def check(self, r):
        """All stages but the attention."""
        self.product(r["qkv"], r["x"], self.qkv, bias=self.b_qkv)
        angle = angles(self.rope, [r["positions"].tolist()], [0] * (D // 2))
        for got, x in zip(r["turned"], (r["q"], r["k"])):
            check_turned(got, x, angle, D // 2)
        self.product(r["h"], r["a"].flatten(1), self.o, residual=r["x"])
        self.product(r["u"], r["h"], self.up, bias=self.b_up, act="gelu_tanh")
        self.product(r["y"], r["u"], self.down, residual=r["h"])


class Cache:
    """Pages of up to 6 * PAGE tokens for each of n sequences."""

    def __init__(self, n, fmt):
        self.cache = g.KVCache.empty(6 * n, PAGE, HK, D, fmt, DEV)
        self.table = torch.randperm(6 * n, generator=torch.Generator().manual_seed(7)).int().view(n, 6).to(DEV)

    def slots(self, seq, at):
        return self.table[seq].long().gather(1, (at // PAGE)[:, None])[:, 0] * PAGE + at % PAGE

    def error(self, q, a, lens):
        """Relative distance of one token's attention of each sequence from its definition on the cached values."""
        off = total = 0.0
        for b, n in enumerate(lens):
            at = torch.arange(n, device=DEV)
            k, v = (t.double().repeat_interleave(HQ // HK, 1) for t in
                    g.nvfp4_kv_read(self.cache, self.slots(torch.full_like(at, b), at)))
            p = torch.softmax(torch.einsum("hd,nhd->hn", q[b].double(), k) / D ** 0.5, -1)
            want = torch.einsum("hn,nhd->hd", p, v)
            off, total = off + float((a[b].double() - want).square().sum()), total + float(want.square().sum())
        return (off / total) ** 0.5


@pytest.mark.parametrize("fmt", [g.NVFP4_KV_E4M3, g.NVFP4_KV_NVFP4])
@pytest.mark.parametrize("mlp", ["nvfp4", "fp6"])
@pytest.mark.parametrize("lens", [[5, 70, 1], [1, 3, 2], [17, 40, 90]])
def test_prompts_then_decode(lens, mlp, fmt):
    n, total = len(lens), sum(lens)
    layer, cache = Layer(mlp), Cache(n, fmt)
    offsets = torch.tensor([0] + lens, device=DEV).cumsum(0).int()
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(lens, device=DEV))
    positions = torch.arange(total, device=DEV) - offsets[seq]
    status = torch.zeros(256, dtype=torch.uint8, device=DEV)

    def prompt(q, k, v):
        g.nvfp4_kv_append(cache.cache, k, v, cache.slots(seq, positions))
        return g.nvfp4_prompt_attention(q, k, v, offsets, workspace=status)

    x = torch.randn(total, HIDDEN, device=DEV, generator=gen(8)).to(BF)
    r = layer(x, positions, prompt)
    layer.check(r)
    p = Prompts(lens, HQ, HK, D)
    p.q, p.k, p.v = *r["turned"], r["v"]
    p.check(r["a"])
    assert g.nvfp4_device_status(status) == (g.NVFP4_OK, 0)

    # one more token of each sequence, captured; the replays see new tokens, positions, slots and lengths
    at = torch.tensor(lens, device=DEV)
    kv_lens, slots, x1 = at.int() + 1, cache.slots(torch.arange(n, device=DEV), at), torch.empty(n, HIDDEN, dtype=BF, device=DEV)
    attention_ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(cache.cache, r["q"][:n], n, 1), dtype=torch.uint8, device=DEV)

    def decode(q, k, v):
        g.nvfp4_kv_append(cache.cache, k, v, slots)
        return g.nvfp4_paged_attention(q, cache.cache, cache.table, kv_lens, workspace=attention_ws)

    x1.copy_(torch.randn(n, HIDDEN, device=DEV, generator=gen(9)))
    eager = layer(x1, at, decode)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = layer(x1, at, decode)
    graph.replay()
    assert all(torch.equal(r[s], eager[s]) for s in ("qkv", "a", "h", "u", "y"))
    for step in range(3):
        if step:
            x1.copy_(torch.randn(n, HIDDEN, device=DEV, generator=gen(9 + step)))
            at += 1
            kv_lens += 1
            slots.copy_(cache.slots(torch.arange(n, device=DEV), at))
            graph.replay()
        layer.check(r)
        # rounding to bf16 is 2^-9 at most; the weights' f16 (a cache's type) adds less than 2^-11
        assert cache.error(r["turned"][0], r["a"], kv_lens.tolist()) < 2.0 ** -8


def test_the_same_bits_on_another_stream_and_beside_another_layer():
    layer, lens = Layer("nvfp4"), [40, 3, 61]
    offsets = torch.tensor([0] + lens, device=DEV).cumsum(0).int()
    xs = [torch.randn(sum(lens), HIDDEN, device=DEV, generator=gen(20 + i)).to(BF) for i in range(2)]
    positions = torch.arange(sum(lens), device=DEV)

    def attend(q, k, v):
        return g.nvfp4_prompt_attention(q, k, v, offsets)

    want = [layer(x, positions, attend)["y"] for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [[] for _ in xs]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(xs[i], positions, attend)["y"])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    assert not np.isnan(to_np(want[0])).any()
