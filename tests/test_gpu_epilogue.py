"""Products with an epilogue (nvfp4_gemm_epilogue, nvfp4_fp6_gemm_epilogue) against the oracle's sums and the
activations' definitions in fp64."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import gemm_nvfp4_gb300 as g
import oracle
from gemm_nvfp4_gb300 import inputs
from helpers import ABS, BF16_REL, DEV, REL, assert_close, to_np

pytestmark = pytest.mark.gpu

ACTS = {"none": g.NVFP4_ACT_NONE, "silu": g.NVFP4_ACT_SILU, "gelu": g.NVFP4_ACT_GELU,
        "gelu_tanh": g.NVFP4_ACT_GELU_TANH, "relu": g.NVFP4_ACT_RELU, "relu2": g.NVFP4_ACT_RELU2}


def activation(act, v):
    """(value, bound of the slope within e of v as a function of e, u of the header's bound)"""
    u = np.zeros_like(v)
    with np.errstate(over="ignore"):  # exp(-v) of a large negative v: the quotient is zero
        if act == "none":
            return v, lambda e: 1.0, u
        if act == "silu":
            return v / (1 + np.exp(-v)), lambda e: 1.13, u
        if act == "gelu":
            return v * np.vectorize(lambda x: math.erfc(-x / math.sqrt(2)) / 2)(v), lambda e: 1.13, u
        if act == "gelu_tanh":
            u = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
            return v / (1 + np.exp(-u)), lambda e: 1.13, np.abs(u)
    r = np.maximum(v, 0)
    return (r, lambda e: 1.0, u) if act == "relu" else (r * r, lambda e: 2 * np.abs(v) + e, u)


def reference(s, A, bias, act, residual, out_dtype):
    """(y, tolerance): include/nvfp4.h's bound, and the rounding of y"""
    v = s if bias is None else s + to_np(bias)
    a, slope, u = activation(act, v)
    y = a if residual is None else a + to_np(residual)
    e = REL * A + ABS + 2.0 ** -23 * np.abs(v)
    tol = slope(e) * e + 2.0 ** -20 * (1 + u) * np.abs(a) + 2.0 ** -24 * np.abs(y) + 1e-30
    if out_dtype == torch.bfloat16:
        tol = tol + BF16_REL * (np.abs(y) + tol)
    return y, tol


class Product:
    """One matrix, its activations and the oracle's sums of their product."""

    def __init__(self, fmt, N, M, K, seed=0):
        self.fmt, self.N, self.M, self.K = fmt, N, M, K
        w = inputs.weights(M, K, seed=seed)
        x = inputs.activations(N, K, seed=seed + 1)
        self.x = x.to(DEV)
        if fmt == "nvfp4":
            self.W = g.nvfp4_quantize(w.to(DEV))
            self.s, self.A = oracle.gemv(inputs.bf16_bits(x), *oracle.quantize(w.numpy()))
        else:
            self.W = g.nvfp4_fp6_quantize(w.to(DEV))
            self.s, self.A = oracle.fp6_gemv(inputs.bf16_bits(x), *oracle.fp6_quantize(w.numpy()))

    def run(self, **kw):
        call = g.nvfp4_gemm_epilogue if self.fmt == "nvfp4" else g.nvfp4_fp6_gemm_epilogue
        return call(self.x, self.W, **kw)

    def plain(self, **kw):
        if self.fmt == "nvfp4":
            return g.nvfp4_gemm_prefill(self.x, self.W, **kw)
        return g.nvfp4_fp6_gemm(self.x, self.W, **kw)

    def vector(self, dtype, seed):
        gen = torch.Generator().manual_seed(seed)
        return torch.randn(self.M, generator=gen).to(dtype).to(DEV)

    def rows(self, dtype, seed, pad=0):
        gen = torch.Generator().manual_seed(seed)
        return (2 * torch.randn(self.N, self.M + pad, generator=gen)).to(dtype).to(DEV)[:, :self.M]


# every kernel that stores a product: the warp-level one (K % 256 != 0; with and without split tiles),
# the tcgen05 skinny one (whole tiles, split ones, clusters), the prefill one (registers, TMA, 192-token
# tiles, split mode with its reduction); odd sizes
SHAPES = [("nvfp4", 1, 48, 272), ("nvfp4", 9, 130, 48), ("nvfp4", 16, 3, 16), ("nvfp4", 1, 4096, 4096), ("nvfp4", 4, 200, 512),
          ("nvfp4", 5, 1, 1024), ("nvfp4", 3, 17000, 256), ("nvfp4", 17, 129, 272), ("nvfp4", 40, 200, 512),
          ("nvfp4", 300, 257, 80), ("nvfp4", 190, 700, 1024), ("nvfp4", 260, 131, 4096),
          ("fp6", 1, 48, 128), ("fp6", 12, 130, 384), ("fp6", 2, 333, 512), ("fp6", 18, 129, 128), ("fp6", 200, 260, 640)]


@pytest.mark.parametrize("fmt,N,M,K", SHAPES)
def test_every_kernel(fmt, N, M, K):
    p = Product(fmt, N, M, K, seed=N + M)
    cases = [("none", None, torch.bfloat16, torch.bfloat16), ("gelu_tanh", torch.bfloat16, None, torch.float32),
             ("silu", torch.float32, torch.float32, torch.float32), ("none", torch.float32, None, torch.bfloat16)]
    for i, (act, b, r, out) in enumerate(cases):
        bias = None if b is None else p.vector(b, 5)
        residual = None if r is None else p.rows(r, 6, pad=i)
        y = p.run(bias=bias, activation=ACTS[act], residual=residual, out_dtype=out)
        ref, tol = reference(p.s, p.A, bias, act, residual, out)
        assert y.dtype == out
        assert_close(to_np(y), ref, tol, f"{act} {b} {r} {out}")


@pytest.mark.parametrize("fmt,N,M,K", [("nvfp4", 200, 260, 8448), ("fp6", 17, 129, 8320), ("fp6", 193, 260, 8448),
                                       ("fp6", 300, 131, 9216), ("fp6", 40, 3, 10240)])
def test_fp32_outputs_of_long_sums(fmt, N, M, K):
    """FP6 sums are added up in parts of 2048 products: a whole number of them, and last ones of 128 to 1024."""
    p = Product(fmt, N, M, K, seed=N)
    bias, residual = p.vector(torch.bfloat16, 5), p.rows(torch.float32, 6, pad=1)
    for act in ("none", "gelu_tanh"):
        y = p.run(bias=bias, activation=ACTS[act], residual=residual)
        assert_close(to_np(y), *reference(p.s, p.A, bias, act, residual, torch.float32))
        assert torch.equal(p.run(bias=bias, activation=ACTS[act], residual=residual), y)
    if fmt == "fp6":  # (without a tensor scale the parts are products of their own, to the bit)
        total = torch.zeros_like(y)
        for k in range(0, K, 2048):
            at = slice(k, min(k + 2048, K))
            W = g.FP6Weight(p.W.codes[:, k // 4 * 3:at.stop // 4 * 3].contiguous(), p.W.scales[:, k // 128:at.stop // 128].contiguous())
            total += g.nvfp4_fp6_gemm_epilogue(p.x[:, at].contiguous(), W)
        assert torch.equal(p.run(), total)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [2, 33])
def test_every_activation(act, N):
    """Sums from -30 to 30, where the activations' tails lie."""
    p = Product("nvfp4", N, 96, 512, seed=3)
    bias = torch.linspace(-30, 30, 96, device=DEV)
    for out in (torch.float32, torch.bfloat16):
        y = p.run(bias=bias, activation=ACTS[act], out_dtype=out)
        ref, tol = reference(p.s, p.A, bias, act, None, out)
        assert_close(to_np(y), ref, tol, act)


@pytest.mark.parametrize("fmt,N,M,K", [("nvfp4", 1, 4096, 4096), ("nvfp4", 9, 130, 272), ("nvfp4", 260, 131, 4096), ("fp6", 40, 200, 256)])
def test_nothing_asked_is_the_plain_product(fmt, N, M, K):
    p = Product(fmt, N, M, K)
    for out in (torch.float32, torch.bfloat16):
        assert torch.equal(p.run(out_dtype=out), p.plain(out_dtype=out))


@pytest.mark.parametrize("N", [1, 7, 16, 17, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place_residual_and_repeated_calls(N, dtype):
    """The residual stream is the output; one workspace serves calls of several shapes, and each repeat gives its bits."""
    p = Product("nvfp4", N, 640, 2304, seed=N)
    start = p.rows(dtype, 8).contiguous()
    ws = torch.zeros(g.nvfp4_workspace_bytes(g.NVFP4_OP_GEMM_PREFILL, N, 640, 2304), dtype=torch.uint8, device=DEV)
    apart = p.run(residual=start, out_dtype=dtype, workspace=ws)
    ref, tol = reference(p.s, p.A, None, "none", start, dtype)
    assert_close(to_np(apart), ref, tol)
    for _ in range(3):
        y = start.clone()
        assert p.run(residual=y, out=y, workspace=ws) is y
        assert torch.equal(y, apart)


@pytest.mark.parametrize("N", [1, 40])
def test_infinities_and_nan_go_through(N):
    p = Product("nvfp4", N, 64, 512)
    bias = torch.zeros(64, device=DEV)
    bias[3], bias[5], bias[7] = math.nan, math.inf, -math.inf
    residual = torch.zeros(N, 64, device=DEV)
    residual[0, 9] = math.nan
    for name, act in ACTS.items():
        y = p.run(bias=bias, activation=act, residual=residual)
        assert torch.isnan(y[:, 3]).all(), name
        assert (y[:, 5] == math.inf).all(), name
        assert torch.isnan(y[0, 9]), name
        if name in ("relu", "relu2"):
            assert (y[:, 7] == 0).all()
        ok = torch.ones(64, dtype=torch.bool, device=DEV)
        ok[[3, 5, 7, 9]] = False
        assert torch.isfinite(y[:, ok]).all(), name


@pytest.mark.parametrize("N", [1, 16, 520])
def test_captured_and_replayed(N):
    """A graph of the call replayed on other activations and residuals."""
    p = Product("nvfp4", N, 384, 1024)
    ws = torch.zeros(g.nvfp4_workspace_bytes(g.NVFP4_OP_GEMM_PREFILL, N, 384, 1024), dtype=torch.uint8, device=DEV)
    bias, residual = p.vector(torch.bfloat16, 1), p.rows(torch.float32, 2).contiguous()
    out = torch.empty(N, 384, device=DEV)
    call = lambda: p.run(bias=bias, activation=g.NVFP4_ACT_SILU, residual=residual, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    p.x.copy_(p.x.flip(0))
    residual.mul_(-1)
    graph.replay()
    got = out.clone()
    assert torch.equal(call(), got)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)


def test_another_stream():
    p = Product("nvfp4", 8, 256, 512)
    want = p.run(bias=p.vector(torch.float32, 1))
    s = torch.cuda.Stream()
    bias = p.vector(torch.float32, 1)
    s.wait_stream(torch.cuda.current_stream())
    got = p.run(bias=bias, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


class Sampled:
    """A product too large for the oracle: its sums at some tokens and rows."""

    def __init__(self, N, M, K, tokens, rows):
        gen = torch.Generator(DEV).manual_seed(N)
        self.x = torch.randn(N, K, device=DEV, generator=gen).to(torch.bfloat16)
        self.W = g.nvfp4_quantize(0.02 * torch.randn(M, K, device=DEV, generator=gen))
        self.at = torch.tensor(tokens)[:, None], torch.tensor(rows)
        self.s, self.A = oracle.gemv(inputs.bf16_bits(self.x[tokens].cpu()), self.W.codes[rows].cpu().numpy(),
                                     self.W.scales[rows].cpu().numpy(), self.W.tensor_scale.cpu().numpy()[0])

    def check(self, y, bias, act, residual):
        part = lambda t, at: None if t is None else t.cpu()[at]  # noqa: E731
        ref, tol = reference(self.s, self.A, part(bias, self.at[1]), act, part(residual, self.at), y.dtype)
        assert_close(to_np(y.cpu()[self.at]), ref, tol, act)


# Operands beyond what L2 holds, and a number of tiles that leaves few for the last wave: whole tiles in a launch of their
# own, the last ones split behind them in a second one that does not wait for it, and a reduction.  One token tile (tiles
# behind row 152 * 128 are the split ones), two of them, and a 27B-class layer's down product of 2048 tokens.
@pytest.mark.parametrize("N,M,K", [(200, 20400, 12032), (300, 19500, 12032), (2048, 5120, 17408)])
def test_split_tiles_behind_whole_ones(N, M, K):
    tokens = sorted({0, 1, N // 2, N - 1, *range(255, N, 256), *range(256, N, 256)})
    rows = sorted({*range(0, M, 97), *range(max(M - 1100, 0), M, 13), M - 1})
    p = Sampled(N, M, K, tokens, rows)
    gen = torch.Generator(DEV).manual_seed(7)
    ws = torch.zeros(g.nvfp4_workspace_bytes(g.NVFP4_OP_GEMM_PREFILL, N, M, K), dtype=torch.uint8, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(g.nvfp4_gemm_epilogue(p.x, p.W, out_dtype=dtype), g.nvfp4_gemm_prefill(p.x, p.W, out_dtype=dtype))
        wide = 2 * torch.randn(N, M + 3, device=DEV, generator=gen).to(dtype)
        residual = wide[:, :M]
        for act, bias in (("none", None), ("gelu_tanh", torch.randn(M, device=DEV, generator=gen)),
                          ("silu", torch.randn(M, device=DEV, generator=gen).to(torch.bfloat16))):
            call = lambda **kw: g.nvfp4_gemm_epilogue(p.x, p.W, bias=bias, activation=ACTS[act], workspace=ws, **kw)  # noqa: E731
            y = call(residual=residual, out_dtype=dtype)
            p.check(y, bias, act, residual)
            p.check(call(out_dtype=dtype), bias, act, None)
            # in place, on the residual that the launch before has just written
            for _ in range(3):
                z = residual * 1
                assert call(residual=z, out=z) is z
                assert torch.equal(z, y)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)


def test_rotary_positions_right_behind_split_tiles():
    """The launch after a product with three launches, a programmatic dependent of the last one, reads tiles of the first."""
    N, M, K = 200, 20480, 12032
    p = Sampled(N, M, K, [0, N - 1], [0, M - 1])
    table = g.RopeTable.make([1e6 ** (-i / 64) for i in range(64)])
    at = torch.arange(N, device=DEV)
    y = g.nvfp4_gemm_epilogue(p.x, p.W, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    want = g.nvfp4_rope(y.view(N, 160, 128), None, at, table)[0]
    for _ in range(20):
        y.zero_()
        g.nvfp4_gemm_epilogue(p.x, p.W, out=y)
        assert torch.equal(g.nvfp4_rope(y.view(N, 160, 128), None, at, table)[0], want)
