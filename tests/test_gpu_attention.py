"""nvfp4_paged_attention against its definition in fp64: head layouts, lengths
from none to long, ragged batches, windows, trees, cross attention, rows that
see nothing, garbage and NaN in masked places, and indices out of bounds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_nvfp4_gb300 as g
import kv_reference as ref
from helpers import DEV

pytestmark = pytest.mark.gpu

FORMATS = [g.NVFP4_KV_E4M3, g.NVFP4_KV_NVFP4]


class Batch:
    """Sequences with random keys in a paged cache whose other bytes are all ones (NaN codes)."""

    def __init__(self, fmt, q_lens, kv_lens, hq, hk, d, page_size, seed=0, spread=1.0, q_scale=1.0, extra_width=1):
        gen = torch.Generator(DEV).manual_seed(seed)
        self.q_lens, self.kv_lens, self.hq, self.hk, self.d = list(q_lens), list(kv_lens), hq, hk, d
        need = [-(-n // page_size) for n in kv_lens]
        pages = sum(need) + 3
        self.cache = g.KVCache.empty(pages, page_size, hk, d, fmt, device=DEV)
        self.cache.pool.fill_(255)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
        self.table = torch.full((len(need), max(need + [0]) + extra_width), -1, dtype=torch.int32)
        self.k, self.v, first = [], [], 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[first:first + n]
            first += n
            k, v = (torch.randn(kv_lens[b], hk, d, device=DEV, generator=gen) for _ in range(2))
            v *= torch.exp2(spread * torch.randn(kv_lens[b], hk, 1, device=DEV, generator=gen))
            self.put(b, k.to(torch.bfloat16), v.to(torch.bfloat16))
        self.table = self.table.to(DEV)
        self.q = (q_scale * torch.randn(sum(q_lens), hq, d, device=DEV, generator=gen)).to(torch.bfloat16)
        self.lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        self.offsets = torch.tensor(np.cumsum([0] + self.q_lens), dtype=torch.int32, device=DEV)

    def slots(self, b, n):
        at = torch.arange(n)
        return (self.table[b].cpu().long()[at // self.cache.page_size] * self.cache.page_size
                + at % self.cache.page_size)

    def put(self, b, k, v):
        if len(k):
            g.nvfp4_kv_append(self.cache, k, v, self.slots(b, len(k)).to(DEV))

    def run(self, **kw):
        uniform = len(set(self.q_lens)) == 1 and not kw.pop("ragged", False)
        return g.nvfp4_paged_attention(self.q, self.cache, self.table, self.lens,
                                       q_offsets=None if uniform else self.offsets,
                                       max_q_len=max(self.q_lens), **kw)

    def want(self, causal=True, window=0, tree=None, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        pool = self.cache.pool.cpu().numpy()
        parts, at = [], 0
        for b, (n, kv) in enumerate(zip(self.q_lens, self.kv_lens)):
            k, v = ref.cache_rows(pool, self.slots(b, kv).numpy(), self.cache.page_size, self.d, self.cache.format)
            see = ref.visible(n, kv, causal, window, None if tree is None else tree[at:at + n].cpu().numpy())
            parts.append(ref.attention(ref.to_np(self.q[at:at + n]), k, v, see, scale))
            at += n
        return tuple(np.concatenate(x) for x in zip(*parts))

    def check(self, got, **kw):
        out, weight, s = self.want(**kw)
        x = ref.to_np(got)
        assert np.array_equal(np.isnan(x), np.isnan(out))
        err, tol = np.abs(x - out), ref.tolerance(out, weight, s, got.dtype)
        ok = np.isnan(out) | (err <= tol)
        assert ok.all(), f"{(~ok).sum()} of {ok.size} out of bounds, worst {np.nanmax(err / tol):.3g} of the bound"


SHAPES = [
    # q_lens, kv_lens, hq, hk, d, page_size
    ([1], [1], 4, 4, 64, 16),
    ([1], [7], 8, 1, 128, 16),
    ([1], [555], 32, 8, 128, 64),
    ([1] * 5, [1, 64, 65, 200, 1031], 40, 8, 128, 32),
    ([1] * 3, [33, 16, 300], 12, 4, 64, 128),
    ([1] * 2, [500, 700], 11, 1, 128, 64),       # 11 query heads on one KV head
    ([1] * 2, [129, 257], 72, 2, 64, 256),       # 36 query heads on one KV head
    ([2] * 3, [2, 90, 301], 16, 4, 128, 16),
    ([4] * 2, [77, 1200], 40, 8, 128, 64),
    ([9], [999], 32, 8, 128, 64),
    ([16] * 2, [16, 515], 40, 8, 128, 32),
    ([3, 1, 0, 7], [30, 1, 5, 700], 16, 8, 64, 16),  # ragged; one sequence adds nothing
    ([33], [33], 6, 2, 64, 16),
    ([70], [300], 8, 8, 128, 64),
    ([129, 1, 40], [129, 400, 41], 16, 4, 64, 32),
    ([130, 257], [700, 257], 10, 2, 128, 64),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens,hq,hk,d,page_size", SHAPES)
def test_causal(fmt, q_lens, kv_lens, hq, hk, d, page_size):
    b = Batch(fmt, q_lens, kv_lens, hq, hk, d, page_size, seed=len(q_lens) + kv_lens[-1])
    for dtype in (torch.bfloat16, torch.float32):
        b.check(b.run(out_dtype=dtype))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [1, 5, 16, 100, 5000])
@pytest.mark.parametrize("q_len", [1, 6, 50, 140])
def test_window(fmt, window, q_len):
    b = Batch(fmt, [q_len] * 2, [q_len + 3, 900], 8, 2, 128, 16, seed=window)
    # pages that lie before every query's window are no longer the sequence's
    for s, kv in enumerate(b.kv_lens):
        gone = max(0, kv - q_len + 1 - window) // 16
        keep = b.table[s, :gone].clone()
        b.table[s, :gone] = -1
        got = b.run(out_dtype=torch.float32, window=window)
        b.table[s, :gone] = keep
    b.check(got, window=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,kv_lens,hq", [(1, [1, 40], 8), (5, [5, 333], 10), (16, [900, 17], 40), (64, [64, 500], 8)])
def test_tree(fmt, q_len, kv_lens, hq):
    b = Batch(fmt, [q_len] * 2, kv_lens, hq, 2, 128, 32, seed=q_len)
    rng = np.random.default_rng(q_len)
    words = [rng.integers(0, 2 ** 63, dtype=np.int64) & (2 ** q_len - 1 if q_len < 64 else -1) for _ in range(2 * q_len)]
    words[0] = 0                          # sees no new token: with kv_len = q_len, nothing at all
    if q_len == 64:
        words[1] = -1                     # the sign bit is new token 63
    tree = torch.tensor(words, device=DEV)
    got = b.run(out_dtype=torch.float32, tree=tree)
    b.check(got, tree=tree)
    if kv_lens[0] == q_len:
        assert (got[0] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [0, 300]), ([5, 40, 3], [77, 0, 130]), ([200], [333])])
def test_cross_attention(fmt, q_lens, kv_lens):
    """Not causal: keys of another length than the queries, none among them."""
    b = Batch(fmt, q_lens, kv_lens, 12, 3, 64, 16, seed=5)
    got = b.run(out_dtype=torch.float32, causal=False)
    b.check(got, causal=False)
    if 0 in kv_lens:
        at = sum(q_lens[:kv_lens.index(0)])
        assert (got[at:at + q_lens[kv_lens.index(0)]] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale,q_scale,spread", [(0.0, 1.0, 1.0), (-0.3, 1.0, 2.0), (0.0883883, 12.0, 0.0), (1.0, 2.0 ** -30, 6.0), (3.0, 4.0, 1.0)])
def test_scales(fmt, scale, q_scale, spread):
    """Flat and sharp softmaxes, V rows of very different magnitudes."""
    for q_len in (1, 48):
        b = Batch(fmt, [q_len], [777], 8, 2, 128, 64, seed=3, q_scale=q_scale, spread=spread)
        b.check(b.run(out_dtype=torch.float32, scale=scale), scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 8, 80, 150])
def test_weight_on_small_values(fmt, q_len):
    """The softmax picks keys whose V is 2^12 times smaller than its neighbours'."""
    b = Batch(fmt, [q_len], [400], 4, 2, 128, 64, seed=8, q_scale=3.0)
    k = torch.randn(400, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    v = torch.randn(400, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(2))
    strong = torch.arange(400, device=DEV) % 7 == 3
    v[~strong] *= 2.0 ** 12
    k[~strong] *= 0.05
    b.put(0, k.to(torch.bfloat16), v.to(torch.bfloat16))
    b.check(b.run(out_dtype=torch.float32, scale=0.5), scale=0.5)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 9, 66, 140])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_numbers(fmt, q_len, bad):
    """NaN and infinities in K, V and q reach the tokens that see them, and no other."""
    kv = 300
    b = Batch(fmt, [q_len], [kv], 8, 2, 128, 32, seed=2)
    k = torch.randn(kv, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(torch.bfloat16)
    v = torch.randn(kv, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).to(torch.bfloat16)
    if q_len > 4:  # seen by the later new tokens only, under one KV head each
        k[kv - 3, 0, 5] = bad
        v[kv - 2, 1, 77] = bad
        b.q[1, 2, 3] = bad
    else:
        v[10, 1, 0] = bad
    b.put(0, k, v)
    got = b.run(out_dtype=torch.float32)
    b.check(got)
    assert torch.isnan(got).any() and not torch.isnan(got).all()
    if q_len > 4:  # before the window's start they are seen by none
        got = b.run(out_dtype=torch.float32, window=1)
        b.check(got, window=1)


@pytest.mark.parametrize("q_len", [1, 20, 160])
def test_strides_streams_and_reuse(q_len):
    """q and out as column ranges of wider rows, on another stream, with one workspace for calls of several shapes."""
    b = Batch(g.NVFP4_KV_NVFP4, [q_len] * 2, [333, 512], 8, 2, 128, 64, seed=1)
    wide = torch.zeros(2 * q_len, 12 * 128 + 8, dtype=torch.bfloat16, device=DEV)
    wide[:, 256:256 + 8 * 128] = b.q.flatten(1)
    q = wide[:, 256:256 + 8 * 128].unflatten(1, (8, 128))
    outs = torch.full((2 * q_len, 10 * 128), 3.0, device=DEV)
    out = outs[:, 128:9 * 128].unflatten(1, (8, 128))
    big = Batch(g.NVFP4_KV_E4M3, [200], [300], 40, 8, 128, 16)
    need = max(g.nvfp4_paged_attention_workspace_bytes(x.cache, x.q, len(x.q_lens), max(x.q_lens)) for x in (b, big))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        g.nvfp4_paged_attention(q, b.cache, b.table, b.lens, out=out, workspace=ws, stream=s)
        other = torch.empty_like(big.q)
        g.nvfp4_paged_attention(big.q, big.cache, big.table, big.lens, out=other, workspace=ws, stream=s)
    s.synchronize()
    b.check(out)
    big.check(other)
    assert (outs[:, :128] == 3).all() and (outs[:, 9 * 128:] == 3).all()
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_graph_replays_with_other_lengths(fmt):
    """One captured decode step, replayed as the sequences grow across page boundaries; repeated calls agree bit for bit."""
    hq, hk, d, ps = 16, 4, 128, 16
    b = Batch(fmt, [1, 1], [15, 130], hq, hk, d, ps, seed=6, extra_width=8)
    free = [p for p in range(b.cache.n_pages + 0) if p not in set(b.table.flatten().tolist())]
    k = torch.zeros(2, hk, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    slots = torch.zeros(2, dtype=torch.int64, device=DEV)
    out = torch.empty_like(b.q)
    ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(b.cache, b.q, 2, 1), dtype=torch.uint8, device=DEV)

    def step():
        g.nvfp4_kv_append(b.cache, k, v, slots, workspace=ws)
        g.nvfp4_paged_attention(b.q, b.cache, b.table, b.lens, out=out, workspace=ws)

    slots.fill_(-1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    gen = torch.Generator(DEV).manual_seed(0)
    for _ in range(4):
        for s in range(2):
            b.kv_lens[s] += 1
            col = (b.kv_lens[s] - 1) // ps
            if b.table[s, col] < 0:
                b.table[s, col] = free.pop()
            slots[s] = b.slots(s, b.kv_lens[s])[-1]
        b.lens.copy_(torch.tensor(b.kv_lens, dtype=torch.int32))
        for x in (k, v, b.q):
            x.copy_(torch.randn(x.shape, device=DEV, generator=gen))
        graph.replay()
        first = out.clone()
        b.check(first)
        graph.replay()
        assert torch.equal(out, first)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)


@pytest.mark.parametrize("q_len", [1, 100])
def test_indices_out_of_bounds_are_left_out_and_reported(q_len):
    b = Batch(g.NVFP4_KV_E4M3, [q_len] * 2, [300, 400], 8, 2, 128, 16, seed=4)
    ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(b.cache, b.q, 2, q_len), dtype=torch.uint8, device=DEV)

    def status():
        return g.nvfp4_device_status(ws)

    b.check(b.run(out_dtype=torch.float32, workspace=ws))
    assert status() == (g.NVFP4_OK, 0)
    for page in (-1, b.cache.n_pages, 2 ** 31 - 1):  # a page outside the pool
        keep = b.table[0, 4].clone()
        b.table[0, 4] = page
        got = b.run(out_dtype=torch.float32, workspace=ws)
        assert status() == (g.NVFP4_ERR_DEVICE_INDEX, 43)
        assert torch.isfinite(got).all()
        b.table[0, 4] = keep
    for length in (2 ** 31 - 1, -5):                 # a length that the table cannot hold
        b.lens[0] = length
        got = b.run(out_dtype=torch.float32, workspace=ws)
        assert status() == (g.NVFP4_ERR_DEVICE_INDEX, 43)
    b.lens[0] = 300
    for bad in ([0, 500, 2 * q_len], [-7, q_len, 2 * q_len], [0, q_len, q_len - 1]):
        b.offsets.copy_(torch.tensor(bad, dtype=torch.int32))
        out = torch.zeros_like(b.q)
        g.nvfp4_paged_attention(b.q, b.cache, b.table, b.lens, q_offsets=b.offsets, max_q_len=q_len, out=out, workspace=ws)
        assert status() == (g.NVFP4_ERR_DEVICE_INDEX, 43)
    if q_len > 50:                                   # fewer keys than new tokens
        b.lens[0] = 50
        got = b.run(out_dtype=torch.float32, workspace=ws)
        assert status() == (g.NVFP4_ERR_DEVICE_INDEX, 43)
        assert (got[:q_len - 50] == 0).all() and torch.isfinite(got).all()
        b.lens[0] = 300
    b.check(b.run(out_dtype=torch.float32, workspace=ws))
    assert status() == (g.NVFP4_OK, 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_context(fmt):
    """Decode and a few tokens over a context long enough to be split over every SM, with page offsets beyond 2^31 bytes."""
    kv, hk, d, ps = 70001, 2, 128, 64
    pages = (1 << 31) // g.nvfp4_kv_page_bytes(ps, hk, d, fmt) + 2 * (kv // ps) + 64
    cache = g.KVCache.empty(pages, ps, hk, d, fmt, device=DEV)
    need = -(-kv // ps)
    table = (pages - 1 - torch.arange(need, dtype=torch.int32)).to(DEV)[None].contiguous()
    gen = torch.Generator(DEV).manual_seed(1)
    k, v = (torch.randn(kv, hk, d, device=DEV, generator=gen).to(torch.bfloat16) for _ in range(2))
    at = torch.arange(kv, device=DEV)
    slots = table[0].long()[at // ps] * ps + at % ps
    g.nvfp4_kv_append(cache, k, v, slots)
    ck, cv = (ref.to_np(x) for x in g.nvfp4_kv_read(cache, slots))
    lens = torch.tensor([kv], dtype=torch.int32, device=DEV)
    for q_len in (1, 7, 40):
        q = torch.randn(q_len, 8, d, device=DEV, generator=gen).to(torch.bfloat16)
        got = g.nvfp4_paged_attention(q, cache, table, lens, out_dtype=torch.float32)
        rows = sorted({0, q_len // 2, q_len - 1})
        see = ref.visible(q_len, kv)[rows]
        out, weight, s = ref.attention(ref.to_np(q)[rows], ck, cv, see, d ** -0.5)
        assert (np.abs(ref.to_np(got)[rows] - out) <= ref.tolerance(out, weight, s, got.dtype)).all()
