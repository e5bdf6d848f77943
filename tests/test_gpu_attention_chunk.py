"""nvfp4_paged_attention with bf16 outputs, whose wide calls (more than 32 rows
per KV head) run on the tensor-core chunk kernel: its row tiles, key tiles,
splits and joins, masks, and what it must keep away from a row."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_nvfp4_gb300 as g
import kv_reference as ref
from helpers import DEV
from test_gpu_attention import FORMATS, Batch

pytestmark = pytest.mark.gpu


def check(b: Batch, got, **kw):
    """The bound of include/nvfp4.h for bf16 outputs: beside the fp32 one, what f16 weights lose
    (below 2^-32 of a row's largest: n * 2^-28 * max |V|), and the rounding of the result."""
    out, weight, s = b.want(**kw)
    pool = b.cache.pool.cpu().numpy()
    lost, at = np.zeros(out.shape), 0
    for i, (n, kv) in enumerate(zip(b.q_lens, b.kv_lens)):
        _, v = ref.cache_rows(pool, b.slots(i, kv).numpy(), b.cache.page_size, b.d, b.cache.format)
        if kv:
            lost[at:at + n] = kv * 2.0 ** -28 * np.nanmax(np.abs(v))
        at += n
    x = ref.to_np(got)
    assert np.array_equal(np.isnan(x), np.isnan(out))
    err, tol = np.abs(x - out), ref.tolerance(out, weight, s, torch.bfloat16) + lost
    ok = np.isnan(out) | (err <= tol)
    assert ok.all(), f"{(~ok).sum()} of {ok.size} out of bounds, worst {np.nanmax(err / tol):.3g} of the bound"


WIDE = [
    # q_lens, kv_lens, hq, hk, d, page_size
    ([33], [33], 1, 1, 64, 16),                  # one row tile, one key tile
    ([33], [1000], 2, 2, 128, 16),
    ([128], [128], 1, 1, 128, 32),               # a full row tile
    ([65] * 3, [65, 129, 700], 4, 2, 64, 256),
    ([16] * 5, [17, 128, 129, 255, 2000], 40, 8, 128, 64),
    ([129], [129], 2, 2, 64, 128),               # just past a row tile
    ([100] * 2, [333, 100], 12, 4, 128, 64),
    ([257], [600], 2, 1, 128, 16),
    ([300, 1, 77, 0, 513], [300, 1500, 77, 40, 900], 8, 2, 64, 32),
    ([260], [4000], 8, 8, 128, 64),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens,hq,hk,d,page_size", WIDE)
def test_wide(fmt, q_lens, kv_lens, hq, hk, d, page_size):
    b = Batch(fmt, q_lens, kv_lens, hq, hk, d, page_size, seed=kv_lens[-1])
    ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(b.cache, b.q, len(q_lens), max(q_lens)),
                     dtype=torch.uint8, device=DEV)
    first = b.run(workspace=ws)
    check(b, first)
    for _ in range(3):
        assert torch.equal(b.run(workspace=ws), first)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [1, 17, 128, 500])
@pytest.mark.parametrize("q_len", [40, 300])
def test_window(fmt, window, q_len):
    b = Batch(fmt, [q_len] * 2, [q_len + 3, 900], 4, 2, 128, 16, seed=window)
    keep = b.table.clone()
    for s, kv in enumerate(b.kv_lens):  # pages before every query's window are no longer the sequence's
        b.table[s, :max(0, kv - q_len + 1 - window) // 16] = -1
    ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(b.cache, b.q, 2, q_len), dtype=torch.uint8, device=DEV)
    got = b.run(window=window, workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)
    b.table.copy_(keep)
    check(b, got, window=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,kv_lens,hq", [(16, [900, 17], 40), (64, [64, 500], 8), (33, [40, 2000], 2), (40, [170, 41], 16)])
def test_tree(fmt, q_len, kv_lens, hq):
    b = Batch(fmt, [q_len] * 2, kv_lens, hq, 2, 128, 32, seed=q_len)
    rng = np.random.default_rng(q_len)
    words = [rng.integers(0, 2 ** 63, dtype=np.int64) & (2 ** q_len - 1 if q_len < 64 else -1) for _ in range(2 * q_len)]
    words[0] = 0
    words[1] = -1 if q_len == 64 else 1 << (q_len - 1)
    tree = torch.tensor(words, device=DEV)
    check(b, b.run(tree=tree), tree=tree)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens", [([50], [1]), ([200, 40, 3], [77, 0, 130]), ([150], [1333])])
def test_cross_attention(fmt, q_lens, kv_lens):
    b = Batch(fmt, q_lens, kv_lens, 6, 3, 64, 16, seed=5)
    got = b.run(causal=False)
    check(b, got, causal=False)
    if 0 in kv_lens:
        assert (got[200:240] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale,q_scale,spread", [(0.0, 1.0, 1.0), (-0.3, 1.0, 2.0), (0.0883883, 12.0, 0.0), (1.0, 2.0 ** -30, 3.0), (3.0, 4.0, 1.0)])
@pytest.mark.parametrize("q_len", [1, 40, 150])
def test_scales(fmt, scale, q_scale, spread, q_len):
    b = Batch(fmt, [q_len], [777], 4, 2, 128, 64, seed=3, q_scale=q_scale, spread=spread)
    check(b, b.run(scale=scale), scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 50, 150])
def test_weight_on_small_values(fmt, q_len):
    """The softmax picks keys whose V is 2^12 times smaller than its neighbours'."""
    b = Batch(fmt, [q_len], [400], 4, 2, 128, 64, seed=8, q_scale=3.0)
    k = torch.randn(400, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    v = torch.randn(400, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(2))
    strong = torch.arange(400, device=DEV) % 7 == 3
    v[~strong] *= 2.0 ** 12
    k[~strong] *= 0.05
    b.put(0, k.to(torch.bfloat16), v.to(torch.bfloat16))
    check(b, b.run(scale=0.5), scale=0.5)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [40, 150])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_numbers(fmt, q_len, bad):
    kv = 300
    b = Batch(fmt, [q_len], [kv], 4, 2, 128, 32, seed=2)
    k = torch.randn(kv, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(torch.bfloat16)
    v = torch.randn(kv, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).to(torch.bfloat16)
    k[kv - 3, 0, 5] = bad
    v[kv - 2, 1, 77] = bad
    b.q[1, 2, 3] = bad
    b.put(0, k, v)
    for window in (0, 1, 20):
        got = b.run(window=window)
        check(b, got, window=window)
        assert torch.isnan(got).any() and not torch.isnan(got).all()


@pytest.mark.parametrize("q_len", [40, 150])
def test_pages_out_of_bounds_are_left_out_and_reported(q_len):
    """The keys of a page that is not there count as not seen."""
    b = Batch(g.NVFP4_KV_NVFP4, [q_len] * 2, [300, 400], 4, 2, 128, 16, seed=4)
    ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(b.cache, b.q, 2, q_len), dtype=torch.uint8, device=DEV)
    keep = b.table[0, 4].clone()
    for page in (-1, b.cache.n_pages):
        b.table[0, 4] = page
        got = b.run(workspace=ws, causal=False)
        assert g.nvfp4_device_status(ws) == (g.NVFP4_ERR_DEVICE_INDEX, 43)
    b.table[0, 4] = keep
    # what is left: the same call on a sequence that never had those 16 keys
    pool = b.cache.pool.cpu().numpy()
    k, v = ref.cache_rows(pool, b.slots(0, 300).numpy(), 16, 128, b.cache.format)
    see = np.ones((q_len, 300), bool)
    see[:, 64:80] = False
    out, weight, s = ref.attention(ref.to_np(b.q[:q_len]), k, v, see, 128 ** -0.5)
    assert (np.abs(ref.to_np(got[:q_len]) - out) <= ref.tolerance(out, weight, s, torch.bfloat16)).all()
    check(b, b.run(workspace=ws))
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_context(fmt):
    """Chunks over a context that many CTAs share, with page offsets beyond 2^31 bytes, on both row-tile forms."""
    kv, hk, d, ps = 40003, 2, 128, 32
    pages = (1 << 31) // g.nvfp4_kv_page_bytes(ps, hk, d, fmt) + kv // ps + 64
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
    for q_len in (20, 131):
        q = torch.randn(q_len, 8, d, device=DEV, generator=gen).to(torch.bfloat16)
        got = g.nvfp4_paged_attention(q, cache, table, lens)
        rows = sorted({0, q_len // 2, q_len - 1})
        see = ref.visible(q_len, kv)[rows]
        out, weight, s = ref.attention(ref.to_np(q)[rows], ck, cv, see, d ** -0.5)
        tol = ref.tolerance(out, weight, s, got.dtype) + kv * 2.0 ** -28 * np.abs(cv).max()
        assert (np.abs(ref.to_np(got)[rows] - out) <= tol).all()
