"""nvfp4_paged_attention where a CTA has several work items, and batches with
more sequences than a CTA has threads: the walk from item to item, for every
form of the kernels, with every kind of mask.  Also the masks of small
speculative verifies with bf16 outputs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_nvfp4_gb300 as g
from helpers import DEV
from test_gpu_attention import FORMATS, Batch
from test_gpu_attention_chunk import check
from test_gpu_attention_isolation import run_and_check

pytestmark = pytest.mark.gpu


def _ragged(seed, seqs, q_most, kv_most, idle):
    """Lengths of a ragged batch: the longest first, short ones, and some that add nothing."""
    rng = np.random.default_rng(seed)
    q = [q_most] + [0 if rng.random() < idle else int(rng.integers(1, q_most + 1)) for _ in range(seqs - 1)]
    kv = [n + int(np.exp(rng.uniform(0, np.log(kv_most)))) for n in q]
    return q, kv


# (sequences, most new tokens, query heads, KV heads, most cached keys): rows of an item, and items a CTA of 152 or 304
FORMS = {
    "8 rows, 2 items a CTA": (80, 1, 32, 8, 700),
    "16 rows, 3 items a CTA": (60, 4, 32, 8, 400),
    "24 rows, 3 items a CTA": (60, 6, 32, 8, 400),
    "128 rows, 3 items a CTA": (60, 32, 16, 8, 300),
    "256 rows, 3 items a CTA": (28, 80, 16, 8, 300),
    "256 rows, 2 blocks a sequence": (20, 140, 16, 8, 100),
    "8 rows, more sequences than threads": (700, 1, 2, 1, 60),
    "32 rows, more sequences than threads": (700, 30, 2, 2, 60),
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("form", FORMS)
def test_ragged_batches(fmt, form):
    seqs, q_most, hq, hk, kv_most = FORMS[form]
    q, kv = _ragged(len(form), seqs, q_most, kv_most, idle=0.0 if q_most == 1 else 0.2)
    if q_most == 30:  # rows cost the reference more than the kernel: a few long ones
        q = [n if i % 9 == 0 else min(n, 2) for i, n in enumerate(q)]
    b = Batch(fmt, q, kv, hq, hk, 64 if fmt == g.NVFP4_KV_E4M3 else 128, 32, seed=1)
    run_and_check(b)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("mode", ["window", "tree", "cross"])
@pytest.mark.parametrize("seqs,q_len,hq", [(80, 1, 8), (40, 4, 32), (40, 6, 32), (40, 16, 16), (20, 60, 40)])
def test_masks_over_many_items(fmt, mode, seqs, q_len, hq):
    d = 128 if fmt == g.NVFP4_KV_E4M3 else 64
    kv = _ragged(q_len, seqs, q_len, 400, 0.0)[1]
    b = Batch(fmt, [q_len] * seqs, [max(n, q_len) for n in kv], hq, 8, d, 64, seed=2)
    words = np.random.default_rng(q_len).integers(0, 2 ** 63, seqs * q_len, dtype=np.int64) & (2 ** q_len - 1)
    run_and_check(b, **{"window": dict(window=50), "cross": dict(causal=False),
                        "tree": dict(tree=torch.from_numpy(words).to(DEV))}[mode])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [3, 6])
@pytest.mark.parametrize("mode", ["causal", "window", "tree", "cross"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_not_numbers_in_a_small_verify(fmt, q_len, mode, bad):
    """bf16 outputs of 12 and 24 rows."""
    kv = 300
    b = Batch(fmt, [q_len], [kv], 8, 2, 128, 32, seed=2)
    k, v = (torch.randn(kv, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(s)).to(torch.bfloat16) for s in (1, 2))
    k[kv - 2, 0, 5] = bad
    v[kv - 1, 1, 77] = bad
    b.q[0, 2, 3] = bad
    b.put(0, k, v)
    tree = torch.tensor([(1 << i) | 1 for i in range(q_len)], device=DEV)
    kw = {"causal": {}, "window": dict(window=2), "cross": dict(causal=False), "tree": dict(tree=tree)}[mode]
    got = b.run(**kw)
    check(b, got, **kw)
    assert torch.isnan(got).any() and (mode == "cross" or not torch.isnan(got).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 6, 40, 140])
def test_window_whose_earlier_pages_are_gone(fmt, q_len):
    """All sequences' pages before their windows are another owner's, in one call, and none is looked at."""
    window = 37
    b = Batch(fmt, [q_len] * 3, [q_len + 3, 900, 500], 8, 2, 128, 16, seed=window)
    keep = b.table.clone()
    for s, kv in enumerate(b.kv_lens):
        b.table[s, :max(0, kv - q_len + 1 - window) // 16] = -1
    ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(b.cache, b.q, 3, q_len), dtype=torch.uint8, device=DEV)
    outs = [b.run(window=window, workspace=ws, out_dtype=t) for t in (torch.bfloat16, torch.float32)]
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)
    b.table.copy_(keep)
    run_and_check(b, window=window)
    for got, t in zip(outs, (torch.bfloat16, torch.float32)):
        assert torch.equal(got, b.run(window=window, out_dtype=t))
