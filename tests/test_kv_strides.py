"""Token strides of the KV-cache calls: one token's is never used, whatever it is."""
from __future__ import annotations

import pytest
import torch

import gemm_nvfp4_gb300 as g
from gemm_nvfp4_gb300 import binding
from helpers import DEV


def _one_token(heads, d, stride, device, fill=None):
    """[1, heads, d] in a row of `stride` elements."""
    x = torch.zeros(2 * stride, dtype=torch.bfloat16, device=device)
    t = x.as_strided((1, heads, d), (stride, d, 1))
    return t if fill is None else t.copy_(fill)


@pytest.mark.parametrize("stride", [1, 128, 513, 520])
def test_token_stride_of_one_token(stride):
    assert binding._head_rows(_one_token(4, 128, 520, "cpu").as_strided((1, 4, 128), (stride, 128, 1)), 4, 128,
                              (torch.bfloat16,), "x") == 512


@pytest.mark.gpu
@pytest.mark.parametrize("stride", [513, 520])
def test_calls_with_one_token_in_an_odd_row(stride):
    cache = g.KVCache.empty(4, 16, 4, 128, g.NVFP4_KV_E4M3, device=DEV)
    gen = torch.Generator(DEV).manual_seed(1)
    k, v, q = (torch.randn(1, 4, 128, device=DEV, generator=gen).to(torch.bfloat16) for _ in range(3))
    slots = torch.zeros(1, dtype=torch.int64, device=DEV)
    g.nvfp4_kv_append(cache, *(_one_token(4, 128, stride, DEV, x) for x in (k, v)), slots)
    out = tuple(_one_token(4, 128, stride, DEV) for _ in range(2))
    g.nvfp4_kv_read(cache, slots, out=out)
    for got, want in zip(out, g.nvfp4_kv_read(cache, slots)):
        assert torch.equal(got, want) and (got != 0).any()
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    got = g.nvfp4_paged_attention(_one_token(4, 128, stride, DEV, q), cache, table, lens, out=_one_token(4, 128, stride, DEV))
    assert torch.equal(got, g.nvfp4_paged_attention(q, cache, table, lens))
