"""The status word of the KV-cache and attention calls: what is reported, and
that a wait that ran out stays visible whatever is reported after it."""
from __future__ import annotations

import pytest
import torch

import gemm_nvfp4_gb300 as g
from helpers import DEV
from test_gpu_attention import Batch

pytestmark = pytest.mark.gpu


def _workspace(b: Batch):
    return torch.zeros(g.nvfp4_paged_attention_workspace_bytes(b.cache, b.q, len(b.q_lens), max(b.q_lens)),
                       dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("q_len", [1, 40])
def test_an_index_does_not_hide_a_timeout(q_len):
    """The self-test's wait runs out (code 127); an attention, append and read with bad indices follow."""
    b = Batch(g.NVFP4_KV_E4M3, [q_len] * 2, [60, 90], 8, 2, 64, 16)
    ws = _workspace(b)
    g.nvfp4_selftest_wait_timeout(ws)
    b.table[0, 1] = -1
    b.run(workspace=ws)
    slots = torch.full((3,), 1 << 40, dtype=torch.int64, device=DEV)
    rows = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    g.nvfp4_kv_append(b.cache, rows, rows, slots, workspace=ws)
    g.nvfp4_kv_read(b.cache, slots, workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_ERR_DEVICE_TIMEOUT, 127)
    b.run(workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_ERR_DEVICE_INDEX, 43)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)


@pytest.mark.parametrize("hq", [8, 72])
def test_more_tokens_than_max_q_len_zero(hq):
    """max_q_len = 0 with offsets that hold tokens: no row is written, and code 43 says so."""
    b = Batch(g.NVFP4_KV_NVFP4, [3, 5], [60, 90], hq, 2, 64, 16)
    out = torch.full_like(b.q, 7.0)
    ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(b.cache, b.q, 2, 0), dtype=torch.uint8, device=DEV)
    g.nvfp4_paged_attention(b.q, b.cache, b.table, b.lens, q_offsets=b.offsets, max_q_len=0, out=out, workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_ERR_DEVICE_INDEX, 43)
    assert (out == 7).all()
    b.offsets.zero_()  # no sequence has any: nothing to report
    g.nvfp4_paged_attention(b.q, b.cache, b.table, b.lens, q_offsets=b.offsets, max_q_len=0, out=out, workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)
