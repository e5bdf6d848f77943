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
