"""The KV-cache calls take tensors of one CUDA device and refuse any other."""
from __future__ import annotations

import pytest
import torch

import gemm_nvfp4_gb300 as g
from gemm_nvfp4_gb300 import build


def _tensors(device):
    """Everything that the calls take, for one token of two heads of 64."""
    cache = g.KVCache.empty(4, 16, 2, 64, g.NVFP4_KV_E4M3, device=device)
    rows = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=device)
    return dict(cache=cache, k=rows, v=rows.clone(), slots=torch.zeros(1, dtype=torch.int64, device=device), q=rows.clone(),
                table=torch.zeros(1, 1, dtype=torch.int32, device=device), lens=torch.ones(1, dtype=torch.int32, device=device),
                offsets=torch.tensor([0, 1], dtype=torch.int32, device=device),
                tree=torch.ones(1, dtype=torch.int64, device=device), out=torch.zeros_like(rows),
                ws=torch.zeros(1 << 22, dtype=torch.uint8, device=device))


def _append(t):
    g.nvfp4_kv_append(t["cache"], t["k"], t["v"], t["slots"], workspace=t["ws"])


def _read(t):
    g.nvfp4_kv_read(t["cache"], t["slots"], out=(t["k"], t["v"]), workspace=t["ws"])


def _attend(t):
    g.nvfp4_paged_attention(t["q"], t["cache"], t["table"], t["lens"], q_offsets=t["offsets"], max_q_len=1, tree=t["tree"],
                            out=t["out"], workspace=t["ws"])


CALLS = [(_append, ("cache", "k", "v", "slots", "ws")), (_read, ("cache", "k", "v", "slots", "ws")),
         (_attend, ("cache", "q", "table", "lens", "offsets", "tree", "out", "ws"))]


@pytest.mark.parametrize("call", [c for c, _ in CALLS])
def test_host_tensors_are_refused(call):
    build.build()
    with pytest.raises(ValueError, match="one CUDA device"):
        call(_tensors("cpu"))


@pytest.mark.gpu
@pytest.mark.parametrize("call,name", [(c, n) for c, names in CALLS for n in names])
def test_one_host_tensor_is_refused(call, name):
    """A host address never reaches a kernel."""
    t = _tensors("cuda:0")
    call(t)
    t[name] = _tensors("cpu")[name]
    with pytest.raises(ValueError, match="one CUDA device"):
        call(t)
    torch.cuda.synchronize()
