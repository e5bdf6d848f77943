"""Refusals of the KV-cache calls (before anything touches a GPU), and pins of
the reference that their GPU tests compare with."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import gemm_nvfp4_gb300 as g
import kv_reference as ref
from gemm_nvfp4_gb300 import binding, build

FAKE = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return g.load_library()


def _cache(**kw):
    f = dict(pool=FAKE, n_pages=4, page_size=64, n_kv_heads=8, head_dim=128, format=0)
    f.update(kw)
    return binding.KVCacheC(**f)


def test_page_bytes(lib):
    assert g.nvfp4_kv_page_bytes(64, 8, 128, g.NVFP4_KV_E4M3) == 64 * 8 * 2 * 129
    assert g.nvfp4_kv_page_bytes(16, 1, 64, g.NVFP4_KV_NVFP4) == 16 * 2 * (32 + 4 + 1)
    for bad in ((0, 8, 128, 0), (48, 8, 128, 0), (8, 8, 128, 0), (512, 8, 128, 0), (64, 0, 128, 0), (64, 1025, 128, 0),
                (64, 8, 96, 0), (64, 8, 256, 0), (64, 8, 128, 2), (64, 8, 128, -1)):
        assert g.nvfp4_kv_page_bytes(*bad) == 0, bad


@pytest.mark.parametrize("call", ["nvfp4_kv_append", "nvfp4_kv_read"])
def test_rows_refuse_bad_arguments(lib, call):
    def run(cache=None, k=FAKE, k_ld=1024, v=FAKE, v_ld=1024, slots=FAKE, n=3, ws=None, wsb=0, **kw):
        c = _cache(**kw) if cache is None else cache
        return getattr(lib, call)(ctypes.byref(c), k, k_ld, v, v_ld, slots, n, ws, wsb, None)

    assert getattr(lib, call)(None, FAKE, 1024, FAKE, 1024, FAKE, 3, None, 0, None) == binding.NVFP4_ERR_INVALID_ARG
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(slots=FAKE + 4),
               dict(k_ld=1016), dict(v_ld=0), dict(k_ld=1028), dict(v_ld=1025), dict(k_ld=1 << 62), dict(n=-1),
               dict(pool=None), dict(pool=FAKE + 8), dict(n_pages=-1), dict(n_pages=1 << 31), dict(ws=FAKE + 4, wsb=256)):
        assert run(**kw) == binding.NVFP4_ERR_INVALID_ARG, kw
    for kw in (dict(page_size=24), dict(head_dim=80), dict(format=5), dict(n_kv_heads=0), dict(n=1 << 27)):
        assert run(**kw) == binding.NVFP4_ERR_UNSUPPORTED_SHAPE, kw
    assert run(ws=FAKE, wsb=255) == binding.NVFP4_ERR_WORKSPACE
    assert run(n=0, k=None, v=None, slots=None) == binding.NVFP4_OK


def test_attention_refuses_bad_arguments(lib):
    base = dict(q=FAKE, q_ld=4096, out=FAKE, out_ld=4096, block_table=FAKE, table_width=10, kv_lens=FAKE, n_seqs=2,
                total_q=2, max_q_len=1, n_q_heads=32, out_dtype=1, causal=1, scale=0.1)

    def run(ws=FAKE, wsb=None, cache=None, **kw):
        a = binding.PagedAttentionArgsC(cache=_cache(**(cache or {})), **{**base, **kw})
        need = lib.nvfp4_paged_attention_workspace_bytes(ctypes.byref(a))
        return lib.nvfp4_paged_attention(ctypes.byref(a), ws, need if wsb is None else wsb, None)

    assert lib.nvfp4_paged_attention(None, FAKE, 1 << 30, None) == binding.NVFP4_ERR_INVALID_ARG
    assert lib.nvfp4_paged_attention_workspace_bytes(None) == 0
    for kw in (dict(q=None), dict(out=None), dict(kv_lens=None), dict(block_table=None), dict(q=FAKE + 8),
               dict(out=FAKE + 8), dict(kv_lens=FAKE + 2), dict(block_table=FAKE + 1), dict(q_offsets=FAKE + 2),
               dict(tree=FAKE + 4), dict(q_ld=4088), dict(out_ld=100), dict(q_ld=4100), dict(out_ld=4097), dict(n_seqs=-1),
               dict(total_q=3), dict(total_q=-2), dict(causal=2), dict(window=-1), dict(window=5, causal=0),
               dict(tree=FAKE, causal=0), dict(tree=FAKE, window=4), dict(scale=math.nan), dict(scale=math.inf),
               dict(out_dtype=3), dict(table_width=-1), dict(ws=None), dict(ws=FAKE + 8), dict(cache=dict(pool=None)),
               dict(cache=dict(n_pages=-1))):
        assert run(**kw) == binding.NVFP4_ERR_INVALID_ARG, kw
    for kw in (dict(n_q_heads=12), dict(n_q_heads=0), dict(n_seqs=65536, total_q=65536), dict(max_q_len=3),
               dict(tree=FAKE, max_q_len=65, total_q=130), dict(cache=dict(page_size=100)), dict(cache=dict(head_dim=32))):
        assert run(**kw) == binding.NVFP4_ERR_UNSUPPORTED_SHAPE, kw
    a = binding.PagedAttentionArgsC(cache=_cache(), **base)
    need = lib.nvfp4_paged_attention_workspace_bytes(ctypes.byref(a))
    assert need >= 256
    assert run(wsb=need - 1) == binding.NVFP4_ERR_WORKSPACE
    assert run(n_seqs=0, total_q=0, max_q_len=0, q=None, out=None) == binding.NVFP4_OK


def test_python_checks():
    cache = g.KVCache(torch.zeros(4, 2, 2, 16 * 65, dtype=torch.uint8), 16, 64, g.NVFP4_KV_E4M3)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="pool"):
        g.nvfp4_kv_append(g.KVCache(cache.pool, 32, 64, g.NVFP4_KV_E4M3), k, k, slots)
    with pytest.raises(ValueError, match="k must"):
        g.nvfp4_kv_append(cache, k.float(), k, slots)
    with pytest.raises(ValueError, match="v must"):
        g.nvfp4_kv_append(cache, k, k[:, :1], slots)
    with pytest.raises(ValueError, match="side by side"):
        g.nvfp4_kv_append(cache, k.transpose(1, 2).contiguous().transpose(1, 2), k, slots)
    with pytest.raises(ValueError, match="slots"):
        g.nvfp4_kv_append(cache, k, k, slots.int())
    with pytest.raises(ValueError, match="tokens"):
        g.nvfp4_kv_append(cache, k, k[:2], slots)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 5, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="same number"):
        g.nvfp4_paged_attention(q, cache, table, lens)
    with pytest.raises(ValueError, match="max_q_len"):
        g.nvfp4_paged_attention(q, cache, table, lens, q_offsets=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="block_table"):
        g.nvfp4_paged_attention(q[:3], cache, table[:2], lens)
    with pytest.raises(ValueError, match="tree"):
        g.nvfp4_paged_attention(q[:3], cache, table, lens, tree=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(g.NVFP4Error):
        g.KVCache.empty(4, 48, 2, 64, device="cpu")


def test_reference_tables_and_rows():
    """Hand-worked values of the reference itself."""
    assert ref.E4M3_VALUES[0x7E] == 448 and ref.E4M3_VALUES[0x08] == 2.0 ** -6 and ref.E4M3_VALUES[1] == 2.0 ** -9
    assert np.array_equal(ref.E4M3_VALUES[:127].astype(np.float32),
                          torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy())
    x = np.zeros(64)
    x[:4] = 448, 17, 19, -17                    # 17 lies between 16 and 18: a tie, to the even code
    codes, _, e = ref.encode_row(x, ref.E4M3)
    assert e == 127 and ref.E4M3_VALUES[codes[:4]].tolist() == [448, 16, 20, -16]
    codes, _, e = ref.encode_row(x * 2, ref.E4M3)
    assert e == 128
    codes, _, e = ref.encode_row(x * 1.01, ref.E4M3)
    assert e == 128                             # past 448: the next power of two
    x = np.zeros(64)
    x[:5] = 2688, -0.25 * 448, 0.75 * 448, 5 * 448, 1e-3
    codes, scales, e = ref.encode_row(x, ref.NVFP4)
    assert e == 127 and scales.tolist() == [0x7E, 0, 0, 0]
    assert codes[:3].tolist() == [7 | 8 << 4, 2 | 6 << 4, 0]
    assert ref.decode_rows(codes, scales, np.array(e), ref.NVFP4)[:4].tolist() == [2688, 0, 448, 1792]
    assert ref.encode_row(np.full(64, math.inf), ref.E4M3)[2] == 255
    assert ref.encode_row(np.zeros(64), ref.NVFP4)[2] == 27


def test_reference_attention():
    """Equal scores average V; one far larger score picks it; a tree word of zero sees the past alone."""
    k, v = np.zeros((3, 1, 4)), np.arange(12.0).reshape(3, 1, 4)
    q = np.zeros((1, 2, 4))
    out, weight, s = ref.attention(q, k, v, np.ones((1, 3), bool), 1.0)
    np.testing.assert_allclose(out[0, 1], v[:, 0].mean(0))
    k[2] = 100
    out, _, _ = ref.attention(np.ones((1, 1, 4)), k, v, np.ones((1, 3), bool), 1.0)
    np.testing.assert_allclose(out[0, 0], v[2, 0])
    assert ref.visible(2, 5, tree=np.array([0, 1])).tolist() == [[True] * 3 + [False] * 2, [True] * 4 + [False]]
    assert ref.visible(2, 4, window=2).tolist() == [[False, True, True, False], [False, False, True, True]]
    assert ref.visible(2, 1).tolist() == [[False], [True]]
