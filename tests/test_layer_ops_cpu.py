"""Refusals of the products with an epilogue, the rotary positions and the attention over whole prompts (before
anything touches a GPU), and the frequency table, which is made on the host."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import gemm_nvfp4_gb300 as g
from gemm_nvfp4_gb300 import binding, build

FAKE = 1 << 20  # an aligned address that is never dereferenced
BAD, SHAPE = binding.NVFP4_ERR_INVALID_ARG, binding.NVFP4_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return g.load_library()


def test_epilogue_refuses_bad_arguments(lib):
    def run(fp6=False, x=FAKE, N=4, codes=FAKE, scales=FAKE, ts=FAKE, M=64, K=128, ep=True, y=FAKE, out=0, ws=FAKE, wsb=1 << 30, **kw):
        e = binding.EpilogueC(**{**dict(bias=FAKE, residual=FAKE, residual_ld=64), **kw})
        e = ctypes.byref(e) if ep else None
        if fp6:
            return lib.nvfp4_fp6_gemm_epilogue(x, N, codes, scales, M, K, e, y, out, ws, wsb, None)
        return lib.nvfp4_gemm_epilogue(x, N, codes, scales, ts, M, K, e, y, out, ws, wsb, None)

    for fp6 in (False, True):
        for kw in (dict(ep=False), dict(x=None), dict(codes=None), dict(scales=None), dict(y=None), dict(x=FAKE + 8), dict(y=FAKE + 4),
                   dict(N=-1), dict(M=-1), dict(out=2), dict(activation=-1), dict(activation=6), dict(bias_dtype=2),
                   dict(residual_dtype=-1), dict(bias=FAKE + 2), dict(bias=FAKE + 1, bias_dtype=1), dict(residual=FAKE + 2),
                   dict(residual=FAKE + 1, residual_dtype=1), dict(residual_ld=63), dict(residual_ld=1 << 61), dict(ws=None),
                   dict(ws=FAKE + 8)):
            assert run(fp6, **kw) == BAD, (fp6, kw)
        assert run(fp6, K=0) == SHAPE
        assert run(fp6, K=40) == SHAPE
        assert run(fp6, wsb=16) == binding.NVFP4_ERR_WORKSPACE
        assert run(fp6, N=0, x=None, y=None) == binding.NVFP4_OK
        assert run(fp6, M=0, y=None, ws=None, wsb=0) == binding.NVFP4_OK
        # in place, but with another type or stride than the output's
        assert run(fp6, residual_dtype=1) == BAD
        assert run(fp6, residual_ld=72) == BAD
    assert run(ts=None) == BAD


def test_rope_refuses_bad_arguments(lib):
    base = dict(q=FAKE, k=FAKE, q_ld=4096, k_ld=1024, q_out=FAKE, k_out=FAKE, q_out_ld=4096, k_out_ld=1024, positions=FAKE,
                positions_ld=3, pairs=FAKE, n_tokens=3, n_axes=2, n_pairs=64, n_q_heads=32, n_k_heads=8, head_dim=128, dtype=1,
                scale=1.0)

    def run(**kw):
        return lib.nvfp4_rope(ctypes.byref(binding.RopeArgsC(**{**base, **kw})), None)

    assert lib.nvfp4_rope(None, None) == BAD
    for kw in (dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(positions=None), dict(pairs=None), dict(q=FAKE + 8),
               dict(k=FAKE + 2), dict(q_out=FAKE + 4), dict(k_out=FAKE + 8), dict(positions=FAKE + 4), dict(pairs=FAKE + 8),
               dict(q_ld=4088), dict(k_ld=1020), dict(q_out_ld=4100), dict(k_out_ld=0), dict(q_ld=1 << 62), dict(positions_ld=2),
               dict(n_tokens=-1), dict(dtype=2), dict(adjacent=2), dict(inverse=-1), dict(scale=math.nan), dict(scale=math.inf),
               dict(dtype=0, q_ld=4098)):
        assert run(**kw) == BAD, kw
    for kw in (dict(head_dim=120 + 4), dict(head_dim=0), dict(head_dim=520), dict(n_pairs=65), dict(n_pairs=-1), dict(n_axes=0),
               dict(n_axes=257), dict(n_q_heads=-1), dict(n_k_heads=8193), dict(n_tokens=1 << 31)):
        assert run(**kw) == SHAPE, kw
    assert run(n_tokens=0, q=None, positions=None) == binding.NVFP4_OK
    assert run(n_q_heads=0, n_k_heads=0, q=None, k=None) == binding.NVFP4_OK


def test_frequency_table_against_exact_arithmetic(lib):
    """Each entry is the nearest integer to inv_freq / (2 pi) * 2^64, modulo 2^64."""
    mpmath = pytest.importorskip("mpmath")
    freq = [1.0, 1e-6, 0.5, -0.25, 12345.678, 2.0 ** 31 - 1, -2.0 ** 30, 1e-30, 5e-324, 0.0, 3.1e-5, math.pi, 2 * math.pi]
    freq += [1e6 ** (-2 * i / 128) for i in range(64)]
    axis = [i % 5 for i in range(len(freq))]
    table = g.nvfp4_rope_pairs(freq, axis)
    turns = table.view(torch.int64)[:, 0].tolist()
    with mpmath.workprec(400):
        for f, t in zip(freq, turns):
            want = int(mpmath.nint(mpmath.mpf(f) / (2 * mpmath.pi) * mpmath.mpf(2) ** 64)) % 2 ** 64
            assert t % 2 ** 64 == want, f
    assert table.view(torch.int32)[:, 2].tolist() == axis
    assert g.RopeTable.make(freq, axis, device="cpu").n_axes == 5 and g.RopeTable.make(freq, device="cpu").n_axes == 1


def test_frequency_table_refusals(lib):
    for bad in ([math.nan], [math.inf], [2.0 ** 31], [-2.0 ** 40]):
        with pytest.raises(g.NVFP4Error):
            g.nvfp4_rope_pairs(bad)
    for axis in ([-1], [256]):
        with pytest.raises(g.NVFP4Error):
            g.nvfp4_rope_pairs([1.0], axis)
    with pytest.raises(ValueError, match="axes"):
        g.nvfp4_rope_pairs([1.0, 2.0], [0])
    assert lib.nvfp4_rope_pairs(None, None, -1, None) == BAD
    assert lib.nvfp4_rope_pairs(None, None, 2, None) == BAD
    assert lib.nvfp4_rope_pairs(None, None, 0, None) == binding.NVFP4_OK


def test_prompt_attention_refuses_bad_arguments(lib):
    base = dict(q=FAKE, k=FAKE, v=FAKE, q_ld=4096, k_ld=1024, v_ld=1024, out=FAKE, out_ld=4096, offsets=FAKE, n_seqs=2, total=9,
                n_q_heads=32, n_kv_heads=8, head_dim=128, out_dtype=1, causal=1, scale=0.1)

    def run(ws=None, wsb=0, **kw):
        return lib.nvfp4_prompt_attention(ctypes.byref(binding.PromptAttentionArgsC(**{**base, **kw})), ws, wsb, None)

    assert lib.nvfp4_prompt_attention(None, None, 0, None) == BAD
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=FAKE + 8), dict(k=FAKE + 8), dict(v=FAKE + 2),
               dict(out=FAKE + 8), dict(offsets=FAKE + 2), dict(offsets=None), dict(q_ld=4088), dict(k_ld=1016), dict(v_ld=1028),
               dict(out_ld=0), dict(q_ld=1 << 40), dict(n_seqs=-1), dict(total=-1), dict(window=-1), dict(window=4, causal=0),
               dict(causal=2), dict(out_dtype=2), dict(scale=math.nan), dict(scale=-math.inf), dict(scale=3e38),
               dict(ws=FAKE + 8, wsb=256)):
        assert run(**kw) == BAD, kw
    for kw in (dict(head_dim=96), dict(head_dim=0), dict(n_q_heads=12), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_seqs=65536),
               dict(n_q_heads=129, n_kv_heads=1), dict(total=1 << 20)):
        assert run(**kw) == SHAPE, kw
    assert run(ws=FAKE, wsb=255) == binding.NVFP4_ERR_WORKSPACE
    assert run(total=0, q=None) == binding.NVFP4_OK
    assert run(n_seqs=0, q=None) == binding.NVFP4_OK


def test_python_checks():
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    W = g.NVFP4Weight(torch.zeros(64, 64, dtype=torch.uint8), torch.zeros(64, 8, dtype=torch.uint8), torch.ones(1))
    ws = torch.zeros(64, dtype=torch.uint8)
    for kw, match in ((dict(x=x.float()), "x must"), (dict(x=x[:, :64]), "x must"), (dict(bias=torch.zeros(63)), "bias"),
                      (dict(residual=torch.zeros(3, 65)), "residual"), (dict(residual=torch.zeros(64, 3).T), "residual"),
                      (dict(out=torch.zeros(3, 128)[:, :64]), "out must"), (dict(bias=torch.zeros(64, dtype=torch.float16)), "dtype"),
                      (dict(out=torch.zeros(3, 64)), "one CUDA device")):
        with pytest.raises(ValueError, match=match):
            g.nvfp4_gemm_epilogue(**{**dict(x=x, W=W, workspace=ws, out=torch.zeros(3, 64)), **kw})
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    table = g.RopeTable.make([1.0] * 32, [i % 2 for i in range(32)], device="cpu")
    at = torch.zeros(2, 3, dtype=torch.int64)
    for args, kw, match in (((q[0], k, at, table), {}, "q must"), ((q, k.float(), at, table), {}, "k must"),
                            ((q, k[:2], at, table), {}, "tokens"), ((q, k, at[0], table), {}, "axes"),
                            ((q, k, at.int(), table), {}, "positions"), ((q, k, at[:, :2], table), {}, "positions"),
                            ((q, None, at, table), dict(out=(q, k)), "out must"), ((q, k, at, table), dict(out=(k, q)), "out"),
                            ((q.half(), None, at, table), {}, "dtype"), ((q, k, at, table), {}, "one CUDA device")):
        with pytest.raises(ValueError, match=match):
            g.nvfp4_rope(*args, **kw)
    off = torch.tensor([0, 3], dtype=torch.int32)
    for args, kw, match in (((q[0], k, k), {}, "must be"), ((q, k, k.float()), {}, "v must"), ((q, k[:2], k), {}, "tokens"),
                            ((q, k, torch.zeros(3, 2, 32, dtype=torch.bfloat16)), {}, "v must"), ((q, k, k), dict(offsets=off.long()), "offsets"),
                            ((q, k, k), dict(offsets=off[:0]), "offsets"), ((q, k, k), dict(out=q.half()), "out must"),
                            ((q.transpose(0, 1), k, k), {}, "side by side|tokens"), ((q, k, k), dict(offsets=off), "one CUDA device")):
        with pytest.raises(ValueError, match=match):
            g.nvfp4_prompt_attention(*args, **kw)


def test_packed_argument_blocks_match_their_structures():
    """The blocks that the binding packs have their ctypes.Structure's fields at the same places."""
    for packed, structure in ((binding._ROPE_ARGS, binding.RopeArgsC), (binding._PROMPT_ARGS, binding.PromptAttentionArgsC)):
        values = [float(i + 1) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(structure._fields_)]
        assert packed.size == ctypes.sizeof(structure)
        assert packed.pack(*values) == bytes(structure(*values))


def test_rope_refuses_strides_between_one_row_and_all(lib):
    """One row of positions for every axis (0) is taken, and whole rows are; nothing between or below."""
    a = dict(q=FAKE, q_ld=512, q_out=FAKE, q_out_ld=512, positions=FAKE, pairs=FAKE, n_tokens=3, n_axes=2, n_pairs=64,
             n_q_heads=4, head_dim=128, dtype=1, scale=1.0)
    for ld in (-1, 1, 2, 1 << 60):
        assert lib.nvfp4_rope(ctypes.byref(binding.RopeArgsC(**a, positions_ld=ld)), None) == BAD, ld


def test_rope_refuses_an_output_that_is_its_input_with_another_stride(lib):
    a = dict(positions=FAKE, pairs=FAKE, n_axes=1, n_pairs=64, n_q_heads=4, n_k_heads=4, head_dim=128, dtype=1, scale=1.0,
             q=FAKE, q_ld=512, q_out=FAKE, q_out_ld=512, k=2 * FAKE, k_ld=520, k_out=2 * FAKE, k_out_ld=520)

    def run(**kw):
        return lib.nvfp4_rope(ctypes.byref(binding.RopeArgsC(**{**a, **kw})), None)

    for kw in (dict(q_ld=520), dict(q_out_ld=1024), dict(k_ld=512), dict(k_out_ld=512)):
        assert run(n_tokens=2, **kw) == BAD, kw


def test_prompt_attention_refuses_an_output_that_is_an_input(lib):
    a = dict(q=FAKE, k=2 * FAKE, v=3 * FAKE, q_ld=4096, k_ld=1024, v_ld=1024, out_ld=4096, n_seqs=1, total=9, n_q_heads=32,
             n_kv_heads=8, head_dim=128, out_dtype=1, causal=1, scale=0.1)
    for out in (FAKE, 2 * FAKE, 3 * FAKE):
        assert lib.nvfp4_prompt_attention(ctypes.byref(binding.PromptAttentionArgsC(**a, out=out)), None, 0, None) == BAD
