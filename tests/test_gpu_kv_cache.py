"""nvfp4_kv_append and nvfp4_kv_read against the format's definition, byte for
byte: formats, head layouts, page sizes, strided inputs, idle slots, rows that
sit on rounding ties, tiny, huge, zero and non-finite rows, and bad slots."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_nvfp4_gb300 as g
import kv_reference as ref
from helpers import DEV

pytestmark = pytest.mark.gpu

FORMATS = [g.NVFP4_KV_E4M3, g.NVFP4_KV_NVFP4]


def _cache(n_pages, page_size, heads, d, fmt, fill=None):
    cache = g.KVCache.empty(n_pages, page_size, heads, d, fmt, device=DEV)
    if fill is None:
        cache.pool.random_(0, 256, generator=torch.Generator(DEV).manual_seed(9))
    else:
        cache.pool.fill_(fill)
    return cache


def _rows(tokens, heads, d, seed):
    """K and V as column ranges of one buffer, of mixed magnitudes."""
    gen = torch.Generator(DEV).manual_seed(seed)
    buf = torch.randn(tokens, 4 * heads * d, device=DEV, generator=gen)
    buf *= torch.exp2(torch.randint(-20, 12, (tokens, 1), device=DEV, generator=gen).float())
    buf = buf.to(torch.bfloat16)
    w = heads * d
    return buf[:, w:2 * w].unflatten(1, (heads, d)), buf[:, 3 * w:].unflatten(1, (heads, d))


def _check(cache, before, k, v, slots):
    """The pool holds the encoded rows at the slots and `before` elsewhere; reading gives their values."""
    want = before.copy()
    ps, d, fmt = cache.page_size, cache.head_dim, cache.format
    codes, scales, e = ref.planes(want, ps, d, fmt)
    blocks = want.reshape(*want.shape[:3], -1)
    cb, sb = codes.shape[-1], scales.shape[-1]
    for t, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        page, at = divmod(s, ps)
        for h in range(cache.n_kv_heads):
            for j, x in enumerate((k, v)):
                c, sc, ex = ref.encode_row(ref.to_np(x[t, h]), fmt)
                block = blocks[page, h, j]
                block[at * cb:(at + 1) * cb] = c
                block[ps * cb + at * sb:ps * cb + (at + 1) * sb] = sc
                block[ps * (cb + sb) + at] = ex
    got = cache.pool.cpu().numpy()
    assert np.array_equal(got, want)
    rk, rv = g.nvfp4_kv_read(cache, slots)
    live = slots.cpu().numpy() >= 0
    wk, wv = ref.cache_rows(want, slots.cpu().numpy()[live], ps, d, fmt)
    for got_rows, want_rows in ((rk, wk), (rv, wv)):
        np.testing.assert_array_equal(ref.to_np(got_rows)[live], want_rows)
        assert (got_rows[torch.from_numpy(~live).to(DEV)] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,heads,d,page_size", [
    (1, 1, 64, 16), (1, 8, 128, 64), (3, 5, 64, 32), (17, 2, 128, 16), (61, 8, 128, 256), (130, 3, 128, 128)])
def test_append_and_read(fmt, tokens, heads, d, page_size):
    pages = -(-tokens // page_size) + 2
    cache = _cache(pages, page_size, heads, d, fmt)
    before = cache.pool.cpu().numpy()
    k, v = _rows(tokens, heads, d, seed=tokens)
    slots = torch.randperm(pages * page_size, generator=torch.Generator().manual_seed(tokens))[:tokens].to(DEV)
    if tokens > 2:
        slots[tokens // 2] = -1
    g.nvfp4_kv_append(cache, k, v, slots)
    _check(cache, before, k, v, slots)


@pytest.mark.parametrize("fmt", FORMATS)
def test_extreme_rows(fmt):
    """Rows chosen for the steps of the quantiser: the edges of the exponent, ties of codes and scales, and what is not a number."""
    d, rows = 128, []

    def row(*head, rest=0.0):
        x = torch.full((d,), rest)
        x[:len(head)] = torch.tensor(head)
        rows.append(x)

    row()                                              # all zero
    row(-0.0, 0.0)
    for top in (448.0, 2688.0, 450.0, 2704.0, 1.0):    # on and just past the largest value of an exponent
        row(top, -top / 2, top / 448, 3.0)
    row(448.0, 104.0, 108.0, 112.0, 116.0, 120.0, 17.0, 19.0, -17.0, -19.0, 0.0009765625, 0.0029296875)  # E4M3 ties
    row(6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -2.5, -5.0)                    # E2M1 ties
    row(2688.0, 672.0, 0.25 * 448, 0.75 * 448, 1.25 * 448, 1.75 * 448, 2.5 * 448, 3.5 * 448, 5 * 448)
    row(2.0 ** -126, 2.0 ** -133)                      # subnormal bf16 values
    row(2.0 ** -91, 2.0 ** -100, -2.0 ** -95)          # near the smallest exponent
    row(448 * 2.0 ** 100, 2.0 ** 100)                  # the largest E4M3 row
    row(450 * 2.0 ** 100, 1.0)                         # E4M3: out of range
    row(2688 * 2.0 ** 100, 2.0 ** 99)
    row(2704 * 2.0 ** 100, 2.0 ** 99)
    row(float("inf"), 1.0)
    row(1.0, -float("inf"))
    row(1.0, float("nan"), 2.0)
    x = torch.stack(rows)
    x = torch.cat((x, x.flip(1), -x)).to(torch.bfloat16).to(DEV)
    k = x[:, None].contiguous()
    v = x.flip(0)[:, None].contiguous()
    n = k.shape[0]
    cache = _cache(n // 16 + 1, 16, 1, d, fmt)
    before = cache.pool.cpu().numpy()
    slots = torch.arange(n, device=DEV)
    g.nvfp4_kv_append(cache, k, v, slots)
    _check(cache, before, k, v, slots)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_bf16_magnitude_of_a_binade_pair(fmt):
    """Rows that hold every bf16 value of a few binades beside maxima of every fraction: ties and near-ties of all kinds."""
    d = 128
    fractions = torch.arange(128) / 128 + 1
    rows = [torch.cat((m[None], fractions[:127] * s)) for m in fractions * 8 for s in (4.0, 0.5, 2.0 ** -6)]
    x = torch.stack(rows).to(torch.bfloat16).to(DEV)[:, None].contiguous()
    n = x.shape[0]
    cache = _cache(n // 64 + 1, 64, 1, d, fmt)
    before = cache.pool.cpu().numpy()
    slots = torch.arange(n, device=DEV)
    v = x.flip(2).contiguous()
    g.nvfp4_kv_append(cache, x, v, slots)
    _check(cache, before, x, v, slots)


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_slots_are_left_out_and_reported(fmt):
    cache = _cache(3, 16, 2, 64, fmt)
    before = cache.pool.cpu().numpy()
    k, v = _rows(5, 2, 64, seed=1)
    slots = torch.tensor([47, 48, -1, 1 << 40, 0], device=DEV)
    ws = torch.zeros(g.nvfp4_workspace_bytes(g.NVFP4_OP_KV_APPEND, 5, 2, 64), dtype=torch.uint8, device=DEV)
    g.nvfp4_kv_append(cache, k, v, slots, workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_ERR_DEVICE_INDEX, 41)
    inside = torch.tensor([47, -1, -1, -1, 0], device=DEV)
    _check(cache, before, k, v, inside)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)
    rk, rv = g.nvfp4_kv_read(cache, slots, workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_ERR_DEVICE_INDEX, 42)
    assert (rk[1:4] == 0).all() and (rv[1:4] == 0).all() and (rk[0] != 0).any()
    # without a workspace nothing is reported, and nothing is written either
    g.nvfp4_kv_append(cache, k, v, torch.full_like(slots, 1 << 50))
    _check(cache, before, k, v, inside)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_tokens_and_a_stream(fmt):
    """More rows than one round of the grid, on a stream of its own; read back into strided rows."""
    heads, d, ps, n = 8, 128, 32, 9001
    cache = _cache(n // ps + 1, ps, heads, d, fmt)
    k, v = _rows(n, heads, d, seed=4)
    slots = torch.arange(n, device=DEV).flip(0).contiguous()
    out = torch.zeros(n, 3 * heads * d, dtype=torch.bfloat16, device=DEV)
    rk = out[:, :heads * d].unflatten(1, (heads, d))
    rv = out[:, 2 * heads * d:].unflatten(1, (heads, d))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g.nvfp4_kv_append(cache, k, v, slots, stream=s)
    g.nvfp4_kv_read(cache, slots, out=(rk, rv), stream=s)
    s.synchronize()
    assert (out[:, heads * d:2 * heads * d] == 0).all()
    for t in (0, 1, 4567, 9000):
        for x, got in ((k, rk), (v, rv)):
            for h in (0, 7):
                c, sc, e = ref.encode_row(ref.to_np(x[t, h]), fmt)
                want = ref.decode_rows(c, sc, np.array(e), fmt)
                np.testing.assert_array_equal(ref.to_np(got[t, h]), want)
    # every row: a second trip through the cache changes nothing
    again = g.KVCache.empty(n // ps + 1, ps, heads, d, fmt, device=DEV)
    g.nvfp4_kv_append(again, rk, rv, slots)
    rk2, rv2 = g.nvfp4_kv_read(again, slots)
    if fmt == g.NVFP4_KV_E4M3:
        assert torch.equal(rk2, rk) and torch.equal(rv2, rv)
    else:  # a scale can move when its block's largest code was not 6; the values stay near
        assert ((rk2.double() - rk.double()).norm() <= 0.2 * rk.double().norm())


def test_no_tokens():
    cache = _cache(2, 16, 2, 64, g.NVFP4_KV_E4M3, fill=7)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    slots = torch.empty(0, dtype=torch.int64, device=DEV)
    g.nvfp4_kv_append(cache, none, none, slots)
    k, v = g.nvfp4_kv_read(cache, slots)
    assert k.shape == v.shape == (0, 2, 64) and (cache.pool == 7).all()
