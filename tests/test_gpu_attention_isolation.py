"""What nvfp4_paged_attention keeps away from a token: keys that it does not
see, whatever their slots hold, and keys of very different magnitudes beside
the ones it does see.  The bound is the one of include/nvfp4.h with nothing in
it but the keys that a token sees."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_nvfp4_gb300 as g
import kv_reference as ref
from helpers import DEV
from test_gpu_attention import FORMATS, Batch

pytestmark = pytest.mark.gpu

# (new tokens, query heads) over 2 KV heads: 8, 16, 24 rows (few-row kernel), 64 and 240 (both row-tile forms of the
# many-row kernel); fp32 outputs take the few-row kernel whatever the rows
SHAPES = [(2, 8), (4, 8), (6, 8), (16, 8), (60, 8)]


def run_and_check(b: Batch, skip=None, scale=None, **kw):
    """Every row, in both output types, against the definition.  `skip`: keys of each sequence; tokens that see one are
    left out."""
    group, scale = b.hq // b.hk, b.d ** -0.5 if scale is None else scale
    pool, tree, at, checked = b.cache.pool.cpu().numpy(), kw.get("tree"), 0, 0
    outs = [b.run(out_dtype=t, **kw) for t in (torch.bfloat16, torch.float32)]
    for i, (n, kv) in enumerate(zip(b.q_lens, b.kv_lens)):
        rows = slice(at, at + n)
        at += n
        k, v = ref.cache_rows(pool, b.slots(i, kv).numpy(), b.cache.page_size, b.d, b.cache.format)
        see = ref.visible(n, kv, kw.get("causal", True), kw.get("window", 0), None if tree is None else tree[rows].cpu().numpy())
        live = ~see[:, skip[i] if skip else []].any(1)
        see = see[live]
        out, weight, s = ref.attention(ref.to_np(b.q[rows])[live], k, v, see, scale)
        for got in outs:
            tol = ref.tolerance(out, weight, s, got.dtype)
            if got.dtype == torch.bfloat16:  # f16 weights lose n * 2^-28 * max |V| over the n keys seen
                for j in np.flatnonzero(see.any(1)):
                    tol[j] += see[j].sum() * 2.0 ** -28 * np.repeat(np.abs(v[see[j]]).max((0, 2)), group)[:, None]
            have = ref.to_np(got[rows])[live]
            assert not np.isnan(have).any(), f"{got.dtype}: {np.isnan(have).sum()} NaN of {have.size}"
            err = np.abs(have - out)
            assert (err <= tol).all(), (f"{got.dtype}: {(err > tol).sum()} of {err.size} out of bounds, "
                                        f"worst {(err / tol).max():.3g} of the bound")
        checked += live.sum()
    assert checked


def batch(fmt, q_len, hq, d, seed=0, kv_lens=(200, 77)):
    return Batch(fmt, [q_len] * len(kv_lens), [max(q_len + 1, n) for n in kv_lens], hq, 2, d, 16, seed=seed)


def idle_tree(q_len, idle, seqs):
    """Tree words in which a token descends from every live one before it, and none holds an idle place."""
    words, above = [], 0
    for i in range(q_len):
        if i not in idle:
            above |= 1 << i
        words.append(above - (1 << 64) if above >> 63 else above)
    return torch.tensor(words * seqs, device=DEV)


def fill_slots(b: Batch, seq, keys, what):
    """Puts bytes that no append writes into the slots of some keys."""
    ps, d, fmt = b.cache.page_size, b.d, b.cache.format
    cb, sb = (d, 0) if fmt == ref.E4M3 else (d // 2, d // 16)
    rng = np.random.default_rng(5)
    pool = b.cache.pool.cpu().numpy()
    for s in b.slots(seq, b.kv_lens[seq]).numpy()[list(keys)]:
        page, at = divmod(int(s), ps)
        for first, n, is_e in ((at * cb, cb, False), (ps * cb + at * sb, sb, False), (ps * (cb + sb) + at, 1, True)):
            value = {"NaN codes": 127 if is_e else 0xFF, "bytes of 255": 255, "largest codes": 254 if is_e else 0x7E,
                     "random": rng.integers(0, 256, (b.hk, 2, n))}[what]
            pool[page, :, :, first:first + n] = value
    b.cache.pool.copy_(torch.from_numpy(pool))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,hq", SHAPES)
@pytest.mark.parametrize("what", ["NaN codes", "bytes of 255", "largest codes", "random"])
@pytest.mark.parametrize("mode", ["tree", "causal", "window"])
def test_slots_never_written(fmt, q_len, hq, what, mode):
    """Idle draft places below kv_len (no slot, no tree bit), the slot of a token that others do not see, a slot that
    has left every window."""
    d = 128 if what != "bytes of 255" else 64
    b = batch(fmt, q_len, hq, d, seed=q_len, kv_lens=(200, 150))
    idle = sorted({1, q_len // 2, q_len - 1} - {0})
    keys = {"tree": [[kv - q_len + i for i in idle] for kv in b.kv_lens], "causal": [[kv - 1] for kv in b.kv_lens],
            "window": [[kv - q_len - 32, kv - 1] for kv in b.kv_lens]}[mode]
    for seq, bad in enumerate(keys):
        fill_slots(b, seq, bad, what)
    run_and_check(b, skip=keys, **{"tree": dict(tree=idle_tree(q_len, idle, 2)), "causal": {}, "window": dict(window=30)}[mode])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,hq", SHAPES)
@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("r", [24, 40, 80])
def test_loud_keys_that_are_not_seen(fmt, q_len, hq, which, r):
    """A few rows 2^r larger than the others, in their tile of keys, reach the tokens that see them alone."""
    d = 64 if r == 40 else 128
    idle = [1, q_len - 1]
    mode = {24: "tree", 40: "causal", 80: "window"}[r] if which != "both" else {24: "causal", 40: "window", 80: "tree"}[r]
    b = batch(fmt, q_len, hq, d, seed=r)
    gen = torch.Generator(DEV).manual_seed(r)
    for seq, kv in enumerate(b.kv_lens):
        k, v = (torch.randn(kv, 2, d, device=DEV, generator=gen) for _ in range(2))
        loud = {"tree": [kv - q_len + i for i in idle], "causal": [kv - 1], "window": [max(0, kv - q_len - 25)]}[mode]
        for x, name in ((k, "k"), (v, "v")):
            if which in (name, "both"):
                x[loud] *= 2.0 ** r
        b.put(seq, k.to(torch.bfloat16), v.to(torch.bfloat16))
    run_and_check(b, **{"tree": dict(tree=idle_tree(q_len, idle, 2)), "causal": {}, "window": dict(window=24)}[mode])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,hq", SHAPES)
@pytest.mark.parametrize("r", [13, 15, 25, 60])
@pytest.mark.parametrize("small_k", [False, True])
def test_keys_far_apart_that_are_seen(fmt, q_len, hq, r, small_k):
    """Few keys, every third with a V 2^r smaller than its neighbours' and, with small_k, a K as much smaller."""
    d, kv = 128, q_len + 12
    b = batch(fmt, q_len, hq, d, seed=r, kv_lens=(kv, kv + 130))
    gen = torch.Generator(DEV).manual_seed(r)
    for seq, n in enumerate(b.kv_lens):
        k, v = (torch.randn(n, 2, d, device=DEV, generator=gen) for _ in range(2))
        small = torch.arange(n, device=DEV) % 3 == 0
        v[~small] *= 2.0 ** r
        if small_k:
            k[small] *= 2.0 ** -r
        b.put(seq, k.to(torch.bfloat16), v.to(torch.bfloat16))
    run_and_check(b, **(dict(causal=False) if r == 15 else dict(window=9) if r == 60 else {}))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,hq", [(16, 8), (60, 8)])
def test_calls_with_far_rows_leave_a_clean_workspace(fmt, q_len, hq):
    """One workspace for calls whose rows lie far apart and for ordinary ones, in turn: the same results each time."""
    loud, calm = batch(fmt, q_len, hq, 128, seed=1), batch(fmt, q_len, hq, 128, seed=2)
    k, v = (torch.randn(200, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(s)) for s in (3, 4))
    v[-1] *= 2.0 ** 40
    loud.put(0, k.to(torch.bfloat16), v.to(torch.bfloat16))
    ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(loud.cache, loud.q, 2, q_len), dtype=torch.uint8, device=DEV)
    first = [b.run(workspace=ws) for b in (loud, calm)]
    for _ in range(3):
        for b, want in zip((loud, calm), first):
            assert torch.equal(b.run(workspace=ws), want)
            assert (ws[:256] == 0).all()
    assert torch.equal(calm.run(), first[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,hq", SHAPES)
@pytest.mark.parametrize("apart", ["interleaved", "blocks"])
@pytest.mark.parametrize("low,high,weak", [(-90, 97, 40), (-60, 60, 20), (0, 97, 30)])
def test_sums_over_values_far_apart(fmt, q_len, hq, apart, low, high, weak):
    """Keys with nearly all of the softmax and a tiny V beside keys of 2^-weak of it and a huge V: the sum of the
    weights is that of the former, whatever the V rows' magnitudes."""
    d = 128
    b = batch(fmt, q_len, hq, d, seed=1, kv_lens=(700, 300))
    gen = torch.Generator(DEV).manual_seed(2)
    # one channel of q and K decides: q . k * scale * log2(e) is 0 for the strong keys, -weak for the others
    b.q.copy_(0.01 * torch.randn(b.q.shape, device=DEV, generator=gen))
    b.q[:, :, 0] = 8.0
    for seq, n in enumerate(b.kv_lens):
        k, v = (torch.randn(n, 2, d, device=DEV, generator=gen) for _ in range(2))
        k *= 0.01
        at = torch.arange(n, device=DEV)
        strong = at % 5 != 2 if apart == "interleaved" else at < n - q_len - 140
        k[:, :, 0] = torch.where(strong, 0.0, -weak / 1.4427 / 8.0 / d ** -0.5)[:, None]
        v *= torch.where(strong, 2.0 ** low, 2.0 ** high)[:, None, None]
        b.put(seq, k.to(torch.bfloat16), v.to(torch.bfloat16))
    run_and_check(b)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,hq", [(16, 8), (60, 8)])
def test_captured_calls_with_far_rows(fmt, q_len, hq):
    """One captured call, replayed over a cache whose rows lie far apart in some replays and not in others."""
    b = batch(fmt, q_len, hq, 128, seed=5)
    k, v = (torch.randn(200, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(s)).to(torch.bfloat16) for s in (6, 7))
    loud = v.clone()
    loud[-1] *= 2.0 ** 40
    out = torch.empty_like(b.q)
    ws = torch.zeros(g.nvfp4_paged_attention_workspace_bytes(b.cache, b.q, 2, q_len), dtype=torch.uint8, device=DEV)
    b.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(out=out, workspace=ws)
        b.run(out=out, workspace=ws)
    for values in (v, loud, loud, v):
        b.put(0, k, values)
        want = b.run()
        graph.replay()
        assert torch.equal(out, want)
        assert (ws[:256] == 0).all()
