"""Attention over whole prompts (nvfp4_prompt_attention) against softmax(q K^T) V in fp64."""
from __future__ import annotations

import math

import pytest
import torch

import gemm_nvfp4_gb300 as g
from helpers import BF16_REL, DEV

pytestmark = pytest.mark.gpu


class Prompts:
    """Packed q, k and v (column ranges of one product's output) of sequences of the given lengths."""

    def __init__(self, lens, hq, hk, d, behind=0, seed=0, spread=1.0):
        gen = torch.Generator(DEV).manual_seed(seed)
        self.lens, self.hq, self.hk, self.d = list(lens), hq, hk, d
        rows = sum(lens) + behind
        x = torch.randn(rows, (hq + 2 * hk) * d, device=DEV, generator=gen)
        x[:, :hq * d] *= spread
        self.qkv = x.to(torch.bfloat16)
        self.q, self.k, self.v = (t.unflatten(1, (-1, d)) for t in self.qkv.split((hq * d, hk * d, hk * d), 1))
        self.offsets = torch.tensor([0] + self.lens, device=DEV).cumsum(0).int()

    def run(self, **kw):
        kw.setdefault("offsets", self.offsets)
        return g.nvfp4_prompt_attention(self.q, self.k, self.v, **kw)

    def reference(self, causal=True, window=0, scale=None):
        """(out, bound of include/nvfp4.h without the output's rounding), by sequence and head; rows in no sequence NaN."""
        scale = self.d ** -0.5 if scale is None else scale
        out = torch.full(self.q.shape, math.nan, dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(out)
        group, begin = self.hq // self.hk, 0
        for n in self.lens:
            i = torch.arange(n, device=DEV)
            see = torch.ones(n, n, dtype=torch.bool, device=DEV)
            if causal:
                see = i <= i[:, None]
                if window:
                    see &= i > i[:, None] - window
            for h in range(self.hq if n else 0):
                q, k, v = (t[begin:begin + n, j].double() for t, j in ((self.q, h), (self.k, h // group), (self.v, h // group)))
                z = (q @ k.T * scale).masked_fill(~see, -math.inf)
                size = (abs(scale) * (q.abs() @ k.abs().T)).masked_fill(~see, 0).nan_to_num().amax(-1, keepdim=True)
                p = torch.softmax(z, -1)
                p, v = torch.where(see, p, 0.0), v
                # a value that no row sees must not meet its zero weight
                clean = torch.where(torch.isfinite(v), v, 0.0)
                o, t = p @ clean, (2.0 ** -8 + 2.0 ** -15 * size) * (p @ clean.abs())
                for j in torch.nonzero(~torch.isfinite(v).all(-1)).flatten().tolist():
                    o = torch.where(see[:, j, None] & ~torch.isfinite(v[j]), math.nan, o)
                out[begin:begin + n, h], tol[begin:begin + n, h] = o, t
            begin += n
        return out, tol

    def check(self, got, **kw):
        want, tol = self.reference(**kw)
        n = sum(self.lens)
        got, want, tol = got[:n].double(), want[:n], tol[:n]
        if kw.get("out_dtype") != torch.float32:
            tol = tol + BF16_REL * (want.abs() + tol)
        finite = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got), finite)
        bad = ~((got - want).abs() <= tol) & finite
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first {torch.nonzero(bad)[0].tolist()}: " \
                              f"{got[bad][0]} for {want[bad][0]}, tolerance {tol[bad][0]}"


@pytest.mark.parametrize("hq,hk,d", [(32, 8, 128), (40, 8, 128), (4, 4, 64), (14, 2, 64), (8, 1, 128), (12, 4, 64), (3, 1, 128),
                                     (128, 1, 64), (96, 1, 128), (33, 3, 64)])
@pytest.mark.parametrize("lens", [[1], [77], [0, 3, 0, 1, 64, 129, 0], [300, 1, 257]])
def test_heads_and_lengths(hq, hk, d, lens):
    p = Prompts(lens, hq, hk, d, seed=len(lens) + hq)
    p.check(p.run())


@pytest.mark.parametrize("n", [2, 15, 16, 31, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 511, 640, 1025])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_around_tiles(n, d):
    p = Prompts([n, 5], 4, 2, d, seed=n)
    for causal in (True, False):
        p.check(p.run(causal=causal), causal=causal)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 128, 129, 500, 5000, 1 << 40])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (4, 4, 128), (16, 1, 128)])
def test_windows(window, hq, hk, d):
    p = Prompts([700, 1, 130], hq, hk, d, seed=window % 1000)
    p.check(p.run(window=window), window=window)


@pytest.mark.parametrize("causal", [True, False])
def test_one_sequence_without_offsets_and_fp32_output(causal):
    p = Prompts([333], 8, 2, 128)
    out = p.run(offsets=None, causal=causal, out_dtype=torch.float32)
    assert out.dtype == torch.float32
    want, tol = p.reference(causal)
    assert ((out.double() - want).abs() <= tol + 2.0 ** -24 * want.abs()).all()
    assert torch.equal(out.to(torch.bfloat16), p.run(offsets=None, causal=causal))


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 0.02])
def test_scales(scale):
    """Peaked and flat softmaxes, and scores whose order the scale turns round."""
    p = Prompts([200], 4, 1, 64, spread=2.0)
    p.check(p.run(scale=scale), scale=scale)


def test_scores_that_rise_along_the_keys():
    """The running maximum moves at every key: by small steps, and by steps far beyond fp32's range of weights."""
    for slope in (0.01, 1.0, 40.0):
        p = Prompts([600], 2, 1, 128, seed=3)
        p.k.mul_(0.01)
        p.q[:, :, 0] = 1.0
        p.k[:, :, 0] = (torch.arange(600, device=DEV) * slope).to(torch.bfloat16)[:, None]
        for sign in (1.0, -1.0):
            p.check(p.run(scale=sign * 0.3), scale=sign * 0.3)


def test_rows_behind_and_between_are_left_alone():
    """Rows behind the last sequence and before the first keep what they held."""
    p = Prompts([40, 0, 90], 4, 2, 64, behind=70)
    out = torch.full(p.q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    p.run(out=out)
    p.check(out)
    assert (out[130:] == 7).all()
    out.fill_(7.0)
    p.run(out=out, offsets=torch.tensor([30, 90], dtype=torch.int32, device=DEV))
    assert (out[:30] == 7).all() and (out[90:] == 7).all() and (out[30:90] != 7).any()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 0)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (2, 2, 64)])
def test_unseen_rows_do_not_leak(bad, causal, window, hq, hk, d):
    """NaN and infinities in V of a token reach the tokens that see it and no other: not the ones before it, nor those
    whose window has passed it, nor another sequence, nor from behind the last one."""
    p = Prompts([150, 333, 1, 64], hq, hk, d, behind=9, seed=1)
    p.v[150 + 140, 0, 5] = bad
    p.v[150 + 332, 1, 0] = bad
    p.v[149, 0, 1] = bad
    p.v[483] = bad  # the sequence of one token
    p.v[548:] = bad
    p.k[548:] = bad
    p.q[548:] = bad
    got = p.run(causal=causal, window=window)
    p.check(got, causal=causal, window=window)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (False, 0)])
def test_bad_keys_and_queries(causal, window):
    """A NaN in K reaches the rows that see its key, a NaN in q its own row."""
    p = Prompts([200, 100], 4, 2, 64, seed=2)
    clean = p.run(causal=causal, window=window)
    p.k[90, 1, 3] = math.nan
    p.q[250, 2, 0] = math.inf
    got = p.run(causal=causal, window=window)
    i = torch.arange(300, device=DEV)
    seen = (i < 200) if not causal else (i >= 90) & (i < (110 if window else 200))
    dirty = torch.zeros(300, 4, dtype=torch.bool, device=DEV)
    dirty[:, 2:] = seen[:, None]
    dirty[250, 2] = True
    assert torch.isnan(got[dirty]).all()
    assert torch.equal(got[~dirty], clean[~dirty])


def test_a_token_does_not_depend_on_its_neighbours():
    """The same sequence alone, and packed between others: the same bits."""
    p = Prompts([70, 261, 33], 8, 2, 128, seed=4)
    packed = p.run()
    for b, n in enumerate(p.lens):
        at = slice(int(p.offsets[b]), int(p.offsets[b + 1]))
        alone = g.nvfp4_prompt_attention(p.q[at], p.k[at], p.v[at])
        assert torch.equal(packed[at], alone)


@pytest.mark.parametrize("hq,hk,d,causal", [(8, 1, 128, True), (4, 4, 64, False)])
def test_repeated_calls_give_the_same_bits(hq, hk, d, causal):
    p = Prompts([3000, 40, 1500], hq, hk, d, seed=6)
    want = p.run(causal=causal)
    for _ in range(20):
        assert torch.equal(p.run(causal=causal), want)


def test_offsets_out_of_bounds():
    """Offsets that descend or pass the end: code 44, nothing outside is touched, the others are computed."""
    p = Prompts([100, 60, 40], 4, 2, 64)
    want = p.run()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    for bad in ([0, 100, 160, 999], [0, 100, 160, -5], [0, 100, 160, 130], [-7, 100, 160, 200]):
        out = torch.full(p.q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
        p.run(offsets=torch.tensor(bad, dtype=torch.int32, device=DEV), out=out, workspace=ws)
        assert g.nvfp4_device_status(ws) == (g.NVFP4_ERR_DEVICE_INDEX, 44), bad
        assert torch.equal(out[100:160], want[100:160]), bad
    p.run(workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)


@pytest.mark.parametrize("n_seqs", [1000, 9000])
def test_many_sequences(n_seqs):
    gen = torch.Generator().manual_seed(n_seqs)
    lens = torch.randint(0, 6, (n_seqs,), generator=gen).tolist()
    lens[n_seqs // 2] = 300
    p = Prompts(lens, 2, 1, 64)
    got = p.run()
    # every sequence at once in fp64: tokens of other sequences masked
    n = sum(lens)
    seq = torch.repeat_interleave(torch.arange(n_seqs), torch.tensor(lens)).to(DEV)
    i = torch.arange(n, device=DEV)
    for lo in range(0, n, 2048):
        hi = min(n, lo + 2048)
        a = max(0, lo - 300)
        see = (seq[a:hi] == seq[lo:hi, None]) & (i[a:hi] <= i[lo:hi, None])
        for h in range(2):
            z = p.q[lo:hi, h].double() @ p.k[a:hi, 0].double().T * 0.125
            size = 0.125 * (p.q[lo:hi, h].double().abs() @ p.k[a:hi, 0].double().abs().T).masked_fill(~see, 0).amax(-1, keepdim=True)
            w = torch.softmax(z.masked_fill(~see, -math.inf), -1)
            want, tol = w @ p.v[a:hi, 0].double(), (2.0 ** -8 + 2.0 ** -15 * size) * (w @ p.v[a:hi, 0].double().abs())
            assert ((got[lo:hi, h].double() - want).abs() <= tol + BF16_REL * (want.abs() + tol)).all()


@pytest.mark.parametrize("n_seqs,at,hq,causal", [(65535, 65534, 128, True), (65535, 40000, 2, False), (40, 0, 8, True), (70, 69, 4, False)])
def test_one_long_sequence_among_many(n_seqs, at, hq, causal):
    """Chunks of sequences without a token, and one with many places in the order of the work."""
    n = 700
    p = Prompts([n], hq, 1, 64, seed=n_seqs)
    offsets = torch.zeros(n_seqs + 1, dtype=torch.int32, device=DEV)
    offsets[at + 1:] = n
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    got = p.run(offsets=offsets, causal=causal, workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)
    p.check(got, causal=causal)
    assert torch.equal(got, p.run(causal=causal))


def test_strides_and_output_views():
    """q, k, v and out in buffers of their own strides."""
    p = Prompts([130, 7], 4, 2, 64)
    want = p.run()
    wide = torch.full((137, 4 * 64 + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    out = wide[:, 8:8 + 256].unflatten(1, (4, 64))
    got = g.nvfp4_prompt_attention(p.q.contiguous(), p.k.contiguous(), p.v.contiguous(), offsets=p.offsets, out=out)
    assert got is out and torch.equal(out, want)
    assert (wide[:, :8] == 7).all() and (wide[:, 264:] == 7).all()


def test_captured_and_replayed_with_other_lengths():
    p = Prompts([100, 200, 50], 8, 2, 128)
    out = torch.empty_like(p.q.contiguous())
    p.run(out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(out=out)
    for lens in ([350, 0, 0], [1, 1, 348], [10, 330, 10]):
        p.lens = lens
        p.offsets.copy_(torch.tensor([0] + lens).cumsum(0))
        graph.replay()
        p.check(out)


def test_two_streams_share_a_status_word():
    a, b = Prompts([700, 90], 8, 2, 128, seed=1), Prompts([30, 900], 4, 4, 64, seed=2)
    want = a.run(), b.run()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for x in (s, t):
        x.wait_stream(torch.cuda.current_stream())
    got = [(a.run(stream=s, workspace=ws), b.run(stream=t, workspace=ws)) for _ in range(4)]
    for x in (s, t):
        torch.cuda.current_stream().wait_stream(x)
    assert all(torch.equal(x, want[0]) and torch.equal(y, want[1]) for x, y in got)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_OK, 0)


def test_nothing_to_do():
    p = Prompts([0, 0], 4, 2, 64)
    assert p.run().shape == (0, 4, 64)
    p = Prompts([0, 0], 4, 2, 64, behind=5)
    out = torch.full(p.q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    assert (p.run(out=out) == 7).all()
    assert (p.run(out=out, offsets=torch.zeros(1, dtype=torch.int32, device=DEV)) == 7).all()


@pytest.mark.slow
def test_a_long_prompt():
    """Last rows of 16384 tokens, 40 and 8 heads, against fp64."""
    p = Prompts([16384], 40, 8, 128, seed=5)
    got = p.run(offsets=None)
    rows = torch.tensor([0, 1, 4095, 8191, 12345, 16383], device=DEV)
    for h in (0, 7, 39):
        q, k, v = p.q[rows, h].double(), p.k[:, h // 5].double(), p.v[:, h // 5].double()
        see = torch.arange(16384, device=DEV) <= rows[:, None]
        w = torch.softmax((q @ k.T * 128 ** -0.5).masked_fill(~see, -math.inf), -1)
        size = 128 ** -0.5 * (q.abs() @ k.abs().T).amax(-1, keepdim=True)
        want, tol = w @ v, (2.0 ** -8 + 2.0 ** -15 * size) * (w @ v.abs())
        assert ((got[rows, h].double() - want).abs() <= tol + BF16_REL * (want.abs() + tol)).all()
