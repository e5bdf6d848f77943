"""Attention over whole prompts (nvfp4_prompt_attention): V of any finite magnitude, and infinities in K."""
from __future__ import annotations

import math

import pytest
import torch

import gemm_nvfp4_gb300 as g
from helpers import BF16_REL, DEV
from test_gpu_prompt_attention import Prompts

pytestmark = pytest.mark.gpu

# magnitudes of V: up to 2^127 (the largest bf16 numbers but for the last rounding), and down to where the bound's absolute
# term, 2^-80, is as large as the rounding of the weights
MAGNITUDES = [2.0 ** e for e in (126, 121, 107, 0, -60, -72)]


def with_magnitude(p, size):
    """V rows of magnitudes in [1, 2) * size (their signs kept)."""
    m = 1 + p.v.float().abs() % 1
    p.v.copy_(torch.copysign(m.clamp(max=1.99), p.v.float()) * size)


def check(p, got, **kw):
    """Against include/nvfp4.h's bound with its absolute term."""
    want, tol = p.reference(**kw)
    assert torch.isfinite(want).all() and torch.isfinite(got).all()
    tol = tol + 2.0 ** -80 * (1 + p.v.double().abs().amax())
    tol = tol + (BF16_REL * (want.abs() + tol) if got.dtype == torch.bfloat16 else 2.0 ** -24 * want.abs())
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][0], want[bad][0], tol[bad][0])


@pytest.mark.parametrize("size", MAGNITUDES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_values_of_any_magnitude(size, d, causal):
    """One key (its own weight alone), and some hundred."""
    p = Prompts([1, 300, 2], 4, 2, d, seed=3)
    with_magnitude(p, size)
    for out_dtype in (torch.bfloat16, torch.float32):
        check(p, p.run(causal=causal, out_dtype=out_dtype), causal=causal)


@pytest.mark.parametrize("size", MAGNITUDES)
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_any_magnitude_under_equal_scores(size, d):
    """Thousands of equal weights on values of one sign: the largest sums there are before the division."""
    p = Prompts([5000], 2, 1, d, seed=4)
    with_magnitude(p, size)
    p.v.abs_()
    p.q.zero_()
    check(p, p.run(causal=False), causal=False)


@pytest.mark.parametrize("size", MAGNITUDES)
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_any_magnitude_under_a_lagging_reference(size, d):
    """Scores that rise after the first key tile by almost as much as the row's reference lets them: by 2^7.9."""
    p = Prompts([3000], 2, 1, d, seed=5)
    with_magnitude(p, size)
    p.v.abs_()
    p.q.zero_()
    p.q[..., 0] = 1.0
    p.k[..., 0] = 0.0
    p.k[128:, :, 0] = 7.9
    check(p, p.run(causal=False, scale=math.log(2)), causal=False, scale=math.log(2))


@pytest.mark.parametrize("bad", [math.inf, -math.inf])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 150), (False, 0)])
@pytest.mark.parametrize("scale", [0.125, -0.125])
@pytest.mark.parametrize("d", [64, 128])
def test_infinities_in_keys(bad, causal, window, scale, d):
    """A score of +infinity makes the row NaN, one of -infinity gives its key no weight, as the softmax has it: among keys
    that every row of a tile sees, and among masked ones."""
    n, at = 500, 20
    p = Prompts([n], 4, 2, d, seed=6)
    p.k[at, :, 3] = bad
    p.k[0, 1, 5] = bad  # (all that the first token sees)
    got = p.run(causal=causal, window=window, scale=scale).double()
    i = torch.arange(n, device=DEV)
    see = i <= i[:, None] if causal else torch.ones(n, n, dtype=torch.bool, device=DEV)
    if window:
        see = see & (i > i[:, None] - window)
    for h in range(4):
        q, k, v = p.q[:, h].double(), p.k[:, h // 2].double(), p.v[:, h // 2].double()
        z = (q @ k.T * scale).masked_fill(~see, -math.inf)
        assert not torch.isnan(z).any()
        w = torch.softmax(z, -1)  # (NaN beside +infinity, and of nothing but -infinity)
        lost = torch.isnan(w).any(-1)
        assert lost.any() and not lost.all()
        assert torch.isnan(got[lost, h]).all()
        size = abs(scale) * torch.where(see & torch.isfinite(z), q.abs() @ k.abs().T, 0.0).amax(-1, keepdim=True)
        want, tol = w @ v, (2.0 ** -8 + 2.0 ** -15 * size) * (w @ v.abs()) + 2.0 ** -80 * (1 + v.abs().amax())
        tol = tol + BF16_REL * (want.abs() + tol)
        assert ((got[:, h] - want).abs() <= tol)[~lost].all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("empty", [0, 30, 75])
def test_sequences_on_the_rows_of_earlier_ones(causal, empty):
    """Behind offsets that descend: a sequence that begins on an earlier one's rows is left out, also 32 sequences and more
    later, and those behind are computed."""
    p = Prompts([100, 50, 50], 4, 2, 64, seed=7)
    want = p.run(causal=causal)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = torch.full(p.q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    offsets = [0, 100, 50] + [50] * empty + [150, 200]
    p.run(causal=causal, offsets=torch.tensor(offsets, dtype=torch.int32, device=DEV), out=out, workspace=ws)
    assert g.nvfp4_device_status(ws) == (g.NVFP4_ERR_DEVICE_INDEX, 44)
    assert torch.equal(out[:100], want[:100]) and torch.equal(out[150:], want[150:])
    assert (out[100:150] == 7).all()
