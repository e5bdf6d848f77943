"""Rotary positions (nvfp4_rope) against their definition in fp64."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import gemm_nvfp4_gb300 as g
from helpers import BF16_REL, DEV, assert_close, to_np

pytestmark = pytest.mark.gpu

# Of scale * (|x| + |y|): angle 2 pi 2^-27, sine and cosine two ulps, and four fp32 roundings of products and sums
TURN_REL = 2 * math.pi * 2.0 ** -27 + 2.0 ** -23 + 4 * 2.0 ** -24


def frequencies(pairs, base=1e6):
    return [base ** (-i / max(pairs, 1)) for i in range(pairs)]


def reference(x, angle, pairs, adjacent, inverse, scale):
    """(y, tolerance) of fp64 rows x [tokens, heads, D] turned by angle [tokens, pairs]."""
    y, tol = x.copy(), np.zeros_like(x)
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + pairs)
        c, s = np.cos(angle[:, i, None]), np.sin(angle[:, i, None]) * (-1 if inverse else 1)
        y[..., a] = scale * (x[..., a] * c - x[..., b] * s)
        y[..., b] = scale * (x[..., a] * s + x[..., b] * c)
        tol[..., a] = tol[..., b] = abs(scale) * TURN_REL * (abs(x[..., a]) + abs(x[..., b]))
    return y, tol


def angles(table, positions, axis):
    """Angles of the table's frequencies at integer positions [axes][tokens], reduced in integers."""
    turns = table.pairs.cpu().view(torch.int64)[:, 0].tolist()
    out = np.empty((len(positions[0]), len(turns)))
    for i, t in enumerate(turns):
        for n, p in enumerate(positions[axis[i]]):
            f = p * t % 2 ** 64
            out[n, i] = 2 * math.pi * ((f - 2 ** 64 if f >= 2 ** 63 else f) / 2.0 ** 64)
    return out


def rows(tokens, heads, d, dtype, seed, pad=0):
    gen = torch.Generator().manual_seed(seed)
    x = (3 * torch.randn(tokens, heads * d + pad, generator=gen)).to(dtype).to(DEV)
    return x[:, :heads * d].unflatten(1, (heads, d))


def check(got, x, angle, pairs, adjacent=False, inverse=False, scale=1.0):
    ref, tol = reference(to_np(x), angle, pairs, adjacent, inverse, scale)
    if got.dtype == torch.bfloat16:
        tol = tol + BF16_REL * (np.abs(ref) + tol)
        tol[..., 2 * pairs:] = 0
    assert_close(to_np(got), ref, tol)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,d,rotary,axes", [
    (1, 32, 8, 128, 128, 1), (7, 40, 8, 128, 128, 3), (33, 16, 16, 64, 32, 2), (5, 3, 1, 80, 80, 2), (130, 2, 2, 96, 48, 3),
    (3, 5, 1, 24, 10, 1), (2, 1, 1, 512, 512, 4), (4, 7, 7, 8, 2, 1), (3, 4, 2, 64, 0, 1), (9, 65, 1, 72, 40, 2),
    (1000, 8, 2, 128, 64, 2)])
def test_turns(dtype, adjacent, tokens, hq, hk, d, rotary, axes):
    pairs = rotary // 2
    axis = [i * axes // max(pairs, 1) for i in range(pairs)]
    table = g.RopeTable.make(frequencies(pairs), axis)
    gen = torch.Generator().manual_seed(1)
    positions = torch.randint(0, 200000, (axes, tokens), generator=gen)
    q, k = rows(tokens, hq, d, dtype, 2, pad=8), rows(tokens, hk, d, dtype, 3, pad=16)
    before = q.clone()
    got_q, got_k = g.nvfp4_rope(q, k, positions.to(DEV) if axes > 1 else positions[0].to(DEV), table, adjacent=adjacent)
    angle = angles(table, positions.tolist(), axis)
    check(got_q, q, angle, pairs, adjacent)
    check(got_k, k, angle, pairs, adjacent)
    assert torch.equal(q, before)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,rotary", [(3000, 5, 2, 10), (12000, 2, 1, 20), (2500, 0, 7, 6)])
def test_odd_pairs_of_many_tokens(tokens, hq, hk, rotary, adjacent):
    """Numbers of pairs that are no multiple of 8, several heads to a warp (one of q and one of k among them)."""
    pairs = rotary // 2
    table = g.RopeTable.make(frequencies(pairs))
    positions = torch.arange(tokens)
    q, k = rows(tokens, hq, 24, torch.bfloat16, 2), rows(tokens, hk, 24, torch.bfloat16, 3)
    got_q, got_k = g.nvfp4_rope(q, k, positions.to(DEV), table, adjacent=adjacent)
    angle = angles(table, [positions.tolist()], [0] * pairs)
    check(got_q, q, angle, pairs, adjacent)
    check(got_k, k, angle, pairs, adjacent)
    g.nvfp4_rope(q, k, positions.to(DEV), table, adjacent=adjacent, out=(q, k))
    assert torch.equal(q, got_q) and torch.equal(k, got_k)


def test_far_and_negative_positions():
    """Where fp32 angles would be off by many turns."""
    freq = [1.0, 0.37, 1e-3, -0.8, 2.0 ** 20 + 0.3, 1e-9, 0.0, math.pi]
    table = g.RopeTable.make(freq)
    positions = [0, 1, -1, 2 ** 20 + 1, 2 ** 31, 2 ** 40 - 1, -2 ** 40 + 7, 123456789, 2 ** 52 + 1]
    q = rows(len(positions), 2, 16, torch.float32, 4)
    got, none = g.nvfp4_rope(q, None, torch.tensor(positions, device=DEV), table)
    assert none is None
    check(got, q, angles(table, [positions], [0] * 8), 8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rotary", [(128, 128), (64, 32), (24, 10)])
def test_in_place_inverse_and_scale(dtype, d, rotary):
    pairs = rotary // 2
    table = g.RopeTable.make(frequencies(pairs))
    positions = torch.arange(50, 69, device=DEV)
    angle = angles(table, [positions.tolist()], [0] * pairs)
    q, k = rows(19, 6, d, dtype, 5, pad=8), rows(19, 2, d, dtype, 6)
    q0, k0 = q.clone(), k.clone()
    want = g.nvfp4_rope(q, k, positions, table, scale=1.25)
    check(want[0], q0, angle, pairs, scale=1.25)
    out = g.nvfp4_rope(q, k, positions, table, scale=1.25, out=(q, k))
    assert out[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    back = g.nvfp4_rope(q0, k0, positions, table, inverse=True)
    check(back[0], q0, angle, pairs, inverse=True)
    check(back[1], k0, angle, pairs, inverse=True)


def test_inverse_is_the_transpose():
    """<dy, R x> = <R^T dy, x>, which makes the inverse the gradient's pass: also by differences."""
    table = g.RopeTable.make(frequencies(32), [i % 3 for i in range(32)])
    positions = torch.randint(0, 9999, (3, 11), device=DEV)
    x, dy = rows(11, 4, 64, torch.float32, 7), rows(11, 4, 64, torch.float32, 8)
    turn = lambda t, **kw: g.nvfp4_rope(t, None, positions, table, scale=0.75, **kw)[0].double()
    a, b = (dy.double() * turn(x)).sum(), (turn(dy, inverse=True) * x.double()).sum()
    bound = 2 * 0.75 * TURN_REL * 2 * float((dy.abs().double() * x.abs().amax()).sum())
    assert abs(float(a - b)) <= bound
    step = torch.zeros_like(x)
    step[3, 2, 17] = 0.5  # the map is linear: a difference of any width is its derivative
    diff = float((dy.double() * (turn(x + step) - turn(x - step))).sum())
    assert abs(diff - float(turn(dy, inverse=True)[3, 2, 17])) <= 4 * TURN_REL * float(dy[3].abs().sum() * (x[3].abs().amax() + 1))


def test_nan_stays_in_its_pair():
    table = g.RopeTable.make(frequencies(32))
    q = rows(3, 2, 64, torch.bfloat16, 9)
    clean = g.nvfp4_rope(q, None, torch.arange(3, device=DEV), table)[0]
    q[1, 1, 5] = math.nan
    got = g.nvfp4_rope(q, None, torch.arange(3, device=DEV), table)[0]
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[1, 1, [5, 37]] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])


def test_captured_replayed_and_on_another_stream():
    table = g.RopeTable.make(frequencies(64))
    q, k = rows(5, 8, 128, torch.bfloat16, 10), rows(5, 2, 128, torch.bfloat16, 11)
    positions = torch.arange(5, device=DEV)
    out = (torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous()))
    call = lambda **kw: g.nvfp4_rope(q, k, positions, table, **kw)
    call(out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out)
    positions.add_(1000)
    graph.replay()
    want = call()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_tokens():
    table = g.RopeTable.make(frequencies(64))
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=DEV)
    out, _ = g.nvfp4_rope(q, None, torch.empty(0, dtype=torch.int64, device=DEV), table)
    assert out.shape == q.shape


def test_many_axes():
    """More axes than a warp has lanes."""
    axis = [3, 40, 31, 32, 0, 63, 7, 62]
    table = g.RopeTable.make(frequencies(8), axis)
    positions = torch.randint(-5000, 5000, (64, 5))
    for pairs_first in (16, 24):  # both kernels' heads: 8 pairs of 16 elements, and with elements that are not turned
        q = rows(5, 3, pairs_first, torch.float32, 12)
        got = g.nvfp4_rope(q, None, positions.to(DEV), table)[0]
        check(got, q, angles(table, positions.tolist(), axis), 8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,d,rotary", [
    (8192, 40, 8, 128, 128), (20001, 5, 3, 128, 128), (10001, 11, 4, 96, 48), (10002, 20, 3, 80, 32), (9733, 0, 9, 512, 512),
    (9999, 70, 1, 24, 16)])
def test_many_tokens(dtype, adjacent, tokens, hq, hk, d, rotary):
    """Several heads to a lane (of q and of k in one warp), elements that are not turned in several rounds, and a last block
    that is not full: some tokens against the definition, all of them against calls of few tokens, and in place."""
    pairs = rotary // 2
    axis = [i % 3 for i in range(pairs)]
    table = g.RopeTable.make(frequencies(pairs), axis)
    positions = torch.randint(0, 200000, (3, tokens), generator=torch.Generator().manual_seed(1))
    at = positions.to(DEV)
    q, k = rows(tokens, hq, d, dtype, 2, pad=8), rows(tokens, hk, d, dtype, 3, pad=16)
    got = g.nvfp4_rope(q, k, at, table, adjacent=adjacent)
    some = list(range(0, tokens, 997)) + [tokens - 2, tokens - 1]
    angle = angles(table, positions[:, some].tolist(), axis)
    check(got[0][some], q[some], angle, pairs, adjacent)
    check(got[1][some], k[some], angle, pairs, adjacent)
    for lo in range(0, tokens, 700):
        part = slice(lo, min(lo + 700, tokens))
        few = g.nvfp4_rope(q[part], k[part], at[:, part], table, adjacent=adjacent)
        assert torch.equal(got[0][part], few[0]) and torch.equal(got[1][part], few[1])
    g.nvfp4_rope(q, k, at, table, adjacent=adjacent, out=(q, k))
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])


@pytest.mark.parametrize("dtype,d,pairs", [(torch.bfloat16, 64, 32), (torch.float32, 40, 10)])
def test_one_row_of_positions_for_every_axis(dtype, d, pairs):
    """Text in a model with several axes: positions.expand(axes, tokens), whose rows are one row."""
    table = g.RopeTable.make(frequencies(pairs), [i % 40 for i in range(pairs)])
    for tokens in (1, 33):
        at = torch.arange(7000, 7000 + tokens, device=DEV)
        q, k = rows(tokens, 4, d, dtype, 2), rows(tokens, 2, d, dtype, 3)
        want = g.nvfp4_rope(q, k, at.repeat(40, 1), table)
        got = g.nvfp4_rope(q, k, at.expand(40, tokens), table)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        check(got[0], q, angles(table, at.repeat(40, 1).tolist(), [i % 40 for i in range(pairs)]), pairs)


def test_one_token_in_place_through_views_of_other_strides():
    """The stride of a single row is not looked at: in place through another view of it."""
    table = g.RopeTable.make(frequencies(32))
    x = rows(1, 2, 64, torch.bfloat16, 4, pad=8)
    want = g.nvfp4_rope(x, None, torch.tensor([9], device=DEV), table)[0]
    g.nvfp4_rope(x, None, torch.tensor([9], device=DEV), table, out=(x.as_strided((1, 2, 64), (128, 64, 1)), None))
    assert torch.equal(x, want)
