"""The quantised KV cache and the attention over it from their definitions
(include/nvfp4.h), in fp64 numpy, one sequence, token and head at a time."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3, NVFP4 = 0, 1
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def e4m3_table() -> np.ndarray:
    """Value of every E4M3 byte."""
    out = np.empty(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = (math.nan if (b & 127) == 127 else mag) * (-1 if b & 128 else 1)
    return out


E4M3_VALUES = e4m3_table()


def nearest_code(x: np.ndarray, values: np.ndarray) -> np.ndarray:
    """Codes 0.. of the nearest of ascending `values` to x >= 0; ties to the even code."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    down, up = x - values[lo], values[hi] - x
    return np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))


def row_bytes(fmt: int, d: int) -> int:
    return d + 1 if fmt == E4M3 else d // 2 + d // 16 + 1


def encode_row(x: np.ndarray, fmt: int):
    """(codes, scales, e) bytes of one row of fp64 values that are bf16 numbers."""
    d = len(x)
    cb, sb = (d, 0) if fmt == E4M3 else (d // 2, d // 16)
    top = 448.0 if fmt == E4M3 else 2688.0
    nan_row = np.zeros(cb, np.uint8), np.zeros(sb, np.uint8), 255
    if not np.isfinite(x).all():
        return nan_row
    amax = np.abs(x).max()
    k = -100
    while amax > top * 2.0 ** k:
        k += 1
    if k > 100:
        return nan_row
    y = x * 2.0 ** -k
    sign = np.signbit(x).astype(np.uint8)
    if fmt == E4M3:
        return nearest_code(np.abs(y), E4M3_VALUES[:127]).astype(np.uint8) | sign << 7, np.zeros(0, np.uint8), k + 127
    codes, scales = np.zeros(d, np.uint8), np.zeros(sb, np.uint8)
    for b in range(sb):
        part = slice(16 * b, 16 * b + 16)
        scales[b] = nearest_code(np.array([np.abs(y[part]).max() / 6]), E4M3_VALUES[:127])[0]
        if scales[b]:
            s = E4M3_VALUES[scales[b]]
            codes[part] = nearest_code(np.abs(y[part]) / s, E2M1) | sign[part] << 3
    return codes[0::2] | codes[1::2] << 4, scales, k + 127


def decode_rows(codes: np.ndarray, scales: np.ndarray, e: np.ndarray, fmt: int) -> np.ndarray:
    """Values of rows [..., bytes]; e [...]."""
    if fmt == E4M3:
        x = E4M3_VALUES[codes]
    else:
        signed = np.concatenate((E2M1, -E2M1))
        x = np.stack((signed[codes & 15], signed[codes >> 4]), -1)
        x = x.reshape(*codes.shape[:-1], 2 * codes.shape[-1])
        x = x * np.repeat(E4M3_VALUES[scales], 16, -1)
    x = x * 2.0 ** (e.astype(np.float64) - 127)[..., None]
    return np.where((e == 255)[..., None], math.nan, x)


def planes(pool: np.ndarray, page_size: int, d: int, fmt: int):
    """Views of pool[page, head, K or V, block]: codes, scales, e, each [page, head, K or V, page_size, ...]."""
    cb, sb = (d, 0) if fmt == E4M3 else (d // 2, d // 16)
    lead = pool.shape[:-1]
    a, b = page_size * cb, page_size * (cb + sb)
    return (pool[..., :a].reshape(*lead, page_size, cb), pool[..., a:b].reshape(*lead, page_size, sb), pool[..., b:])


def cache_rows(pool: np.ndarray, slots: np.ndarray, page_size: int, d: int, fmt: int):
    """K and V values [slots, heads, d] of non-negative slots."""
    codes, scales, e = planes(pool, page_size, d, fmt)
    page, at = slots // page_size, slots % page_size
    x = decode_rows(codes[page, :, :, at], scales[page, :, :, at], e[page, :, :, at], fmt)
    return x[:, :, 0], x[:, :, 1]


def attention(q, k, v, see, scale):
    """out, and the two sums of its error bound: q [n, hq, d]; k, v [keys, hk, d]; see [n, keys] bool.
    Returns out, sum_j softmax_j |v_j| (both [n, hq, d]) and S = max_j |scale| sum_d |q_d k_jd| ([n, hq, 1])."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    out, weight, s = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq, 1))
    for i in range(n):
        seen = np.flatnonzero(see[i])
        if len(seen) == 0:
            continue
        for h in range(hq):
            kk, vv = k[seen, h // group], v[seen, h // group]
            if np.isnan(kk).any() or np.isnan(vv).any() or not np.isfinite(q[i, h]).all():
                out[i, h] = math.nan
                continue
            z = kk @ q[i, h] * scale
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h] = p @ vv
            weight[i, h] = p @ np.abs(vv)
            s[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, weight, s


def visible(n, kv, causal=True, window=0, tree=None):
    """[n, kv] bool: which keys the n new tokens of a sequence see (tree: their n words)."""
    j = np.arange(kv)[None]
    if not causal:
        return np.ones((n, kv), bool)
    past = kv - n
    p = past + np.arange(n)[:, None]
    if tree is not None:
        bit = np.clip(j - past, 0, 63).astype(np.uint64)
        return (j < past) | ((tree[:, None].astype(np.uint64) >> bit) & np.uint64(1) == 1)
    see = j <= p
    return see & (j > p - window) if window else see


def tolerance(out, weight, s, dtype):
    """The bound of include/nvfp4.h, and the rounding of a bf16 result."""
    tol = (2.0 ** -10 + 2.0 ** -15 * s) * weight + 1e-30
    return tol + 2.0 ** -8 * np.abs(out) if dtype == torch.bfloat16 else tol


def to_np(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()
