"""Timing cases of the quantised paged KV cache and the attention that reads it.

Three operators (see include/nvfp4.h):

* append     bf16 K and V rows of new tokens are quantised into pages of the
             cache (8-bit E4M3 codes, or NVFP4: 4-bit E2M1 codes with an E4M3
             scale per 16 elements; both with one power of two per row);
* read       rows of the cache come back as bf16;
* attention  new tokens (one per sequence in decode, a few in a speculative
             verify, a chunk in prefill) attend to their sequences' pages.

`run` computes them in plain torch operations in fp32 (`own` false) or through
the library (`own` true).  `exact` evaluates the definitions in fp64.

The cache is one uint8 pool[page][kv_head][2 (K, V)][block]; a block holds the
rows of one page: page_size rows of codes, then (NVFP4) page_size rows of
head_dim / 16 scale bytes, then page_size row exponents e (value 2^(e - 127),
255 marks a row that is not a number).
"""
from __future__ import annotations

import math

import torch

own = False

E4M3, NVFP4 = "e4m3", "nvfp4"
_DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _rows(name, op, fmt, tokens, kv_heads=8, head_dim=128, page_size=64, padding=0):
    return {"name": name, "op": op, "fmt": fmt, "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim,
            "page_size": page_size, "padding": padding}


def _attn(name, fmt, seqs, q_len, past_min, past_max, q_heads=32, kv_heads=8, head_dim=128, page_size=64,
          ragged=False, causal=True, window=0, tree=False):
    return {"name": name, "op": "attention", "fmt": fmt, "seqs": seqs, "q_len": q_len, "past_min": past_min,
            "past_max": past_max, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "page_size": page_size, "ragged": ragged, "causal": causal, "window": window, "tree": tree}


def listed():
    """Head layouts: 32 query and 8 KV heads of 128 are the 9B-class layer's
    (QKV 6144 = (32 + 2 * 8) * 128, O 4096), 40 and 8 the 27B-class layer's
    (QKV 7168, O 5120).  Token counts: 1 (decode), 4 and 16 (verify), 512 and
    2048 (prefill) are the benchmark's."""
    return [
        # one decoded token of one sequence enters the cache: pure latency
        _rows("append one token e4m3", "append", E4M3, 1),
        # one decode step of a batch of 61 sequences, three slots of it idle
        _rows("append batch nvfp4", "append", NVFP4, 61, padding=3, page_size=16),
        # a prefill of 8192 tokens enters the cache
        _rows("append prefill nvfp4", "append", NVFP4, 8192),
        # a prefix of odd length is read back (to be moved or re-paged)
        _rows("read prefix e4m3", "read", E4M3, 4999, page_size=32),
        # a long context is read back
        _rows("read context nvfp4", "read", NVFP4, 65536),
        # decode of one sequence with a short context: the smallest attention call
        _attn("decode short e4m3", E4M3, 1, 1, 555, 555),
        # decode of one sequence with a long context, 27B-class heads
        _attn("decode long nvfp4", NVFP4, 1, 1, 131071, 131071, q_heads=40),
        # decode of a batch whose contexts differ thirty-fold
        _attn("decode batch e4m3", E4M3, 64, 1, 257, 8191),
        # speculative verify of 16-token trees, 27B-class heads
        _attn("verify tree nvfp4", NVFP4, 8, 16, 2000, 6001, q_heads=40, tree=True),
        # a prefill chunk of 512 tokens behind a cached prefix, sliding window
        _attn("chunk window e4m3", E4M3, 2, 512, 5000, 7003, window=4096),
        # ragged prefill chunks without a prefix, heads of 64
        _attn("prefill ragged nvfp4", NVFP4, 4, 1500, 1, 1, q_heads=16, kv_heads=4, head_dim=64, ragged=True),
        # a chunk of 2048 tokens behind a long prefix, 27B-class heads: the largest
        _attn("chunk long e4m3", E4M3, 1, 2048, 14336, 14336, q_heads=40),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Append and read: 1 to 8192 and 65536 tokens.  Attention: decode (1 to
    128 sequences, contexts up to 131072), verify (2 to 16 tokens, causal or
    tree), chunks of 17 to 2048 tokens, and cross attention to states of
    another length; heads in groups of 1 to 8."""
    fmt = rng.choice([E4M3, NVFP4])
    page_size = rng.choice([16, 32, 64, 128])
    if rng.random() < 0.35:
        op = rng.choice(["append", "read"])
        c = _rows("", op, fmt, _log(rng, 1, 8192 if op == "append" else 65536), rng.choice([1, 2, 4, 8]),
                  rng.choice([64, 128, 128]), page_size, rng.choice([0, 0, 1, 5]))
    else:
        hq, hk, d = rng.choice([(32, 8, 128), (40, 8, 128), (16, 16, 64), (12, 4, 64), (8, 1, 128), (24, 8, 128)])
        kind = rng.choice(["decode", "decode", "verify", "chunk", "cross"])
        past = _log(rng, 1, 131000 if kind == "decode" else 14000)
        seqs = _log(rng, 1, max(1, min(128, 131072 // max(past, 1024))))
        q_len, ragged, causal, tree, window = 1, False, True, False, 0
        if kind == "verify":
            q_len, tree, seqs = rng.randint(2, 16), rng.random() < 0.5, min(seqs, 16)
        elif kind == "chunk":
            q_len, ragged, seqs = _log(rng, 17, 2048), rng.random() < 0.5, min(seqs, 4)
        elif kind == "cross":
            q_len, causal, seqs, past = _log(rng, 1, 512), False, min(seqs, 4), min(past, 6000)
        if causal and not tree and rng.random() < 0.25:
            window = _log(rng, 16, 8192)
        if seqs * q_len > 2048:
            seqs = max(1, 2048 // q_len)
        c = _attn("", fmt, seqs, q_len, max(1, past // rng.choice([1, 2, 8])), past, hq, hk, d, page_size, ragged,
                  causal, window, tree)
    del c["name"]
    return c


def _past_lens(c):
    """Cached tokens before the call, per sequence: spread evenly over the logarithm."""
    n, lo, hi = c["seqs"], c["past_min"], c["past_max"]
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (b / (n - 1)))) for b in range(n)]


def _q_lens(c):
    if not c["ragged"]:
        return [c["q_len"]] * c["seqs"]
    return [c["q_len"] if b == 0 else 1 + (b * 7919 + 311) % c["q_len"] for b in range(c["seqs"])]


def _kv_lens(c):
    """Tokens in the cache during the call: the new ones are in it, unless the keys are another sequence's."""
    return [p + (n if c["causal"] else 0) for p, n in zip(_past_lens(c), _q_lens(c))]


def _row_bytes(fmt, d):
    return (d if fmt == E4M3 else d // 2 + d // 16) + 1


def work(case):
    c = case
    if c["op"] != "attention":
        values = c["tokens"] * c["kv_heads"] * c["head_dim"] * 2
        cached = c["tokens"] * c["kv_heads"] * 2 * _row_bytes(c["fmt"], c["head_dim"])
        if c["op"] == "read":
            return {"bytes": cached + 2 * values + 8 * c["tokens"], "flops": 0}
        # read bf16, write codes, read them back, write bf16
        return {"bytes": 2 * values + 2 * cached + 2 * values + 8 * c["tokens"], "flops": 0}
    pairs = keys = 0
    for past, n, kv in zip(_past_lens(c), _q_lens(c), _kv_lens(c)):
        if not c["causal"]:
            pairs, keys = pairs + n * kv, keys + kv
            continue
        w = c["window"] or kv
        first = max(0, past + 1 - w)
        keys += kv - first
        pairs += sum(min(past + i + 1, w) for i in range(n))
    total_q = sum(_q_lens(c))
    return {"bytes": keys * c["kv_heads"] * 2 * _row_bytes(c["fmt"], c["head_dim"])
            + 2 * 2 * total_q * c["q_heads"] * c["head_dim"],
            "flops": 4 * c["head_dim"] * c["q_heads"] * pairs}


# ---------------------------------------------------------------------------
# The cache format in plain torch operations
# ---------------------------------------------------------------------------

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_E2M1_FROM = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]  # where codes 1 to 7 begin; a tie goes to the even code


def _exponent(amax, top):
    """The smallest k with amax <= top * 2^k, at least -100 (fp32, exact)."""
    f, e = torch.frexp(amax)
    ft, et = math.frexp(top)
    return torch.clamp(e - et + (f > ft), min=-100)


def _encode(x, fmt):
    """bf16 rows [..., D] to codes, scales (None for E4M3) and exponents, uint8."""
    x = x.float()
    d = x.shape[-1]
    amax = x.abs().amax(-1)
    k = _exponent(amax, 448.0 if fmt == E4M3 else 2688.0)
    bad = ~torch.isfinite(amax) | torch.isnan(x).any(-1) | (k > 100)
    k = torch.where(bad, torch.zeros_like(k), k)
    x = torch.where(bad[..., None], torch.zeros_like(x), x)
    y = torch.ldexp(x, -k[..., None])
    e = torch.where(bad, torch.full_like(k, 255), k + 127).to(torch.uint8)
    if fmt == E4M3:
        return y.to(torch.float8_e4m3fn).view(torch.uint8), None, e
    y = y.unflatten(-1, (d // 16, 16))
    bamax = torch.ldexp((x.abs().unflatten(-1, (d // 16, 16)).amax(-1) / 6), -k[..., None])
    scale = bamax.to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    q = torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    begin = torch.tensor(_E2M1_FROM, device=x.device)
    begin[0::2] = torch.nextafter(begin[0::2], begin[0::2] + 1)
    code = torch.bucketize(q.abs(), begin, right=True).to(torch.uint8)
    code |= (torch.signbit(q) & (s > 0)).to(torch.uint8) << 3
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8), e


def _decode(codes, scales, e):
    """Codes, scales and exponents (uint8) to fp32 rows."""
    if scales is None:
        x = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(_E2M1 + [-v for v in _E2M1], device=codes.device)
        x = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
        x = (x.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)
    x = torch.ldexp(x, e.int()[..., None] - 127)
    return torch.where((e == 255)[..., None], torch.full_like(x, math.nan), x)


def _planes(pool, page_size, d, fmt):
    """Views of a pool[..., block]: codes, scales or None, exponents, each [..., page_size, bytes of a row]."""
    cb = d if fmt == E4M3 else d // 2
    sb = 0 if fmt == E4M3 else d // 16
    codes = pool[..., :page_size * cb].unflatten(-1, (page_size, cb))
    scales = pool[..., page_size * cb:page_size * (cb + sb)].unflatten(-1, (page_size, sb)) if sb else None
    return codes, scales, pool[..., page_size * (cb + sb):]


# ---------------------------------------------------------------------------
# States
# ---------------------------------------------------------------------------

def _rand_kv(gen, tokens, heads, d):
    """[tokens, heads, 2 (K, V), d]: K with a few strong channels, V with token norms that differ, as trained layers have them."""
    dev = gen.device
    k = torch.randn(tokens, heads, d, device=dev, generator=gen)
    k *= 1 + 5 * (torch.rand(1, heads, d, device=dev, generator=gen) < 0.03)
    v = torch.randn(tokens, heads, d, device=dev, generator=gen)
    v *= torch.exp(0.7 * torch.randn(tokens, heads, 1, device=dev, generator=gen))
    return torch.stack((k, v), 2).to(torch.bfloat16)


def _store(pool, page_size, fmt, kv, slots, idle=None):
    """Writes bf16 rows kv[tokens, heads, 2 (K, V), D] to the slots of a pool, but for those of `idle` tokens."""
    planes = _planes(pool, page_size, kv.shape[-1], fmt)
    page, at = slots // page_size, slots % page_size
    codes, scales, exps = _encode(kv, fmt)
    if idle is not None:
        keep = idle[:, None, None]
        codes = torch.where(keep[..., None], planes[0][page, :, :, at], codes)
        scales = None if scales is None else torch.where(keep[..., None], planes[1][page, :, :, at], scales)
        exps = torch.where(keep, planes[2][page, :, :, at], exps)
    planes[0][page, :, :, at] = codes
    planes[2][page, :, :, at] = exps
    if scales is not None:
        planes[1][page, :, :, at] = scales


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=_DEVICE)
    gen.manual_seed(seed)
    fmt, ps, hk, d = c["fmt"], c["page_size"], c["kv_heads"], c["head_dim"]
    block = ps * _row_bytes(fmt, d)
    s = {"case": c}
    if c["op"] != "attention":
        n = c["tokens"]
        pages = -(-n // ps) + 3
        s["pool"] = torch.randint(0, 256, (pages, hk, 2, block), dtype=torch.uint8, device=_DEVICE, generator=gen)
        order = torch.randperm(pages - 1, device=_DEVICE, generator=gen)  # the last page stays free
        at = torch.arange(n, device=_DEVICE)
        slots = order[at // ps] * ps + at % ps
        # K and V are slices of a fused projection's output: rows of all heads, strided
        qkv = torch.ones(n, (4 + 2) * hk * d, dtype=torch.bfloat16, device=_DEVICE)
        kv = _rand_kv(gen, n, hk, d)
        s["k"] = qkv[:, 4 * hk * d:5 * hk * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, 5 * hk * d:].unflatten(1, (hk, d))
        s["k"].copy_(kv[:, :, 0])
        s["v"].copy_(kv[:, :, 1])
        if c["op"] == "read":
            _store(s["pool"], ps, fmt, kv, slots)
        slots[max(1, n - c["padding"]):] = -1  # idle places of a batch of fixed size
        s["slots"] = slots
        s["out"] = tuple(torch.empty(n, hk, d, dtype=torch.bfloat16, device=_DEVICE) for _ in range(2))
        if own:
            import gemm_nvfp4_gb300 as g
            s["workspace"] = torch.zeros(g.nvfp4_workspace_bytes(g.NVFP4_OP_KV_APPEND, n, hk, d), dtype=torch.uint8,
                                         device=_DEVICE)
        return s
    past, ql, kl = _past_lens(c), _q_lens(c), _kv_lens(c)
    need = [-(-n // ps) for n in kl]
    order = torch.randperm(sum(need) + 2, device=_DEVICE, generator=gen)
    s["pool"] = torch.zeros(sum(need) + 2, hk, 2, block, dtype=torch.uint8, device=_DEVICE)
    width = max(need)
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=_DEVICE)
    first = 0
    for b, n in enumerate(need):
        table[b, :n] = order[first:first + n].int()
        at = torch.arange(kl[b], device=_DEVICE)
        slots = table[b].long()[at // ps] * ps + at % ps
        _store(s["pool"], ps, fmt, _rand_kv(gen, kl[b], hk, d), slots)
        first += n
    total = sum(ql)
    s["block_table"] = table
    s["kv_lens"] = torch.tensor(kl, dtype=torch.int32, device=_DEVICE)
    s["q"] = (1.5 * torch.randn(total, c["q_heads"], d, device=_DEVICE, generator=gen)).to(torch.bfloat16)
    s["q_offsets"] = torch.tensor([0] + ql, device=_DEVICE).cumsum(0).int() if c["ragged"] else None
    s["tree"] = None
    if c["tree"]:
        # bit j of token i's word: i descends from the sequence's new token j (or is it)
        n = c["q_len"]
        parent = torch.rand(c["seqs"], n, generator=gen, device=_DEVICE)
        words = torch.zeros(c["seqs"], n, dtype=torch.int64, device=_DEVICE)
        rows = torch.arange(c["seqs"], device=_DEVICE)
        for i in range(n):
            up = words[rows, (parent[:, i] * i).long()] if i else 0
            words[:, i] = up | (1 << i)
        s["tree"] = words.flatten()
    s["out"] = torch.empty(total, c["q_heads"], d, dtype=torch.bfloat16, device=_DEVICE)
    if own:
        import gemm_nvfp4_gb300 as g
        # the scratch that a serving program keeps for all its attention calls
        need = g.nvfp4_paged_attention_workspace_bytes(_cache(s), s["q"], len(ql), max(ql))
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device=_DEVICE)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _cache(s):
    import gemm_nvfp4_gb300 as g
    c = s["case"]
    return g.KVCache(s["pool"], c["page_size"], c["head_dim"], g.NVFP4_KV_E4M3 if c["fmt"] == E4M3 else g.NVFP4_KV_NVFP4)


def _run_own(s):
    import gemm_nvfp4_gb300 as g
    c, cache = s["case"], _cache(s)
    if c["op"] == "attention":
        return g.nvfp4_paged_attention(s["q"], cache, s["block_table"], s["kv_lens"], q_offsets=s["q_offsets"],
                                       max_q_len=c["q_len"], causal=c["causal"], window=c["window"], tree=s["tree"],
                                       out=s["out"], workspace=s["workspace"])
    if c["op"] == "append":
        g.nvfp4_kv_append(cache, s["k"], s["v"], s["slots"], workspace=s["workspace"])
    return g.nvfp4_kv_read(cache, s["slots"], out=s["out"], workspace=s["workspace"])


def run(state):
    """One pass: append and read return the slots' K and V rows in bf16 (zeros
    for an idle slot, -1), attention its output [tokens, heads, D] in bf16."""
    if own:
        return _run_own(state)
    if state["case"]["op"] == "attention":
        return _plain_attention(state)
    return _plain_rows(state)


def _plain_rows(s):
    c = s["case"]
    pool, slots, ps, d, fmt = s["pool"], s["slots"], c["page_size"], c["head_dim"], c["fmt"]
    idle = slots < 0
    codes, scales, exps = _planes(pool, ps, d, fmt)
    # idle tokens go to the last page, where no slot is looked at, and leave it as it is
    to = torch.where(idle, torch.full_like(slots, pool.shape[0] * ps - 1), slots)
    page, at = to // ps, to % ps
    if c["op"] == "append":
        _store(pool, ps, fmt, torch.stack((s["k"], s["v"]), 2), to, idle)
    x = _decode(codes[page, :, :, at], None if scales is None else scales[page, :, :, at], exps[page, :, :, at])
    x = torch.where(idle[:, None, None, None], torch.zeros_like(x), x).to(torch.bfloat16)
    return x[:, :, 0].contiguous(), x[:, :, 1].contiguous()


def _plain_attention(s):
    """softmax(q . K^T / sqrt(D), masked) . V in fp32, all sequences padded to the longest."""
    c = s["case"]
    ps, d, fmt, hk = c["page_size"], c["head_dim"], c["fmt"], c["kv_heads"]
    g = c["q_heads"] // hk
    b, width = s["block_table"].shape
    q, kv_lens, dev = s["q"], s["kv_lens"].long(), s["q"].device
    # the cache's rows, [b, hk, keys, d]
    pages = s["pool"][s["block_table"].clamp(min=0).long()]
    planes = _planes(pages, ps, d, fmt)
    k, v = (_decode(*(None if p is None else p[:, :, :, j].transpose(1, 2).flatten(2, 3) for p in planes))
            for j in range(2))
    j = torch.arange(width * ps, device=dev)
    inside = j < kv_lens[:, None]
    v = torch.where(inside[:, None, :, None], v, torch.zeros_like(v))
    # the queries, [b, hk, g * n, d]
    n = c["q_len"]
    first = s["q_offsets"].long() if s["q_offsets"] is not None else torch.arange(b + 1, device=dev) * n
    i = torch.arange(n, device=dev)
    lens = first[1:] - first[:-1]
    row = (first[:-1, None] + torch.minimum(i, lens[:, None] - 1))
    qs = q[row].float().view(b, n, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * n, d)
    # which keys a new token sees, [b, n, keys]
    past = kv_lens - lens if c["causal"] else kv_lens
    pos = past[:, None] + i
    see = inside[:, None, :].expand(b, n, -1)
    if c["tree"]:
        bit = (j[None] - past[:, None]).clamp(0, 63)
        marked = (s["tree"].view(b, n)[:, :, None] >> bit[:, None, :]) & 1
        see = see & ((j[None, None] < past[:, None, None]) | (marked == 1))
    elif c["causal"]:
        see = see & (j <= pos[..., None])
        if c["window"]:
            see = see & (j > pos[..., None] - c["window"])
    scores = (qs @ k.transpose(2, 3)).view(b, hk, g, n, -1) * d ** -0.5
    scores = scores.masked_fill(~see[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1)
    out = (p.view(b, hk, g * n, -1) @ v).view(b, hk, g, n, d) / torch.where(total == 0, 1.0, total)[..., None]
    out = out.permute(0, 3, 1, 2, 4).reshape(b, n, hk * g, d).to(torch.bfloat16)
    if s["q_offsets"] is None:
        return out.reshape(b * n, hk * g, d)
    return out[i < lens[:, None]]


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_values():
    """The value of every E4M3 byte, in fp64."""
    out = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out.append(math.nan if byte & 127 == 127 else -x if byte & 128 else x)
    return torch.tensor(out, dtype=torch.float64)


def _nearest(x, values):
    """The nearest of ascending `values` to x >= 0, a tie to the even place; above the last: the last."""
    mid = (values[1:] + values[:-1]) / 2
    at = torch.searchsorted(mid, x.contiguous())  # places strictly below x, in mid
    tie = x == mid[at.clamp(max=mid.numel() - 1)]
    return values[torch.where(tie & (at % 2 == 1), at + 1, at)]


def _exact_row_values(x, fmt):
    """What rows of x (fp64) are worth once they are in the cache."""
    e4 = _e4m3_values()[:127].to(x.device)
    e2 = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    amax = x.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(amax / (448 if fmt == E4M3 else 2688)))
    top = 448 if fmt == E4M3 else 2688
    k = torch.where(amax > top * torch.exp2(k), k + 1, torch.where(amax <= top * torch.exp2(k - 1), k - 1, k))
    unit = torch.exp2(torch.clamp(k, min=-100))
    if fmt == E4M3:
        return torch.sign(x) * _nearest(x.abs() / unit, e4) * unit
    blocks = x.unflatten(-1, (-1, 16))
    scale = _nearest(blocks.abs().amax(-1, keepdim=True) / 6 / unit[..., None], e4)
    code = _nearest(torch.where(scale > 0, blocks.abs() / unit[..., None] / scale.clamp(min=2.0 ** -20), 0.0), e2)
    return (torch.sign(blocks) * code * scale * unit[..., None]).flatten(-2)


def _exact_cached(s, b, length):
    """K and V rows of a sequence's first `length` keys from the bytes of its pages, in fp64: [length, hk, d] each."""
    c = s["case"]
    ps, d, hk, pool = c["page_size"], c["head_dim"], c["kv_heads"], s["pool"]
    cb = d if c["fmt"] == E4M3 else d // 2
    values = _e4m3_values().to(pool.device)
    nibble = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device=pool.device)
    where = torch.arange(length, device=pool.device)
    page, at = s["block_table"][b, where // ps].long(), where % ps
    flat = pool.view(pool.shape[0], -1)
    base = torch.arange(hk * 2, device=pool.device) * (flat.shape[1] // (hk * 2))

    def take(offset, width):  # bytes [length, hk * 2, width] at `offset` + row * width of each block
        col = base[None, :, None] + (offset + at[:, None, None] * width) + torch.arange(width, device=pool.device)
        return flat[page[:, None, None], col].long()

    if c["fmt"] == E4M3:
        x = values[take(0, d)]
        e = take(ps * d, 1)
    else:
        raw = take(0, cb)
        x = torch.empty(length, hk * 2, d, dtype=torch.float64, device=pool.device)
        x[..., 0::2], x[..., 1::2] = nibble[raw % 16], nibble[raw // 16]
        x *= values[take(ps * cb, d // 16)].repeat_interleave(16, -1)
        e = take(ps * (cb + d // 16), 1)
    x = (x * torch.exp2(e.double() - 127)).view(length, hk, 2, d)
    return x[:, :, 0], x[:, :, 1]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] != "attention":
        kv = [_exact_row_values(x.double(), c["fmt"]) for x in (s["k"], s["v"])]
        return tuple(torch.where((s["slots"] < 0)[:, None, None], torch.zeros_like(x), x) for x in kv)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    g = c["q_heads"] // c["kv_heads"]
    begin = 0
    for b, (past, n, kl) in enumerate(zip(_past_lens(c), _q_lens(c), _kv_lens(c))):
        k, v = _exact_cached(s, b, kl)
        at = torch.arange(kl, device=out.device)
        for lo in range(0, n, 256):
            hi = min(n, lo + 256)
            see = torch.ones(hi - lo, kl, dtype=torch.bool, device=out.device)
            if c["causal"]:
                here = torch.arange(past + lo, past + hi, device=out.device)[:, None]
                see = at <= here
                if c["window"]:
                    see &= at > here - c["window"]
                if c["tree"]:
                    bits = s["tree"][begin + lo:begin + hi, None] >> (at - past).clamp(min=0, max=63)
                    see = (at < past) | (bits % 2 != 0)
            for h in range(c["q_heads"]):
                z = (s["q"][begin + lo:begin + hi, h].double() @ k[:, h // g].T) / math.sqrt(c["head_dim"])
                z = torch.softmax(torch.where(see, z, -math.inf), -1)
                out[begin + lo:begin + hi, h] = z @ v[:, h // g]
        begin += n
    return out
