"""Timing cases of what a decoder layer's attention half needs around its cache.

Three operators (see include/nvfp4.h):

* product   y = residual + act(x . dequant(W)^T + bias) for NVFP4 and FP6
            weights: the QKV product with its bias, the O and down products
            with their residual, an up product with its activation;
* rotate    rotary positions of q and k with one position per axis and token
            (text: one axis; images and video: height and width, or time,
            height and width);
* prompt    attention of packed whole prompts over their own K and V in bf16:
            causal, in a sliding window, or every token to every other.

`run` computes them in plain torch operations in fp32 (`own` false) or through
the library (`own` true).  `exact` evaluates the definitions in fp64.
"""
from __future__ import annotations

import math

import torch

own = False

NVFP4, FP6 = "nvfp4", "fp6"
_DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _product(name, fmt, n, k, m, bias="", act="none", residual="", out="bf16"):
    return {"name": name, "op": "product", "fmt": fmt, "n": n, "k": k, "m": m, "bias": bias, "act": act,
            "residual": residual, "out": out}


def _rotate(name, tokens, q_heads, kv_heads, head_dim, rotary, axes, adjacent=False, dtype="bf16", first=0):
    return {"name": name, "op": "rotate", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary": rotary, "axes": axes, "adjacent": adjacent, "dtype": dtype, "first": first}


def _prompt(name, seqs, len_min, len_max, q_heads=32, kv_heads=8, head_dim=128, causal=True, window=0, empty=0,
            behind=0):
    return {"name": name, "op": "prompt", "seqs": seqs, "len_min": len_min, "len_max": len_max, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "causal": causal, "window": window, "empty": empty,
            "behind": behind}


def listed():
    """Products and head layouts are the 9B-class layer's (QKV 4096 -> 6144 =
    (32 + 2 * 8) * 128) and the 27B-class layer's (O 5120 -> 5120, gate and up
    5120 -> 17408, down 17408 -> 5120, 40 and 8 heads); token counts 1, 4, 512
    and 2048 are the benchmark's."""
    return [
        # one decoded token's QKV product with its bias
        _product("qkv bias one token", NVFP4, 1, 4096, 6144, bias="bf16"),
        # a verify of four tokens adds its O product to the residual stream
        _product("o residual verify", NVFP4, 4, 5120, 5120, residual="bf16"),
        # a prefill of an odd number of tokens through an ungated MLP's first product
        _product("up gelu ragged", NVFP4, 509, 5120, 17408, bias="bf16", act="gelu_tanh"),
        # a prefill's down product in FP6 weights onto an fp32 residual stream
        _product("down residual fp6", FP6, 2048, 17408, 5120, residual="f32", out="f32"),
        # one decoded token far into its text: pure latency
        _rotate("rotate one token", 1, 32, 8, 128, 128, 1, first=100000),
        # a prompt of text, images and video: time, height and width
        _rotate("rotate three axes", 8192, 40, 8, 128, 128, 3),
        # patches of an image tower: height and width, neighbouring elements paired, half of each head, fp32
        _rotate("rotate patches", 4999, 16, 16, 64, 32, 2, adjacent=True, dtype="f32"),
        # one short prompt: the smallest call
        _prompt("prompt short", 1, 77, 77),
        # a batch of prompts that differ hundredfold, packed into a buffer with idle rows
        _prompt("prompts packed", 24, 19, 2500, empty=1, behind=5),
        # a sliding window layer, heads of 64
        _prompt("prompt window", 1, 8191, 8191, q_heads=16, kv_heads=4, head_dim=64, window=1024),
        # images whose tokens all see one another, a KV head per query head
        _prompt("images", 5, 577, 2305, q_heads=16, kv_heads=16, head_dim=64, causal=False),
        # one long prompt, 27B-class heads: the largest
        _prompt("prompt long", 1, 16384, 16384, q_heads=40),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu", "relu2"]


def draw(rng):
    """Products of 1 to 2048 tokens and matrices up to 17408 x 5120; rotations
    of 1 to 8192 tokens with one to four axes; prompts of 1 to 64 sequences and
    up to 16384 tokens in all."""
    op = rng.choice(["product", "rotate", "prompt", "prompt"])
    if op == "product":
        fmt = rng.choice([NVFP4, NVFP4, FP6])
        n = _log(rng, 1, 16) if rng.random() < 0.5 else _log(rng, 17, 2048)
        wide, deep = _log(rng, 100, 17408), _log(rng, 100, 5120)
        m, k = (wide, deep) if rng.random() < 0.6 else (deep, wide)
        unit = 128 if fmt == FP6 else rng.choice([16, 64, 256])
        c = _product("", fmt, n, max(unit, k // unit * unit), m, rng.choice(["", "bf16", "f32"]), rng.choice(_ACTS),
                     rng.choice(["", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"]))
    elif op == "rotate":
        hq, hk = rng.choice([(32, 8), (40, 8), (16, 16), (12, 4), (8, 1), (7, 7)])
        d = rng.choice([64, 128, 128, 80, 96])
        rotary = rng.choice([d, d, d // 2, d // 4])
        c = _rotate("", _log(rng, 1, 8192), hq, hk, d, rotary, rng.choice([1, 2, 3, 3, 4]), rng.random() < 0.3,
                    rng.choice(["bf16", "bf16", "f32"]), rng.choice([0, 0, 5000, 131072, 1000000]))
    else:
        hq, hk, d = rng.choice([(32, 8, 128), (40, 8, 128), (16, 16, 64), (12, 4, 64), (8, 1, 128), (24, 8, 128),
                                (14, 2, 64)])
        seqs = _log(rng, 1, 64)
        longest = _log(rng, 1, 16384 // seqs if seqs > 1 else 12000)
        causal = rng.random() < 0.75
        if not causal:
            longest = min(longest, 6000)
        window = _log(rng, 1, 4096) if causal and rng.random() < 0.3 else 0
        c = _prompt("", seqs, max(1, longest // rng.choice([1, 3, 40])), longest, hq, hk, d, causal, window,
                    rng.choice([0, 0, 1, 3]), rng.choice([0, 0, 1, 130]))
    del c["name"]
    return c


def _lens(c):
    """Lengths of a case's sequences: spread evenly over the logarithm, out of order, some of them empty."""
    n, lo, hi = c["seqs"], c["len_min"], c["len_max"]
    lens = [hi] if n == 1 else [int(round(lo * (hi / lo) ** (b / (n - 1)))) for b in range(n)]
    lens = sorted(lens, key=lambda x: (x * 7919 + 311) % 1009)
    for e in range(c["empty"]):
        lens.insert(e * 2, 0)
    return lens


def work(case):
    c = case
    if c["op"] == "product":
        n, k, m = c["n"], c["k"], c["m"]
        size = {"": 0, "bf16": 2, "f32": 4}
        weights = m * k // 2 + m * k // 16 if c["fmt"] == NVFP4 else m * k * 3 // 4 + m * k // 128
        return {"bytes": weights + 2 * n * k + size[c["bias"]] * m + (size[c["residual"]] + size[c["out"]]) * n * m,
                "flops": 2 * n * m * k}
    if c["op"] == "rotate":
        heads = c["tokens"] * (c["q_heads"] + c["kv_heads"])
        return {"bytes": 2 * heads * c["head_dim"] * (4 if c["dtype"] == "f32" else 2) + 8 * c["axes"] * c["tokens"],
                "flops": 3 * heads * c["rotary"]}
    pairs = tokens = 0
    for n in _lens(c):
        tokens += n
        if not c["causal"]:
            pairs += n * n
        else:
            w = min(c["window"] or n, n)
            pairs += w * (w + 1) // 2 + (n - w) * w
    return {"bytes": 2 * tokens * c["head_dim"] * 2 * (c["q_heads"] + c["kv_heads"]),
            "flops": 4 * c["head_dim"] * c["q_heads"] * pairs}


# ---------------------------------------------------------------------------
# Weight formats in plain torch operations
# ---------------------------------------------------------------------------

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_E2M3 = [j / 8 for j in range(8)] + [2.0 ** e * (1 + j / 8) for e in range(3) for j in range(8)]


def _nearest_code(x, values):
    """Index of the nearest of ascending values (a tie to the even index), magnitudes beyond the last to the last."""
    v = torch.tensor(values, device=x.device)
    mid = (v[1:] + v[:-1]) / 2
    mid[0::2] = torch.nextafter(mid[0::2], mid[0::2] + 1)  # a tie between codes 0 and 1 stays at 0, 2 and 3 at 2
    return torch.bucketize(x, mid, right=True).to(torch.uint8)


def _quantize(w, fmt):
    """fp32 weights to codes, scales and (NVFP4) the tensor scale."""
    m, k = w.shape
    if fmt == NVFP4:
        ts = w.abs().amax() / 2688
        blocks = w.view(m, k // 16, 16)
        scales = (blocks.abs().amax(-1) / 6 / ts).to(torch.float8_e4m3fn)
        d = (scales.float() * ts)[..., None]
        y = torch.where(d > 0, blocks / d.clamp(min=1e-30), torch.zeros_like(blocks)).view(m, k)
        codes = _nearest_code(y.abs(), _E2M1) | (y < 0).to(torch.uint8) << 3
        return codes[:, 0::2] | codes[:, 1::2] << 4, scales.view(torch.uint8), ts.view(1)
    blocks = w.view(m, k // 128, 128)
    shared = (torch.frexp(blocks.abs().amax(-1))[1] - 3).clamp(min=-127)
    y = torch.ldexp(blocks, -shared[..., None]).view(m, k)
    codes = (_nearest_code(y.abs(), _E2M3) | (y < 0).to(torch.uint8) << 5).view(m, k // 4, 4).int()
    word = codes[..., 0] | codes[..., 1] << 6 | codes[..., 2] << 12 | codes[..., 3] << 18
    packed = torch.stack((word & 255, word >> 8 & 255, word >> 16), -1).to(torch.uint8)
    return packed.view(m, k // 4 * 3), (shared + 127).to(torch.uint8), None


def _dequantize(codes, scales, ts):
    """fp32 weights from codes, scales and the tensor scale (None: FP6)."""
    m = codes.shape[0]
    if ts is not None:
        table = torch.tensor(_E2M1 + [-v for v in _E2M1], device=codes.device)
        x = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).view(m, -1, 16)
        return (x * (scales.view(torch.float8_e4m3fn).float()[..., None] * ts)).view(m, -1)
    table = torch.tensor(_E2M3 + [-v for v in _E2M3], device=codes.device)
    b = codes.view(m, -1, 3).int()
    word = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16
    x = torch.stack([table[(word >> s & 63).long()] for s in (0, 6, 12, 18)], -1).view(m, -1, 128)
    return torch.ldexp(x, (scales.int() - 127)[..., None]).view(m, -1)


# ---------------------------------------------------------------------------
# States
# ---------------------------------------------------------------------------

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _heads(gen, tokens, q_heads, kv_heads, d, dtype, v_heads):
    """Q, K (and V) as column ranges of one product's output."""
    total = (q_heads + kv_heads + v_heads) * d
    x = torch.randn(tokens, total, device=_DEVICE, generator=gen)
    # a few strong channels, as trained layers have them
    x[:, :(q_heads + kv_heads) * d] *= 1 + 3 * (torch.rand((q_heads + kv_heads) * d, device=_DEVICE, generator=gen) < 0.03)
    x = x.to(dtype)
    q, k, v = x.split((q_heads * d, kv_heads * d, v_heads * d), 1)
    return q.unflatten(1, (q_heads, d)), k.unflatten(1, (kv_heads, d)), v.unflatten(1, (v_heads, d)) if v_heads else None


def _inv_freq(c):
    """Frequency of each pair: base 10^6 over the rotary elements."""
    return [1e6 ** (-2 * i / c["rotary"]) for i in range(c["rotary"] // 2)]


def _axis(c):
    """Axis of each pair: sections in order (16, 24 and 24 of 64 pairs for time, height and width)."""
    pairs = c["rotary"] // 2
    later = {1: 0, 2: pairs // 2, 3: pairs * 3 // 8, 4: pairs // 4}[c["axes"]]
    first = pairs - later * (c["axes"] - 1)
    return [0 if i < first else 1 + (i - first) // later for i in range(pairs)]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=_DEVICE)
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "product":
        n, k, m = c["n"], c["k"], c["m"]
        s["w"] = _quantize(0.02 * torch.randn(m, k, device=_DEVICE, generator=gen), c["fmt"])
        s["x"] = torch.randn(n, k, device=_DEVICE, generator=gen).to(torch.bfloat16)
        s["bias"] = s["residual"] = None
        if c["bias"]:
            s["bias"] = torch.randn(m, device=_DEVICE, generator=gen).to(_DTYPE[c["bias"]])
        if c["residual"]:
            s["residual"] = (2 * torch.randn(n, m, device=_DEVICE, generator=gen)).to(_DTYPE[c["residual"]])
        s["out"] = torch.empty(n, m, dtype=_DTYPE[c["out"]], device=_DEVICE)
        if own:
            import gemm_nvfp4_gb300 as g
            op = g.NVFP4_OP_GEMM_PREFILL if c["fmt"] == NVFP4 else g.NVFP4_OP_FP6_GEMM
            s["workspace"] = torch.zeros(max(16, g.nvfp4_workspace_bytes(op, n, m, k)), dtype=torch.uint8, device=_DEVICE)
        return s
    if c["op"] == "rotate":
        n, d = c["tokens"], c["head_dim"]
        q, k, _ = _heads(gen, n, c["q_heads"], c["kv_heads"], d, _DTYPE[c["dtype"]], 0)
        s["q"], s["k"] = q, k
        # runs of text (all axes advance together) and of images 32 patches wide (the first axis stands still)
        t = torch.arange(n, device=_DEVICE)
        image = (t // 1024) % 2 == 1
        rows = [torch.where(image, t // 1024 * 1024, t), torch.where(image, t // 1024 * 1024 + t % 1024 // 32, t),
                torch.where(image, t // 1024 * 1024 + t % 32, t), t]
        if c["axes"] == 2:
            rows = rows[1:]
        shift = int(torch.randint(0, 1000, (1,), device=_DEVICE, generator=gen)) + c["first"]
        s["positions"] = torch.stack(rows[:c["axes"]]) + shift
        s["out"] = tuple(torch.empty(n, h, d, dtype=q.dtype, device=_DEVICE) for h in (c["q_heads"], c["kv_heads"]))
        if own:
            import gemm_nvfp4_gb300 as g
            s["table"] = g.RopeTable.make(_inv_freq(c), _axis(c), device=_DEVICE)
        else:
            s["inv_freq"] = torch.tensor(_inv_freq(c), dtype=torch.float64, device=_DEVICE)
            s["axis"] = torch.tensor(_axis(c), device=_DEVICE)
        return s
    lens = _lens(c)
    rows = sum(lens) + c["behind"]
    s["q"], s["k"], s["v"] = _heads(gen, rows, c["q_heads"], c["kv_heads"], c["head_dim"], torch.bfloat16, c["kv_heads"])
    s["offsets"] = None
    if len(lens) > 1 or c["behind"]:
        s["offsets"] = torch.tensor([0] + lens, device=_DEVICE).cumsum(0).int()
    s["out"] = torch.zeros(rows, c["q_heads"], c["head_dim"], dtype=torch.bfloat16, device=_DEVICE)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_own(s):
    import gemm_nvfp4_gb300 as g
    c = s["case"]
    if c["op"] == "product":
        act = {"none": g.NVFP4_ACT_NONE, "silu": g.NVFP4_ACT_SILU, "gelu": g.NVFP4_ACT_GELU,
               "gelu_tanh": g.NVFP4_ACT_GELU_TANH, "relu": g.NVFP4_ACT_RELU, "relu2": g.NVFP4_ACT_RELU2}[c["act"]]
        call, w = ((g.nvfp4_gemm_epilogue, g.NVFP4Weight(*s["w"])) if c["fmt"] == NVFP4
                   else (g.nvfp4_fp6_gemm_epilogue, g.FP6Weight(*s["w"][:2])))
        return call(s["x"], w, bias=s["bias"], activation=act, residual=s["residual"], out=s["out"],
                    workspace=s["workspace"])
    if c["op"] == "rotate":
        return g.nvfp4_rope(s["q"], s["k"], s["positions"], s["table"], adjacent=c["adjacent"], out=s["out"])
    return g.nvfp4_prompt_attention(s["q"], s["k"], s["v"], offsets=s["offsets"], causal=c["causal"],
                                    window=c["window"], out=s["out"])


def run(state):
    """One pass: a product's y, a rotation's (q, k), a prompt's attention output [tokens, heads, D] (rows behind the
    last sequence as they were: zero)."""
    if own:
        return _run_own(state)
    return {"product": _plain_product, "rotate": _plain_rotate, "prompt": _plain_prompt}[state["case"]["op"]](state)


def _plain_product(s):
    c = s["case"]
    y = s["x"].float() @ _dequantize(*s["w"]).T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = y * (0.5 * (1 + torch.erf(y * 0.5 ** 0.5)))
    elif c["act"] == "gelu_tanh":
        y = y * (0.5 * (1 + torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y * y * y))))
    elif c["act"] in ("relu", "relu2"):
        y = y.clamp(min=0)
        y = y * y if c["act"] == "relu2" else y
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return y.to(_DTYPE[c["out"]])


def _plain_rotate(s):
    c = s["case"]
    pairs, adjacent = c["rotary"] // 2, c["adjacent"]
    angle = s["positions"].double()[s["axis"]].T * s["inv_freq"]  # 64 bits: far positions
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def one(x):
        f = x.float()
        rest = f[..., 2 * pairs:]
        if adjacent:
            a, b = f[..., 0:2 * pairs:2], f[..., 1:2 * pairs:2]
            y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = f[..., :pairs], f[..., pairs:2 * pairs]
            y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((y, rest), -1).to(x.dtype)

    return one(s["q"]), one(s["k"])


def _plain_prompt(s):
    """softmax(q . K^T / sqrt(D), masked) . V in fp32, sequence by sequence, in row chunks whose scores fit in 4 GB."""
    c = s["case"]
    hq, hk, d, w = c["q_heads"], c["kv_heads"], c["head_dim"], c["window"]
    out = torch.zeros_like(s["out"])
    begin = 0
    for n in _lens(c):
        q, k, v = (s[x][begin:begin + n].float().transpose(0, 1) for x in ("q", "k", "v"))
        q = q.reshape(hk, hq // hk, n, d)
        chunk = max(1, min(n, 2 ** 30 // (hq * max(n, 1))))
        for lo in range(0, n, chunk):
            hi = min(n, lo + chunk)
            first, last = (max(0, lo + 1 - w) if w else 0, hi) if c["causal"] else (0, n)
            z = q[:, :, lo:hi] @ k[:, None, first:last].transpose(2, 3) * d ** -0.5
            if c["causal"]:
                i = torch.arange(lo, hi, device=z.device)[:, None]
                j = torch.arange(first, last, device=z.device)
                unseen = j > i
                if w:
                    unseen = unseen | (j <= i - w)
                z = z.masked_fill(unseen, -math.inf)
            p = torch.exp(z - z.amax(-1, keepdim=True))
            o = (p @ v[:, None, first:last]) / p.sum(-1, keepdim=True)
            out[begin + lo:begin + hi] = o.reshape(hq, hi - lo, d).transpose(0, 1).to(out.dtype)
        begin += n
    return out


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _weights_64(s):
    """The weights' values, from their bytes."""
    codes, scales, ts = s["w"]
    m, k = s["case"]["m"], s["case"]["k"]
    dev = codes.device
    if ts is not None:
        e4 = []
        for byte in range(256):
            e, f = byte >> 3 & 15, byte & 7
            e4.append((math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)) * (-1 if byte & 128 else 1))
        e2 = [(b & 1) / 2 if b & 7 < 2 else math.ldexp(2 + (b & 1), (b >> 1 & 3) - 2) for b in range(8)]
        e2 = torch.tensor(e2 + [-x for x in e2], dtype=torch.float64, device=dev)
        w = torch.empty(m, k, dtype=torch.float64, device=dev)
        w[:, 0::2], w[:, 1::2] = e2[(codes % 16).long()], e2[(codes // 16).long()]
        return w * torch.tensor(e4, dtype=torch.float64, device=dev)[scales.long()].repeat_interleave(16, 1) * ts.double()
    value = []
    for code in range(64):
        e, f = code >> 3 & 3, code & 7
        value.append((f / 8 if e == 0 else math.ldexp(8 + f, e - 4)) * (-1 if code & 32 else 1))
    value = torch.tensor(value, dtype=torch.float64, device=dev)
    w = torch.empty(m, k, dtype=torch.float64, device=dev)
    for i in range(4):  # code 4 j + i begins at bit 6 i of bytes 3 j ..
        at = 6 * i // 8
        two = codes[:, at::3].int() + (codes[:, at + 1::3].int() * 256 if at < 2 else 0)
        w[:, i::4] = value[(two // 2 ** (6 * i % 8) % 64).long()]
    return w * torch.exp2(scales.double() - 127).repeat_interleave(128, 1)


def _exact_product(s):
    c = s["case"]
    y = torch.matmul(s["x"].double(), _weights_64(s).t())
    if s["bias"] is not None:
        y += s["bias"].double()
    if c["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif c["act"] == "gelu":
        y = y * torch.special.erfc(-y / math.sqrt(2)) / 2
    elif c["act"] == "gelu_tanh":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    elif c["act"] == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif c["act"] == "relu2":
        y = torch.where(y > 0, y ** 2, 0.0)
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_rotate(s):
    c = s["case"]
    half = c["rotary"] // 2
    outs = [s["q"].double().clone(), s["k"].double().clone()]
    for i, (f, axis) in enumerate(zip(_inv_freq(c), _axis(c))):
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=outs[0].device), s["positions"][axis].double() * f)
        at, by = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + half)
        for x in outs:
            z = torch.complex(x[..., at], x[..., by]) * turn[:, None]
            x[..., at], x[..., by] = z.real, z.imag
    return tuple(outs)


def _exact_prompt(s):
    c = s["case"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    group = c["q_heads"] // c["kv_heads"]
    end = 0
    for n in _lens(c):
        start, end = end, end + n
        for h in range(c["q_heads"]):
            q, k, v = s["q"][start:end, h].double(), s["k"][start:end, h // group].double(), s["v"][start:end, h // group].double()
            for lo in range(0, n, 2048):
                hi = min(n, lo + 2048)
                a, b = 0, n
                if c["causal"]:
                    a, b = (max(0, lo - c["window"] + 1) if c["window"] else 0), hi
                z = torch.einsum("id,jd->ij", q[lo:hi], k[a:b]) / math.sqrt(c["head_dim"])
                if c["causal"]:
                    gap = torch.arange(lo, hi, device=z.device)[:, None] - torch.arange(a, b, device=z.device)
                    z = torch.where((gap >= 0) & (gap < (c["window"] or n)), z, -math.inf)
                out[start + lo:start + hi, h] = torch.softmax(z, -1) @ v[a:b]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"product": _exact_product, "rotate": _exact_rotate, "prompt": _exact_prompt}[case["op"]](s)
