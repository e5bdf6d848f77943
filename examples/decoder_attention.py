"""The attention half of a decoder layer on the library: QKV product with its
bias, rotary positions, KV-cache append, attention (over the prompt itself, or
over the pages), O product onto the residual stream.

    python examples/decoder_attention.py [--format e4m3|nvfp4]

Random NVFP4 weights of the 9B-class layer (32 query and 8 KV heads of 128)
serve three sequences the way a server does: a prefill in two chunks (the first
attends to the prompt's own K and V, the second to the pages), decode steps
replayed from one CUDA graph, and a speculative verify of a token tree.  Each
stage prints how far its attention output is from the fp64 definition on the
values that it attends to.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_nvfp4_gb300 as g  # noqa: E402

HIDDEN, HQ, HK, D = 4096, 32, 8, 128
PAGE = 64


class PagedSequences:
    """Page tables and lengths of a batch of sequences over one pool."""

    def __init__(self, n_seqs: int, max_tokens: int, fmt: int, device):
        self.width = -(-max_tokens // PAGE)
        self.cache = g.KVCache.empty(n_seqs * self.width, PAGE, HK, D, fmt, device)
        pages = torch.randperm(n_seqs * self.width, dtype=torch.int32)
        self.table = pages.view(n_seqs, self.width).to(device)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device=device)

    def next(self, new: int) -> tuple[torch.Tensor, torch.Tensor]:
        """Positions and slots of the `new` tokens that follow each sequence's last one, [n_seqs * new]."""
        at = self.lens[:, None].long() + torch.arange(new, device=self.lens.device)
        return at.flatten(), (self.table.long().gather(1, at // PAGE) * PAGE + at % PAGE).flatten()


class Attention:
    """x -> O . attention(QKV . x), for any number of tokens of each sequence."""

    def __init__(self, seed: int, device):
        gen = torch.Generator(device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device=device, generator=gen) * 0.02  # noqa: E731
        self.qkv = g.nvfp4_quantize(rand((HQ + 2 * HK) * D, HIDDEN))
        self.qkv_bias = rand((HQ + 2 * HK) * D).to(torch.bfloat16)
        self.o = g.nvfp4_quantize(rand(HIDDEN, HQ * D))
        self.rope = g.RopeTable.make([1e6 ** (-2 * i / D) for i in range(D // 2)], device=device)
        self.workspaces: dict = {}

    def workspace(self, key, need: int, device) -> torch.Tensor:
        if need > self.workspaces.get(key, torch.empty(0)).numel():
            self.workspaces[key] = torch.zeros(need, dtype=torch.uint8, device=device)
        return self.workspaces[key]

    def product(self, x, w, **epilogue):
        n = x.shape[0]  # few tokens: a workspace of their own, with counters that other calls must not touch
        ws = self.workspace((w.M, n <= 16), g.nvfp4_workspace_bytes(g.NVFP4_OP_GEMM_PREFILL, n, w.M, w.K), x.device)
        return g.nvfp4_gemm_epilogue(x, w, out_dtype=torch.bfloat16, workspace=ws, **epilogue)

    def __call__(self, x, seqs: PagedSequences, new: int, positions, slots, lens, tree=None, prompt=None):
        """x [n_seqs * new, HIDDEN], the residual stream; lens counts the new tokens; prompt: the offsets of sequences
        that begin with these tokens.  Returns (y, (q, k, v) after the rotation, attention output)."""
        qkv = self.product(x, self.qkv, bias=self.qkv_bias).unflatten(1, (HQ + 2 * HK, D))
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:]
        g.nvfp4_rope(q, k, positions, self.rope, out=(q, k))
        ws = self.workspace("attention", g.nvfp4_paged_attention_workspace_bytes(seqs.cache, q, len(lens), new), x.device)
        g.nvfp4_kv_append(seqs.cache, k, v, slots, workspace=ws)
        if prompt is not None:
            a = g.nvfp4_prompt_attention(q, k, v, prompt, workspace=ws)
        else:
            a = g.nvfp4_paged_attention(q, seqs.cache, seqs.table, lens, max_q_len=new, tree=tree, workspace=ws)
        return self.product(a.flatten(1), self.o, residual=x), (q, k, v), a


def error(seqs, qkv, a, new, lens, tree=None, prompt=False) -> float:
    """Relative distance of attention outputs from softmax(q K^T / sqrt(D)) V in fp64, on the cached values or (prompt)
    on the new tokens' own."""
    off = total = 0.0
    for b, n in enumerate(lens.tolist()):
        at = torch.arange(n, device=a.device)
        rows = slice(b * new, (b + 1) * new)
        if prompt:
            kv = (t[rows] for t in qkv[1:])
        else:
            kv = g.nvfp4_kv_read(seqs.cache, seqs.table[b].long()[at // PAGE] * PAGE + at % PAGE)
        k, v = (t.double().repeat_interleave(HQ // HK, 1).transpose(0, 1) for t in kv)
        past, i = n - new, torch.arange(new, device=a.device)[:, None]
        see = at <= past + i
        if tree is not None:
            see = (at < past) | ((tree[rows, None] >> (at - past).clamp(min=0)) & 1 == 1)
        z = qkv[0][rows].double().transpose(0, 1) @ k.transpose(1, 2) / D ** 0.5
        want = (torch.softmax(z.masked_fill(~see, float("-inf")), -1) @ v).transpose(0, 1)
        off += float((a[rows].double() - want).square().sum())
        total += float(want.square().sum())
    return (off / total) ** 0.5


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--format", choices=("e4m3", "nvfp4"), default="e4m3")
    args = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    gen = torch.Generator(dev).manual_seed(1)
    rand = lambda n: torch.randn(n, HIDDEN, device=dev, generator=gen).to(torch.bfloat16)  # noqa: E731
    n_seqs = 3
    seqs = PagedSequences(n_seqs, 600, g.NVFP4_KV_E4M3 if args.format == "e4m3" else g.NVFP4_KV_NVFP4, dev)
    layer, errors = Attention(0, dev), {}

    # prefill: 400 tokens of each sequence in two chunks
    for chunk in (250, 150):
        positions, slots = seqs.next(chunk)
        first = chunk == 250
        prompt = torch.arange(n_seqs + 1, dtype=torch.int32, device=dev) * chunk if first else None
        seqs.lens += chunk
        _, qkv, a = layer(rand(n_seqs * chunk), seqs, chunk, positions, slots, seqs.lens, prompt=prompt)
        errors[f"prefill chunk of {chunk}"] = error(seqs, qkv, a, chunk, seqs.lens, prompt=first)

    # decode: one captured step, replayed; lengths, positions and slots are device buffers that change between replays
    x, (positions, slots) = rand(n_seqs), seqs.next(1)
    seqs.lens += 1
    layer(x, seqs, 1, positions, slots, seqs.lens)  # warm-up: workspaces are there before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, qkv, a = layer(x, seqs, 1, positions, slots, seqs.lens)
    for _ in range(8):
        x.copy_(rand(n_seqs))
        for buffer, value in zip((positions, slots), seqs.next(1)):
            buffer.copy_(value)
        seqs.lens += 1
        graph.replay()
        errors["decode"] = max(errors.get("decode", 0.0), error(seqs, qkv, a, 1, seqs.lens))

    # verify: the last token and a tree of drafts: 1 and 2 follow 0, 3 follows 1, 4 follows 2
    words, depth = [0b00001, 0b00011, 0b00101, 0b01011, 0b10101], [0, 1, 1, 2, 2]
    tree = torch.tensor(words * n_seqs, device=dev)
    _, slots = seqs.next(5)
    positions = (seqs.lens[:, None].long() + torch.tensor(depth, device=dev)).flatten()
    lens = seqs.lens + 5
    _, qkv, a = layer(rand(5 * n_seqs), seqs, 5, positions, slots, lens, tree=tree)
    errors["verify of a tree of 5"] = error(seqs, qkv, a, 5, lens, tree)

    assert g.nvfp4_device_status(layer.workspaces["attention"]) == (g.NVFP4_OK, 0)
    for stage, e in errors.items():
        print(f"{stage}: attention is {e:.2e} from its definition (relative)")
    return errors


if __name__ == "__main__":
    main()
