"""A decoder block served from a paged cache, end to end on the library's calls.

Three conversations with prompts of different lengths are read in one ragged
pass, then drawn token by token: each decode step is one HIP graph, captured
once and replayed as the conversations grow, since positions, lengths and the
page table are device tensors.  A block runs

    q, k, v   = products of the normed input          matmul_grouped
    q, cache <- norms and rotation, k and v appended  kv_append
    y         = attention over the cache              attention
    h, x      = residual step after O, norm before FFN  matmul, residual_norm
    h, x      = residual step after the FFN           matmul_grouped, matmul, residual_norm

with random Q4_0 weights.  Run it as  python examples/decoder_block.py  (it
checks the decoded steps against one pass over the whole text).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_q4_amd as q4  # noqa: E402
import synth  # noqa: E402

DEV = "cuda:0"


class Block:
    """One block: hidden width, query and key/value heads of `dim`, FFN width."""

    def __init__(self, width, heads, kv_heads, dim, ffn, seed=0, window=0, sinks=0):
        self.width, self.heads, self.kv_heads, self.dim, self.ffn = width, heads, kv_heads, dim, ffn
        self.window, self.sinks = window, sinks
        shapes = {"q": (heads * dim, width), "k": (kv_heads * dim, width),
                  "v": (kv_heads * dim, width), "o": (width, heads * dim), "gate": (ffn, width),
                  "up": (ffn, width), "down": (width, ffn)}
        self.w = {}
        for i, (name, (out, in_)) in enumerate(shapes.items()):
            blocks = torch.from_numpy(synth.make_blocks(out, in_, seed=seed + i).reshape(-1)).to(DEV)
            self.w[name] = (q4.repacked(blocks, out, in_), out, in_)
        g = torch.Generator(device=DEV).manual_seed(seed)
        one = lambda n: 1.0 + 0.1 * torch.randn(n, device=DEV, generator=g)
        self.norms = {n: one(width) for n in ("after_attention", "before_ffn", "after_ffn", "next")}
        inv = 10000.0 ** (-torch.arange(0, dim, 2, device=DEV, dtype=torch.float64) / dim)
        self.rot = q4.rotary(inv.float(), q_norm=one(dim), k_norm=one(dim))

    def products(self, names, x):
        """The named products of x's rows, one grouped call."""
        n = x.shape[0]
        ys = [torch.empty(n, self.w[m][1], device=DEV) for m in names]
        q4.matmul_grouped([(self.w[m][0], x, y, self.w[m][1], self.w[m][2])
                           for m, y in zip(names, ys)], q4.dtype_code(x), n)
        return ys

    def __call__(self, h, x, cache, batch):
        """(h, x) of the next block from the residual h and its normed x."""
        q, k, v = self.products(("q", "k", "v"), x)
        q = q4.kv_append(cache, self.rot, q, k, v, batch["positions"], batch["slots"])
        y = q4.attention(cache, q, batch["q_start"], batch["kv_len"], batch["table"],
                         window=self.window, sinks=self.sinks)
        o, = self.products(("o",), y.flatten(1))
        h, x = q4.residual_norm(h, o, self.norms["before_ffn"], post=self.norms["after_attention"])
        gate, up = self.products(("gate", "up"), x)
        d, = self.products(("down",), torch.nn.functional.silu(gate) * up)
        return q4.residual_norm(h, d, self.norms["next"], post=self.norms["after_ffn"])


def new_cache(block, pages, page_size):
    shape = (pages, block.kv_heads, page_size, block.dim)
    return torch.zeros(shape, dtype=torch.float16, device=DEV), torch.zeros(
        shape, dtype=torch.float16, device=DEV)


def place(batch, new, lengths, page_size):
    """Fill the batch's device tensors: `new` tokens of each conversation, the
    last of its `lengths` positions (host lists; a scheduler's work)."""
    owner = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(new, lengths)])
    start = torch.tensor([0] + new).cumsum(0)
    table = batch["table"].cpu().long()
    batch["q_start"].copy_(start.int())
    batch["kv_len"].copy_(torch.tensor(lengths, dtype=torch.int32))
    batch["positions"].copy_(pos.int())
    batch["slots"].copy_(table[owner, pos // page_size] * page_size + pos % page_size)


def new_batch(tokens, table):
    i32 = dict(dtype=torch.int32, device=DEV)
    return {"q_start": torch.zeros(table.shape[0] + 1, **i32),
            "kv_len": torch.zeros(table.shape[0], **i32),
            "positions": torch.zeros(tokens, **i32), "table": table,
            "slots": torch.zeros(tokens, dtype=torch.int64, device=DEV)}


def run(prompts=(37, 5, 70), steps=12, page_size=16, seed=0, width=256, heads=4, kv_heads=2,
        dim=64, ffn=512, window=32, sinks=2):
    """(decoded, whole): the block's x rows of every conversation's drawn tokens,
    decoded step by step after a prefill pass, and from one pass over all of
    it."""
    block = Block(width, heads, kv_heads, dim, ffn, seed, window, sinks)
    g = torch.Generator(device=DEV).manual_seed(seed + 100)
    total = [p + steps for p in prompts]
    text = [torch.randn(n, width, device=DEV, generator=g) for n in total]
    per = (max(total) + page_size - 1) // page_size
    table = torch.randperm(per * len(prompts), device=DEV, generator=g).int().view(len(prompts), per)
    norm = block.norms["next"]

    def first(rows):
        return q4.residual_norm(rows, pre=norm)[1]

    # one pass over everything
    cache = new_cache(block, per * len(prompts), page_size)
    batch = new_batch(sum(total), table)
    place(batch, list(total), list(total), page_size)
    rows = torch.cat(text)
    _, x = block(rows, first(rows), q4.kv_cache(*cache), batch)
    whole = torch.stack([part[-steps:] for part in x.split(list(total))], dim=1)

    # the prompts in one pass, then a captured decode step
    cache = new_cache(block, per * len(prompts), page_size)
    batch = new_batch(sum(prompts), table)
    place(batch, list(prompts), list(prompts), page_size)
    rows = torch.cat([t[:p] for t, p in zip(text, prompts)])
    block(rows, first(rows), q4.kv_cache(*cache), batch)

    n = len(prompts)
    batch, rows = new_batch(n, table), torch.zeros(n, width, device=DEV)
    descriptor = q4.kv_cache(*cache)
    place(batch, [1] * n, [p + 1 for p in prompts], page_size)
    rows.copy_(torch.stack([t[p] for t, p in zip(text, prompts)]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                 # once eagerly: it loads the kernels' code
        block(rows, first(rows), descriptor, batch)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, x = block(rows, first(rows), descriptor, batch)
    decoded = []
    for i in range(steps):
        place(batch, [1] * n, [p + 1 + i for p in prompts], page_size)
        rows.copy_(torch.stack([t[p + i] for t, p in zip(text, prompts)]))
        graph.replay()
        decoded.append(x.clone())
    torch.cuda.synchronize()
    return torch.stack(decoded), whole


if __name__ == "__main__":
    got, want = run()
    off = float((got - want).norm() / want.norm())
    print(f"{got.shape[0]} decode steps of {got.shape[1]} conversations against one pass: "
          f"relative difference {off:.1e}")
    # decode rounds activations to 22 bits, a pass of more rows to binary16
    sys.exit(0 if off < 5e-3 else 1)
