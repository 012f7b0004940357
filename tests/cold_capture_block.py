"""Run in a fresh process by test_gpu_block.py: the first calls of the block
operators are made inside a graph capture; every replay is compared with the
eager calls made afterwards.  Prints one JSON line {name: equal}."""
from __future__ import annotations

import json
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_q4_amd as q4  # noqa: E402

DEV = "cuda:0"


def main() -> None:
    torch.manual_seed(1)
    n, hq, hk, dim, width = 3, 8, 2, 128, 40
    kc, vc = (torch.randn(n * width, hk, 16, dim, device=DEV).half() for _ in range(2))
    table = torch.randperm(n * width, device=DEV).int().view(n, width)
    lens = torch.tensor([600, 17, 301], dtype=torch.int32, device=DEV)
    start = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    pos = lens - 1
    at = table.long().gather(1, (pos // 16).long()[:, None])[:, 0]
    slots = at * 16 + pos % 16
    qkv = torch.randn(n, (hq + 2 * hk) * dim, device=DEV)
    w, inv = torch.ones(hq * dim, device=DEV), torch.rand(dim // 2, device=DEV)
    h = torch.randn(n, hq * dim, device=DEV)
    cache, rot = q4.kv_cache(kc, vc), q4.rotary(inv)
    q, y = torch.empty(n, hq, dim, device=DEV), torch.empty(n, hq, dim, device=DEV)
    y16 = torch.empty(n, hq, dim, device=DEV, dtype=torch.float16)
    q16 = torch.randn(n, hq, dim, device=DEV).half()
    oh, oy = torch.empty_like(h), torch.empty_like(h)
    ws = torch.empty(q4.WORKSPACE_MAX, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()

    def calls():
        parts = qkv.split([hq * dim, hk * dim, hk * dim], dim=1)
        q4.kv_append(cache, rot, *parts, pos, slots, q_out=q)
        q4.attention(cache, q, start, lens, table, y=y, ws=ws)
        q4.attention(cache, q16, start, lens, table, window=200, sinks=4, y=y16, ws=ws)
        q4.residual_norm(h, y.flatten(1), w, w, h_out=oh, y=oy)

    outs = {"q": q, "y": y, "y16": y16, "h": oh, "x": oy, "k": kc, "v": vc}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    replays = []
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        replays.append({k: t.clone() for k, t in outs.items()})
    for name in ("q", "y", "y16", "h", "x"):
        outs[name].zero_()
    calls()
    torch.cuda.synchronize()
    print(json.dumps({k: all(torch.equal(r[k], t) for r in replays) for k, t in outs.items()}))


if __name__ == "__main__":
    main()
