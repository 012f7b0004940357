"""Run in a fresh process by test_gpu_step.py: the first calls of a drafted step's
operators are made inside a graph capture; every replay is compared with the
eager calls made afterwards.  Prints one JSON line {name: equal}."""
from __future__ import annotations

import json
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

from test_gpu_step import new_ws, step_calls  # noqa: E402


def main() -> None:
    call, out = step_calls()       # (repacks the table, no other call of the library)
    ws = new_ws()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws)
    replays = []
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        replays.append({k: t.clone() for k, t in out.items()})
        ws.fill_(255)
    for t in out.values():
        t.zero_()
    call(ws)
    torch.cuda.synchronize()
    print(json.dumps({k: all(torch.equal(r[k], t) for r in replays) for k, t in out.items()}))


if __name__ == "__main__":
    main()
