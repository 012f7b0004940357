"""The block operators on the GPU where they can go wrong beyond their ordinary
sizes, against the float64 definitions (oracle/block.py).

Tolerances are those of test_gpu_block.py, whose helpers these tests use.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_q4_amd as q4
from oracle import block
from test_gpu_block import DEV, H16, append_tol, dev, near

pytestmark = pytest.mark.gpu


# ---- descriptors ------------------------------------------------------------
def test_calls_follow_replaced_tensors():
    """A norm weight and a cache that were given new memory, as Module.to gives
    it, are used as they are now."""
    rng = np.random.default_rng(1)
    n, heads, dim = 3, 2, 64
    rows = rng.standard_normal((n, heads * dim)).astype(np.float32)
    kc, vc = (torch.zeros(1, heads, 16, dim, dtype=torch.float16, device=DEV) for _ in range(2))
    weight = torch.nn.Parameter(torch.ones(dim, device=DEV), requires_grad=False)
    cache, rot = q4.kv_cache(kc, vc), q4.rotary(q_norm=weight, k_norm=weight, eps=1e-6)
    slots = torch.arange(n, device=DEV)
    first = kc
    wanted = (1 + rng.random(dim)).astype(np.float32)
    weight.data = dev(wanted)
    kc.data = torch.zeros(2, heads, 16, dim, dtype=torch.float16, device=DEV)
    vc.data = torch.zeros_like(kc)
    held = torch.full((dim,), 99.0, device=DEV)        # likely where the old weight lay
    q = q4.kv_append(cache, rot, dev(rows), dev(rows), dev(rows), None, slots)
    torch.cuda.synchronize()
    empty = np.zeros((2, heads, 16, dim))
    rq, rk, rv = block.append(empty, empty, rows, rows, rows, np.zeros(n), np.arange(n),
                              q_norm=wanted, k_norm=wanted)
    tol = append_tol(rq, rows.reshape(n, heads, dim), False, wanted, False)
    near(q, rq, tol)
    assert first is kc and held[0] == 99.0
    near(kc[0, :, :n].transpose(0, 1), rk[0, :, :n].transpose(1, 0, 2),
         append_tol(rk[0, :, :n].transpose(1, 0, 2), rows.reshape(n, heads, dim), True, wanted,
                    False))
    near(vc, rv, np.abs(rv) * H16)
