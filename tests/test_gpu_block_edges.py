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
from test_gpu_block import DEV, H16, H32, append_tol, attention_tol, dev, near

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


# ---- attention: scores of any size -------------------------------------------
def plain(lengths, dim, seed, pages=20):
    """Caches of `pages` pages of 16 keys and 2 heads, the lengths' tables."""
    rng = np.random.default_rng(seed)
    kc, vc = (rng.standard_normal((pages, 2, 16, dim)).astype(np.float16) for _ in range(2))
    width = max((kv + 15) // 16 for _, kv in lengths)
    table = rng.integers(0, pages, (len(lengths), width)).astype(np.int32)
    start = np.concatenate([[0], np.cumsum([new for new, _ in lengths])]).astype(np.int32)
    return rng, kc, vc, start, np.array([kv for _, kv in lengths], np.int32), table


def attend(kc, vc, q, start, lens, table, window=0, sinks=0, scale=1.0):
    tk, tv = dev(kc), dev(vc)
    y = q4.attention(q4.kv_cache(tk, tv), dev(q), dev(start), dev(lens), dev(table), window, sinks,
                     scale)
    torch.cuda.synchronize()
    return y


LENGTHS = [[(1, 90), (1, 7)], [(40, 90)], [(300, 300)]]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("half,magnitude,scale,zero_keys", [
    (False, 1e-25, 1e-21, False), (False, 4e-45, 0.0625, False), (False, 1.0, 1e-45, False),
    (False, 1e30, 1e30, True), (False, 1.0, 3.2e38, True),
    (True, 1.0, 1e-45, False), (True, 1.0, 3.2e38, True), (True, 60000.0, 3.4e38, True)])
def test_attention_factors_beyond_float32(half, magnitude, scale, zero_keys, lengths):
    """The scale and the query's magnitude leave float32 together: below it every
    visible key weighs the same; above it equal scores still do."""
    rng, kc, vc, start, lens, table = plain(lengths, 64, 3)
    if zero_keys:
        kc[:] = 0
    q = rng.standard_normal((start[-1], 4, 64)) * magnitude
    q = np.clip(q, -65504, 65504).astype(np.float16) if half else q.astype(np.float32)
    y = attend(kc, vc, q, start, lens, table, scale=scale)
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, 0, 0, float(np.float32(scale)))
    assert score.max() < 1e-30
    near(y, ref, attention_tol(ref, absolute, score, 300, 64, half))


@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 2)])
@pytest.mark.parametrize("lengths", LENGTHS + [[(1, 1500)], [(70, 900), (1, 1300)]])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("power", [10, 20, 22, 23, 24, 26, 28, 31, 60, 100])
def test_attention_scores_of_any_size(power, half, lengths, window, sinks):
    """Keys at whole levels, two of the cache's to a level, and queries that make
    a step of one level a score of 2^power: a row's result is the mean of the
    values at the highest level it sees.  Every score is exact, so no rounding
    but that of the weights' sum and of the result is left; the other levels'
    weights are at most exp(-2^10)."""
    rng, kc, vc, start, lens, table = plain(lengths, 64, power, pages=100)
    level = rng.permutation(np.repeat(np.arange(800), 2)).reshape(100, 16) - 400.0
    kc[:] = 0
    kc[:, 0, :, 3], kc[:, 1, :, 5] = level, -level
    table = np.stack([rng.permutation(100)[:table.shape[1]] for _ in lengths]).astype(np.int32)
    q = np.zeros((start[-1], 4, 64), np.float16 if half else np.float32)
    shift = min(power, 14) if half else power
    q[:, :2, 3] = q[:, 2:, 5] = 2.0 ** shift
    scale = 2.0 ** (power - shift)
    y = attend(kc, vc, q, start, lens, table, window, sinks, scale)
    ref, absolute, _ = block.attend(kc, vc, q, start, lens, table, window, sinks, scale)
    near(y, ref, np.abs(ref) * (H16 if half else H32) + absolute * 8 * H32 + 2.0 ** -25)
