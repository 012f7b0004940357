"""The step operators where they are most easily wrong, on the GPU against the
float64 definitions (oracle/step.py, oracle/block.py): weights next to nothing and
batches of many parts in verification, value scales far apart and sums over many
keys in attention over 8 bits.  Tolerances as in test_gpu_step.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_q4_amd as q4
from oracle import step
from test_gpu_block import DEV, dev
from test_gpu_step import check_verify, drafts
from test_verify_host import faint_rows

pytestmark = pytest.mark.gpu


# ---- verification ------------------------------------------------------------
@pytest.mark.parametrize("copies", [1, 40])
def test_verify_faint_weights(copies):
    """A token is never drawn from a part whose weights are none beside the row's
    largest, whatever the number; few rows and many (four waves to a part, and one)."""
    cases = faint_rows() * copies
    n = 2 * len(cases)
    logits, tokens = np.zeros((n, 5000), np.float32), np.zeros(n, np.int32)
    uniform = np.full((n, 2), 2.0, np.float32)
    for i, (row, draft, u, _) in enumerate(cases):
        logits[2 * i], tokens[2 * i + 1], uniform[2 * i, 1] = row, draft, u
    call = (dev(tokens), torch.arange(0, n + 1, 2, dtype=torch.int32, device=DEV), dev(uniform))
    accepted, following = q4.verify(dev(logits), *call)
    assert accepted.tolist() == [0] * len(cases)
    assert following.tolist() == [c[3] for c in cases]
    heat = torch.full((len(cases),), 0.25, device=DEV)
    assert q4.verify(dev(logits / 4), *call, temperature=heat)[1].tolist() == [c[3] for c in cases]


@pytest.mark.parametrize("half", [False, True])
def test_verify_draft_models_of_many_parts(half):
    """More parts of conversations than run at once (two to a unit): the judgement is a
    launch of its own.  Drawn, picked, empty and no distribution among them."""
    rng = np.random.default_rng([21, half])
    rows = [4, 1, 0, 6, 3, 2, 5, 1] * 5
    vocab = 33001
    units = torch.cuda.get_device_properties(DEV).multi_processor_count
    assert len(rows) * ((vocab + 2047) // 2048) > 2 * units
    logits, tokens, start, uniform, drafted = drafts(rng, rows, vocab, half, True)
    heat = np.tile(np.array([1.0, 0.8, 0.0, 1.2, 0.6, 0.9, 0.0], np.float32), 6)[:len(rows)]
    a, t = check_verify(logits, tokens, start, uniform, drafted, heat, pad=5)
    assert 0 < a.sum() < sum(rows) - len(rows) and (t == -1).sum() == 5
    check_verify(logits, tokens, start, uniform, drafted)
    for s in range(0, len(rows), 3):
        if rows[s]:
            x = (logits, drafted)[s % 2]
            x[start[s], rng.integers(0, vocab)] = [np.nan, np.inf][s % 4 // 2]
    logits[start[11]] = -np.inf
    logits[start[12], 100:] = -np.inf
    _, t = check_verify(logits, tokens, start, uniform, drafted, heat)
    assert (t == -1).sum() > 10


def test_verify_draft_models_of_many_parts_and_long_rows():
    """The same with vocabularies past 262144 tokens."""
    rng = np.random.default_rng(22)
    rows, vocab = [2, 3, 1, 2], 300007
    assert len(rows) * ((vocab + 2047) // 2048) > 512
    for heat in (1.0, 3.0, 0.0):
        logits, tokens, start, uniform, drafted = drafts(rng, rows, vocab, False, True)
        logits[:, 290000:] += 1.5
        check_verify(logits, tokens, start, uniform, drafted, np.full(4, heat, np.float32))


@pytest.mark.parametrize("modelled", [False, True])
def test_verify_the_largest_batch(modelled):
    """65536 conversations, most without rows: past one dimension of a grid's."""
    rng = np.random.default_rng([23, modelled])
    rows = np.zeros(65536, int)
    rows[rng.permutation(65536)[:9000]] = rng.integers(1, 4, 9000)
    rows[[0, 32767, 32768, 40000, 65535]] = 3
    logits, tokens, start, uniform, drafted = drafts(rng, rows, 23, False, modelled)
    check_verify(logits, tokens, start, uniform, drafted)
