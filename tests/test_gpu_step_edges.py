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
