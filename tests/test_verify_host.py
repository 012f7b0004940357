"""Verification's kernels compiled for the CPU (tests/host: lanes as contexts that meet
at barriers and moves between lanes), against the float64 definition, with every
array and every row of logits ending at a page that may not be touched: what the
kernels read and write, for few parts and for many, without a GPU.
"""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import step

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CLANG = shutil.which("amdclang++") or "/opt/rocm/bin/amdclang++"


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """run(.., cus) -> (accepted, next): the call on a device of `cus` units."""
    if not os.path.exists(CLANG):
        pytest.skip("no clang++ to build the kernels for the CPU")
    lib = str(tmp_path_factory.mktemp("host") / "verify.so")
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-O2", "-fPIC", "-shared", "-w",
                    "-I", os.path.join(HERE, "host"), "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "gemm_q4_amd", "csrc"),
                    os.path.join(HERE, "host", "verify.cpp"), "-o", lib], check=True)
    entry = ctypes.CDLL(lib).host_verify

    def call(logits, tokens, start, uniform, drafted=None, heat=None, cus=256, marked=None):
        keep = [None if x is None else np.ascontiguousarray(x, t) for x, t in (
            (logits, logits.dtype), (drafted, logits.dtype), (marked, np.uint8), (tokens, np.int32),
            (start, np.int32), (heat, np.float32), (uniform, np.float32))]
        at = [None if x is None else ctypes.c_void_p(x.ctypes.data) for x in keep]
        batch, out = len(start) - 1, np.zeros(2 * (len(start) - 1), np.int32)
        i64 = ctypes.c_int64
        status = entry(at[0], at[1], at[2], ctypes.c_int(logits.dtype == np.float16),
                       i64(logits.shape[1]), at[3], at[4], i64(len(logits)), i64(batch), at[5],
                       at[6], ctypes.c_int(cus), ctypes.c_void_p(out.ctypes.data))
        assert status == 0, f"ended by signal {status & 127}, status {status >> 8}"
        return out[:batch], out[batch:]

    return call


def rows_of(rng, rows, vocab, half=False, modelled=True, spread=2.0):
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    n, dt = int(start[-1]), np.float16 if half else np.float32
    logits = (spread * rng.standard_normal((n, vocab))).astype(dt)
    drafted = (logits + 0.7 * rng.standard_normal((n, vocab))).astype(dt)
    source = (drafted if modelled else logits).astype(float)
    tokens = np.zeros(n, np.int32)
    tokens[1:] = (source + 0.7 * rng.gumbel(size=source.shape)).argmax(-1)[:-1]
    return logits, tokens, start, rng.random((n, 2)).astype(np.float32), drafted if modelled else None


def unjudged(start, n, heat):
    """Rows that judge no draft by draft logits: every conversation's last, all of one
    that takes the greatest, and those that no conversation holds."""
    none = np.ones(n, np.uint8)
    for s in range(len(start) - 1):
        if heat is None or heat[s] > 0:
            none[start[s]:start[s + 1] - 1] = 0
    return none


def agree(run, args, **kw):
    want = step.verify(*args[:5], kw.get("heat"))
    got = run(*args, **kw)
    assert got[0].tolist() == want[0].tolist() and got[1].tolist() == want[1].tolist()
    return got


# units of a device: of 256 a call of this size has few parts (four waves to each, the
# sums judging for themselves); of one it has many (a wave to each, a launch that judges)
@pytest.mark.parametrize("cus", [256, 1])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("modelled", [False, True])
def test_against_the_definition(run, modelled, half, cus):
    rng = np.random.default_rng([modelled, half])
    args = rows_of(rng, [1, 4, 0, 3, 9, 2], 4099, half, modelled)
    agree(run, args, cus=cus)
    agree(run, args, heat=np.array([1.0, 0.7, 1.0, 0.0, 1.5, 0.9], np.float32), cus=cus)


@pytest.mark.parametrize("cus", [256, 1])
def test_rows_that_judge_nothing_are_not_read(run, cus):
    rng = np.random.default_rng(5)
    args = list(rows_of(rng, [2, 4, 1, 3, 2], 2500))
    heat = np.array([1.0, 0.8, 1.0, 0.0, 0.6], np.float32)
    for h in (None, heat):
        agree(run, args, heat=h, cus=cus, marked=unjudged(args[2], 12, h))
    # leading and trailing rows that no conversation holds
    args[2] = args[2][1:-1]
    agree(run, args, heat=heat[1:-1], cus=cus, marked=unjudged(args[2], 12, heat[1:-1]))
    one = rows_of(rng, [1], 300)
    agree(run, one, cus=cus, marked=np.ones(1, np.uint8))


# ---- weights next to nothing ---------------------------------------------------
# A weight below 2^-980 of its row's largest counts as none: a logit 679.3 below it.
def faint_rows():
    """(logits, tokens, uniform, next): rows of two (a pick that is refused, then the
    row after it) of 5000 tokens, three parts."""
    def row(**at):
        x = np.full(5000, -np.inf, np.float32)
        for k, v in at.items():
            x[int(k[1:])] = v
        return x
    return [
        # the last part holds the draft, and a token whose weight beside the draft's is one and
        # beside the row's largest is none
        (row(t7=0.0, t4500=-450.0, t4600=-740.0), 4500, 1.0, 7),
        (row(t7=0.0, t4500=-600.0, t4600=-690.0), 4500, 2.0, 7),
        # .. and one whose weight is just one beside the row's largest
        (row(t7=0.0, t4500=-450.0, t4600=-679.0), 4500, 1.0, 4600),
        # the draft is the row's largest: nothing else has a weight, or just one token
        (row(t7=-680.0, t4500=0.0, t4600=-690.0), 4500, 0.5, 4500),
        (row(t7=-680.0, t4500=0.0, t4600=-679.0), 4500, 0.5, 4600),
        (row(t7=-679.0, t4500=0.0, t4600=-680.0), 4500, 1.0, 7),
        # the draft's part holds nothing else
        (row(t7=3.0, t4500=3.0), 4500, 1.0, 7),
        (row(t4500=3.0), 4500, 0.0, 4500),
        # the lowest token with a weight, in the part of the others and in one of its own
        (row(t7=-680.0, t8=-679.0, t9=0.0, t20=0.0), 9, 0.0, 8),
        (row(t7=-680.0, t3000=-679.0, t4500=0.0), 20, 0.0, 3000),
        (row(t7=-680.0, t3000=-690.0, t4500=0.0, t4999=-680.0), 20, 1.0, 4500),
    ]


@pytest.mark.parametrize("cus", [256, 1])
def test_faint_weights(run, cus):
    cases = faint_rows()
    n = 2 * len(cases)
    logits, tokens = np.zeros((n, 5000), np.float32), np.zeros(n, np.int32)
    uniform = np.full((n, 2), 2.0, np.float32)
    for i, (row, draft, u, _) in enumerate(cases):
        logits[2 * i], tokens[2 * i + 1], uniform[2 * i, 1] = row, draft, u
    start = np.arange(0, n + 1, 2, dtype=np.int32)
    accepted, following = run(logits, tokens, start, uniform, cus=cus)
    assert accepted.tolist() == [0] * len(cases)
    assert following.tolist() == [c[3] for c in cases]
    # with temperatures: logits as many times as far apart (a power of two: exactly)
    heat = np.full(len(cases), 0.25, np.float32)
    assert run(logits / 4, tokens, start, uniform, heat=heat, cus=cus)[1].tolist() == [
        c[3] for c in cases]
    # one row each, nothing refused: all of p
    rows, us = logits[::2], np.array([[0.0, x] for x in (0.0, 1.0)], np.float32)
    for u in us:
        _, t = run(rows, tokens[::2], np.arange(len(rows) + 1, dtype=np.int32),
                   np.tile(u, (len(rows), 1)), cus=cus)
        for x, got in zip(rows, t.tolist()):
            some = np.nonzero(x - x.max() >= -679.28)[0]
            assert got == (some[0] if u[1] == 0.0 else some[-1])


@pytest.mark.parametrize("cus", [256, 1])
def test_faint_weights_of_draft_models(run, cus):
    """Where the target has next to nothing, and where the draft has."""
    p, q = (np.full((2, 5000), -np.inf, np.float32) for _ in range(2))
    p[0, [5, 3000]] = 0.0
    q[0, 5] = 0.0
    p[0, 4000:4900] = -682.0                            # 900 of 2^-984: more than 2^-980 together
    run2 = lambda u: run(p, np.array([0, 5], np.int32), np.array([0, 2], np.int32),
                         np.array([[1.5, u], [0, 0]], np.float32), q, cus=cus)
    assert [int(run2(u)[1][0]) for u in (0.0, 0.5, 1.0)] == [3000] * 3
    p[0, 4800] = -679.0
    assert [int(run2(u)[1][0]) for u in (0.5, 1.0)] == [3000, 4800]
    q[0, 4800] = 0.0
    assert int(run2(1.0)[1][0]) == 3000
