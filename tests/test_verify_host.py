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
