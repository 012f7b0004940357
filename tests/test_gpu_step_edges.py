"""The step operators where they are most easily wrong, on the GPU against the
float64 definitions (oracle/step.py, oracle/block.py): weights next to nothing and
batches of many parts in verification, value scales far apart and sums over many
keys in attention over 8 bits.  Tolerances as in test_gpu_step.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_q4_amd as q4
from oracle import block, step
from test_gpu_block import DEV, H16, H32, dev, near
from test_gpu_step import check_verify, drafts, i32, tol8
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


# ---- attention over 8 bits: value scales far apart -----------------------------
# (new tokens, keys), the rows of the tiles that take them, and (query, key/value) heads
KINDS = [(2, 2, 32, (4, 2)), (5, 300, 32, (8, 2)), (40, 130, 32, (4, 2)), (400, 400, 64, (32, 16)),
         (1100, 1100, 128, (32, 16))]


def far_apart(new, kv, heads, dim, half, seed, spots, rest, window=0, sinks=0, page=64):
    """One conversation whose values' scales are `rest`, but for those of keys `spots`
    (key: scale); what the call gives and what it should, rows sampled."""
    rng = np.random.default_rng([seed, new, dim])
    hq, hk = heads
    pages = (kv + page - 1) // page
    kc, vc = (rng.integers(-127, 128, (pages, 1, page, dim)).astype(np.int8) for _ in range(2))
    ks = (np.exp(0.3 * rng.standard_normal((pages, 1, page))) / 70).astype(np.float32)
    vs = np.full((pages, 1, page), rest, np.float32)
    for j, x in spots.items():
        vs[j // page, 0, j % page] = x
    table = np.arange(pages, dtype=np.int32)[None]
    q = rng.standard_normal((new, 1, dim)).astype(np.float16 if half else np.float32)
    wide = lambda a: dev(np.ascontiguousarray(np.repeat(a, hk, 1)))
    cache = q4.kv_cache8(*(wide(a) for a in (kc, vc, ks, vs)))
    tq = dev(np.ascontiguousarray(np.repeat(q, hq, 1)))
    scale = dim ** -0.5
    y = q4.attention(cache, tq, i32(0, new), i32(kv), dev(table), window, sinks, scale)
    assert torch.equal(y[:, :1].expand(-1, hq, -1).isnan(), y.isnan())
    rows = sorted({*range(0, new, max(1, new // 23)), *(j - (kv - new) + d for j in spots
                                                         for d in (-1, 0, 1))} & set(range(new)))
    numbers = step.numbers(kc, ks), step.numbers(vc, vs)
    want = [block.attend(*numbers, q[t:t + 1], [0, 1], [kv - new + t + 1], table, window, sinks,
                         scale) for t in rows]
    return y[rows, :1], *(np.concatenate([w[i] for w in want]) for i in range(3))


def near8(y, ref, absolute, score, keys, dim, half, rows):
    """As tol8's, and what binary16 parts lose of a weight: half of their least step, where
    the row's strongest key has 2^3 (2^-4 in passes of binary16 rows, one part), times the
    codes.  The strongest key's largest code is above 100: the row's largest element
    tells its share.  What does not fit binary16 is infinite."""
    lost = 2.0 ** (-21 if half and rows > 32 else -28) * keys * 1.3
    with np.errstate(invalid="ignore"):
        ref = np.where(np.abs(ref) > 65504 * 1.0001, np.sign(ref) * np.inf, ref) if half else ref
    fine = np.where(np.isfinite(ref), ref, 0.0)
    tol = tol8(fine, absolute, score, keys, dim, half, 2.0 ** -25 if half else 1e-37)
    near(y, ref, tol + lost * absolute.max(-1, keepdims=True))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,kv,rows,heads", KINDS)
def test_attention8_scales_that_a_row_does_not_see(new, kv, rows, heads, dim, half):
    """A later token's values far larger than the others': rows before it are as if it
    were not there, rows from it on as the definition has them."""
    c = q4.q4_0_kv_cache8(0, 0, 0, 0, 1, heads[1], 64, dim)
    assert q4.q4_0_select_attention8(c, heads[0], q4.F16 if half else q4.F32, new,
                                     (kv + 63) // 64, 1) == rows
    late = kv - 1 if new < 9 else kv - new + new * 2 // 3
    for i, (rest, much) in enumerate([(1e-3, 2.0 ** 25 * 1e-5), (2.0 ** -9, 1e30), (1e-4, 0.2),
                                      (1e-3, 1e36)] + ([] if half else [(1e-12, 1.0), (1e-30, 1e8)])):
        y, *want = far_apart(new, kv, heads, dim, half, i, {late: much}, rest)
        near8(y, *want, kv, dim, half, rows)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,kv,rows,heads", KINDS[1:])
def test_attention8_scales_out_of_the_window(new, kv, rows, heads, dim, half):
    """Far larger values that leave the window, and far smaller ones before them."""
    spots = {0: 1e30, 7: 1e30, kv - new - 3: 1e25, kv - new // 2: 2e-9, kv - 2: 3e-7}
    for window, sinks in ((20, 0), (64, 0), (20, 1)):
        y, *want = far_apart(new, kv, heads, dim, half, 31, spots, 2.0 ** -9, window, sinks)
        near8(y, *want, kv, dim, half, rows)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,kv,rows,heads", KINDS[1:] + [(1, 3000, 32, (4, 2))])
def test_attention8_scales_of_every_magnitude(new, kv, rows, heads, dim, half):
    """Scales of every key its own, over sixty powers of two (as far as binary16 rows
    carry: thirty), rising, falling and mixed."""
    rng = np.random.default_rng([41, dim])
    bits = np.linspace(-33 if half else -45, -3 if half else 15, kv)
    for order in (np.arange(kv), np.arange(kv)[::-1], rng.permutation(kv)):
        spots = dict(enumerate(np.float32(2.0) ** bits[order]))
        y, *want = far_apart(new, kv, heads, dim, half, 42, spots, 1.0)
        near8(y, *want, kv, dim, half, rows)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("new,rows", [(1, 32), (2, 32), (900, 64)])
@pytest.mark.parametrize("first", [False, True])
def test_attention8_large_values_of_little_weight(first, new, rows, half):
    """A key of weight 2^-30 with values 2^30 times the others' counts as much as they
    do; of weight 2^-60 it is nothing; the strong keys are in other tiles, before or
    after it."""
    dim, kv, page, heads = 64, 700 if new < 9 else 1500, 64, 16
    pages = (kv + page - 1) // page
    for down in (30, 60):
        kc = torch.zeros(pages, heads, page, dim, dtype=torch.int8, device=DEV)
        vc = torch.ones_like(kc)
        ks = torch.ones(pages, heads, page, device=DEV)
        vs = torch.full_like(ks, 2.0 ** -20)
        at = 3 if first else 300                       # seen by every row
        kc[at // page, :, at % page, 0] = -1
        vc[at // page, :, at % page] = 3
        vs[at // page, :, at % page] = 2.0 ** 10
        q = torch.zeros(new, heads, dim, dtype=torch.float16 if half else torch.float32, device=DEV)
        q[:, :, 0] = down
        c = q4.kv_cache8(kc, vc, ks, vs)
        assert q4.q4_0_select_attention8(c, heads, q4.F16 if half else q4.F32, new, pages, 1) == rows
        scale = float(np.float32(np.log(2.0)))
        y = q4.attention(c, q, i32(0, new), i32(kv), torch.arange(pages, device=DEV).int()[None],
                         scale=scale)
        w = np.exp(-scale * down)
        n = np.arange(kv - new, kv)
        want = ((n * 2.0 ** -20 + 3 * 2.0 ** 10 * w) / (n + w))[:, None, None]
        # scores of 60 at most, off by their roundings; a weight's (2^-12 in passes of binary16
        # rows); sums of kv
        steps = (60 * 8 + 2 * (kv + 18)) * H32 + (2 * H16 if half else 0.0) + 2.0 ** -22
        near(y, np.broadcast_to(want, y.shape),
             np.broadcast_to(want * steps + 2.0 ** -25 * half, y.shape))


# ---- attention over 8 bits: sums of many keys ------------------------------------
LONG = [  # conversations, new tokens of each, query and key/value heads, dim, keys
    (1, 320, 32, 8, 256, 131072), (1, 320, 32, 8, 128, 131072), (128, 1, 8, 8, 64, 131072),
    (48, 1, 32, 8, 256, 131072), (48, 3, 8, 8, 128, 131072), (128, 1, 8, 8, 128, 131072),
    (128, 1, 8, 8, 256, 131072)]


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("batch,new,hq,hk,dim,keys", LONG)
def test_attention8_sums_of_unsplit_contexts(batch, new, hq, hk, dim, keys, apart):
    """Calls that fill the device without cutting the key axis: a wave takes hundreds of
    tiles.  One strong key of weight 1 and value 1 among others of weight 2^-28.46 and value
    -1: 32 of them, what one product adds, are 1.45 steps of the sum beside it.
    apart: one key's value scale far below the others', so that rows have their own
    exponents."""
    page, gap = 256, 28.46
    pages = (keys + page - 1) // page
    kc = torch.zeros(pages, hk, page, dim, dtype=torch.int8, device=DEV)
    vc = torch.full_like(kc, -1)
    kc[0, :, 5, 0], vc[0, :, 5] = 127, 1
    one = torch.ones(pages, hk, page, device=DEV)
    vs = one.clone()
    if apart:
        vs[1, :, 7] = 2.0 ** -30                       # (a key less of 10^5)
    q = torch.zeros(batch * new, hq, dim, device=DEV)
    q[:, :, 0] = gap / np.log2(np.e) / 127
    c = q4.kv_cache8(kc, vc, one, vs)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).expand(batch, pages).contiguous()
    call = (hq, q4.F32, batch * new, pages, batch)
    assert q4.q4_0_select_attention8(c, *call) == 32
    assert q4.q4_0_attention8_workspace_size(c, *call) == 0
    start = torch.arange(0, batch * new + 1, new, dtype=torch.int32, device=DEV)
    y = q4.attention(c, q, start, torch.full((batch,), keys, dtype=torch.int32, device=DEV), table,
                     scale=1.0).double()
    weight = np.exp(-127 * float(q[0, 0, 0]))
    n = torch.arange(keys - new, keys, dtype=torch.float64, device=DEV).repeat(batch)
    want = ((1 - weight * (n - int(apart))) / (1 + weight * n))[:, None, None]
    # beside the strong key's, at most 96 tiles of 64 keys: four products (32 keys, two parts)
    # and a sum, each off by half a step of 1 at most; a weight, 2^-15.5 with the strong key's
    # at 2^13, is off by half a step of the least numbers, 2^-25; the gap's own rounding
    tol = (96 * 5 + 24 + 2 * gap) * H32 + weight * keys * (2.0 ** -9.5 + 2 * gap * H32)
    assert (y - want).abs().max() < tol < weight * keys / 4


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("gap", [3.0, 14.0, 18.0])
def test_attention8_faint_weights_of_a_split_context(gap, half):
    """One strong key and 40000 of weight e^-gap, one token, the key axis in parts: their
    sum has to survive, within bounds that a call which loses it misses."""
    n, dim, page, pages = 40001, 64, 256, 160
    kc, vc = (torch.zeros(pages, 1, page, dim, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, 1, page), x, device=DEV) for x in (8.0 / 127, 1.0 / 64))
    kc[0, 0, 0, 0] = 127
    vc[:, 0, :, 1] = 64
    vc[0, 0, 0, 1] = -64
    q = torch.zeros(1, 2, dim, dtype=torch.float16 if half else torch.float32, device=DEV)
    q[:, :, 0] = gap
    c = q4.kv_cache8(kc, vc, ks, vs)
    dtype = q4.F16 if half else q4.F32
    assert q4.q4_0_attention8_workspace_size(c, 2, dtype, 1, pages, 1) > 0
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    y = q4.attention(c, q, i32(0, 1), i32(n), table, scale=0.125)
    score = float(ks[0, 0, 0]) * 127 * 0.125 * gap
    faint = (n - 1) * np.exp(-score)
    want = (faint - 1.0) / (faint + 1.0)
    # beside the strong key's: the tiles of one wave (628 in all, over four waves at least of
    # eleven parts at least: 15), four products and a sum each; eight waves and 256 parts
    # joined; a score of `gap` and its weight, two parts
    tol = (15 * 5 + 8 + 256 + 24 + 4 * gap) * H32 + 2.0 ** -21 + H16 * abs(want) * half
    assert abs(want - -1.0) > 2 * tol                  # the result without any of them
    assert (y[0, :, 1].double() - want).abs().max() < tol
    assert (y[0, :, 2:] == 0).all()


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news,kvs,hq,hk", [((1, 3, 5), (700, 90, 333), 8, 2),
                                            ((150, 1, 90), (150, 40, 300), 32, 16),
                                            ((900, 260), (900, 300), 32, 16)])
def test_attention8_captured_calls_take_either_way(news, kvs, hq, hk, dim, half):
    """A captured call whose cache gets scales far apart between replays, in one
    conversation: that one's rows as the definition has them, the others' bits as they
    were; and back again."""
    page, rng = 32, np.random.default_rng([51, dim])
    widths = [(kv + page - 1) // page for kv in kvs]
    kc, vc = (rng.integers(-127, 128, (sum(widths), hk, page, dim)).astype(np.int8) for _ in range(2))
    ks, vs = ((np.exp(0.3 * rng.standard_normal((sum(widths), hk, page))) / 70).astype(np.float32)
              for _ in range(2))
    table = np.zeros((len(kvs), max(widths)), np.int32)
    for s, w in enumerate(widths):
        table[s, :w] = sum(widths[:s]) + np.arange(w)
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = rng.standard_normal((start[-1], hq, dim)).astype(np.float16 if half else np.float32)
    tvs, tq = dev(vs), dev(q)
    y, ws = torch.empty_like(tq), torch.empty(q4.WORKSPACE_MAX, dtype=torch.uint8, device=DEV)
    call = (q4.kv_cache8(dev(kc), dev(vc), dev(ks), tvs), tq, dev(start),
            dev(np.array(kvs, np.int32)), dev(table))
    usual = q4.attention(*call)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.attention(*call, y=y, ws=ws)
    far = vs.copy()
    far[table[0, widths[0] // 2], :, 7] *= np.float32(2.0 ** -20)
    far[table[0, widths[0] - 1], :, (kvs[0] - 1) % page] *= np.float32(2.0 ** (8 if half else 30))
    for k in range(4):
        tvs.copy_(dev(far if k % 2 else vs))
        y.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        n = start[1]
        assert torch.equal(y[n:], usual[n:])
        if k % 2 == 0:
            assert torch.equal(y, usual)
            continue
        assert torch.equal(y, q4.attention(*call))
        for t in {0, 1, n // 2, n - 2, n - 1} & set(range(n)):
            at = [np.ascontiguousarray(a[:, :1]) for a in (kc, vc, ks, far)]
            numbers = step.numbers(at[0], at[2]), step.numbers(at[1], at[3])
            want = block.attend(*numbers, q[t:t + 1, :1], [0, 1], [kvs[0] - n + t + 1], table[:1], 0,
                                0, dim ** -0.5)
            near8(y[t:t + 1, :1], *want, kvs[0], dim, half, 33 if max(news) > 64 else 32)
