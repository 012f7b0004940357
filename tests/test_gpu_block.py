"""The operators between a block's products on the GPU against their float64
definitions (oracle/block.py): cache append with norms and rotation, attention
over the paged cache, residual norms.

Tolerances follow from the roundings a result passes through, in units of half
a step (binary16 2^-11, float32 2^-24), with worst-case sums:
- a float32 sum of N products is off by at most (N + 1) 2^-24 times the sum of
  their absolute values;
- float32 attention takes q and the weights as two binary16 parts, off by
  2^-22; binary16 attention rounds each weight once (2^-11);
- a score that is off by d changes a weight, its share of the sum included, by
  at most 2 d (1 % added for the second order).
"""
from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

import gemm_q4_amd as q4
from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H16, H32 = 2.0 ** -11, 2.0 ** -24


def dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def near(got, want, tol):
    """Every value within tol, infinities and NaN in the same places."""
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got)
    want, tol = np.asarray(want), np.broadcast_to(tol, np.shape(want))
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    off = np.abs(got[fine] - want[fine])
    assert (off <= tol[fine]).all(), f"off by up to {off.max()}"


# ---- append -----------------------------------------------------------------
def append_tol(ref, rows, half, weight=None, rotated=True):
    """Half steps of the output's type on the value, and float32 roundings of
    the norm and the rotation, which scale with the row's largest element."""
    top = np.abs(rows).max(axis=-1, keepdims=True)
    steps = (ref.shape[-1] + 8 if weight is not None else 0) + (8 if rotated else 0)
    return np.abs(ref) * (H16 if half else H32) + steps * H32 * 1.5 * top + (2.0 ** -25 if half else 1e-37)


CASES = [  # n, heads, kv_heads, dim, rot_dim, page, interleaved, norm, x half, q_out half, first
    (1, 4, 2, 128, 128, 16, False, True, False, True, 0),
    (1, 1, 1, 64, 64, 16, True, False, True, True, 7),
    (5, 3, 1, 64, 32, 16, False, True, True, False, 100),
    (33, 8, 8, 128, 64, 32, True, True, False, False, 400000),
    (17, 6, 2, 256, 256, 16, False, False, True, True, 65535),
    (9, 2, 2, 96, 96, 64, False, True, False, True, 3),
    (7, 5, 1, 8, 8, 16, True, True, False, False, 1),
    (3, 2, 1, 512, 128, 16, False, True, True, True, 2000000),
    (40, 7, 1, 72, 24, 16, False, False, False, False, 12),
    (300, 32, 8, 128, 128, 16, False, True, False, True, 5000),
    (4, 2, 1, 64, 0, 16, False, True, False, True, 0),
]


@pytest.mark.parametrize("case", CASES)
def test_append(case):
    n, hq, hk, dim, rot_dim, page, inter, norm, xh, qh, first = case
    rng = np.random.default_rng(list(case[:6]))
    pages = (n + page - 1) // page + 2
    xt = np.float16 if xh else np.float32
    # q, k, v as slices of one product's rows, with columns of others between them
    wide = rng.standard_normal((n, (hq + 2 * hk) * dim + 16)).astype(xt)
    q, k, v = (wide[:, a:b] for a, b in ((0, hq * dim), (hq * dim, (hq + hk) * dim),
                                         ((hq + hk) * dim, (hq + 2 * hk) * dim)))
    kc, vc = (rng.standard_normal((pages, hk, page, dim)).astype(np.float16) for _ in range(2))
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    if n > 4:
        slots[1], slots[3] = -1, pages * page            # two padded tokens
    pos = (first + np.arange(n)).astype(np.int32)
    inv = (10000.0 ** (-np.arange(0, rot_dim, 2) / max(rot_dim, 1))).astype(np.float32)
    qw, kw = ((1 + 0.1 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2))
    amp, off = (1.0, 0.0) if n % 2 else (1.25, 0.5)
    args = dict(inv_freq=inv, interleaved=inter, amplitude=amp, eps=1e-5, offset=off,
                q_norm=qw if norm else None, k_norm=kw if norm else None)
    rq, rk, rv = block.append(kc, vc, q, k, v, pos, slots, **args)

    w, tkc, tvc = dev(wide), dev(kc), dev(vc)
    d = dict(inv_freq=dev(inv) if rot_dim else None, interleaved=inter, amplitude=amp, eps=1e-5,
             weight_offset=off, q_norm=dev(qw) if norm else None, k_norm=dev(kw) if norm else None)
    out = torch.full((n, hq, dim), float("nan"), dtype=torch.float16 if qh else torch.float32,
                     device=DEV)
    got = q4.kv_append(q4.kv_cache(tkc, tvc), q4.rotary(**d), w[:, :hq * dim],
                       w[:, hq * dim:(hq + hk) * dim], w[:, (hq + hk) * dim:(hq + 2 * hk) * dim],
                       dev(pos), dev(slots), q_out=out)
    torch.cuda.synchronize()
    assert got is out
    near(out, rq, append_tol(rq, rq, qh, qw if norm else None, rot_dim > 0))
    assert torch.equal(tvc, dev(rv.astype(np.float16)))      # one rounding of the value itself
    near(tkc, rk, append_tol(rk, rk, True, kw if norm else None, rot_dim > 0))
    written = np.zeros((pages, hk, page, dim), bool)
    for s in slots[(slots >= 0) & (slots < pages * page)]:
        written[s // page, :, s % page] = True
    assert np.array_equal(tkc.cpu().numpy()[~written], kc[~written])


def test_append_without_q_and_without_rotation():
    k = torch.randn(3, 2, 64, device=DEV)
    kc, vc = (torch.zeros(1, 2, 16, 64, dtype=torch.float16, device=DEV) for _ in range(2))
    slots = torch.tensor([2, 0, 15], device=DEV)
    assert q4.kv_append(q4.kv_cache(kc, vc), None, None, k, 2 * k, None, slots) is None
    assert torch.equal(kc[0][:, slots].transpose(0, 1), k.half())
    assert torch.equal(vc[0][:, slots].transpose(0, 1), (2 * k).half())
    assert kc[0, :, 1].abs().sum() == 0


def test_append_non_finite_values_stay_in_their_row():
    k = torch.randn(3, 2, 64, device=DEV)
    k[1, 0, 5], k[2, 1, 7] = float("inf"), float("nan")
    kc, vc = (torch.zeros(1, 2, 16, 64, dtype=torch.float16, device=DEV) for _ in range(2))
    slots = torch.arange(3, device=DEV)
    pos = slots.int()
    inv = torch.ones(32, device=DEV)
    q4.kv_append(q4.kv_cache(kc, vc), q4.rotary(inv, k_norm=torch.ones(64, device=DEV)), None, k,
                 k, pos, slots)
    clean = torch.isfinite(kc[0, :, :3]).all(-1)
    assert clean.tolist() == [[True, False, True], [True, True, False]]
    assert torch.equal(torch.isinf(vc[0, 0, 1]).nonzero().flatten().cpu(), torch.tensor([5]))


# ---- attention --------------------------------------------------------------
def batch_inputs(lengths, hq, hk, dim, page, half, seed, window=0, sinks=0, q_scale=1.0):
    """Caches filled with NaN wherever no token of the call sees, tables with
    invalid entries there, pages in a shuffled order."""
    rng = np.random.default_rng(seed)
    widths = [max(0, (kv + page - 1) // page) for _, kv in lengths]
    width, pages = max(max(widths), 1), sum(widths) + 2
    order = rng.permutation(pages)
    kc, vc = (np.full((pages, hk, page, dim), np.nan, np.float16) for _ in range(2))
    table = np.full((len(lengths), width), -7, np.int32)
    at = 0
    for s, (new, kv) in enumerate(lengths):
        for w in range(widths[s]):
            seen = [j for j in range(w * page, min(kv, (w + 1) * page))
                    if any(block.sees(p, j, window, sinks) for p in range(max(0, kv - new), kv))]
            if seen:
                table[s, w] = order[at]
                offs = [j % page for j in seen]
                for c in (kc, vc):
                    c[order[at]][:, offs] = rng.standard_normal((hk, len(offs), dim))
            at += 1
    n = sum(new for new, _ in lengths)
    q = (q_scale * rng.standard_normal((n, hq, dim))).astype(np.float16 if half else np.float32)
    start = np.concatenate([[0], np.cumsum([new for new, _ in lengths])]).astype(np.int32)
    return kc, vc, q, start, np.array([kv for _, kv in lengths], np.int32), table


def attention_tol(ref, absolute, score, keys, dim, half):
    d = score[..., None] * (2.0 ** -22 + (dim + 8) * H32)
    weight = (H16 if half else 0.0) + 2.0 ** -22 + 2 * (keys + 16) * H32
    return absolute * (2.02 * d + weight) + np.abs(ref) * (H16 if half else H32) + 2.0 ** -25


def check(lengths, hq, hk, dim, page, window, sinks, half, seed=0, q_scale=1.0, pad=0):
    kc, vc, q, start, lens, table = batch_inputs(lengths, hq, hk, dim, page, half, seed, window,
                                                 sinks, q_scale)
    scale = dim ** -0.5
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, window, sinks, scale)
    tq = dev(q)
    if pad:                                            # rows that are slices of wider ones
        wide = torch.full((q.shape[0], hq * dim + pad), float("nan"), dtype=tq.dtype, device=DEV)
        wide[:, :hq * dim] = tq.flatten(1)
        tq = wide[:, :hq * dim].unflatten(1, (hq, dim))
    y = torch.full(q.shape, 7.0, dtype=tq.dtype, device=DEV)
    tk, tv = dev(kc), dev(vc)
    args = (q4.kv_cache(tk, tv), tq, dev(start), dev(lens), dev(table), window, sinks, scale)
    q4.attention(*args, y=y)
    torch.cuda.synchronize()
    near(y, ref, attention_tol(ref, absolute, score, max(kv for _, kv in lengths), dim, half))
    again = q4.attention(*args)                        # no order of arrival in any sum
    assert torch.equal(y, again)


HEADS = [(1, 1), (4, 1), (8, 2), (6, 2), (5, 1), (16, 1), (7, 7), (40, 1)]


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", HEADS)
def test_attention_decode(heads, dim, half):
    """One token per conversation, lengths around the edges of pages and tiles,
    an empty conversation among them."""
    lengths = [(1, kv) for kv in (1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 200)] + [(0, 0), (0, 5)]
    check(lengths, *heads, dim, 16, 0, 0, half, seed=dim + heads[0])


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 0), (63, 70), (64, 4),
                                          (100, 17), (128, 500), (1000, 2)])
def test_attention_window(window, sinks, dim, half):
    """Windows and first tokens, decode and prefill rows in one batch."""
    check([(1, 190), (40, 133), (1, 3), (70, 70), (3, 260)], 4, 2, dim, 32, window, sinks, half,
          seed=window)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(4, 1), (3, 3), (6, 2), (16, 2)])
def test_attention_prefill(heads, dim, half):
    check([(150, 150), (1, 1), (33, 290), (65, 66)], *heads, dim, 16, 0, 0, half, seed=3)


@pytest.mark.parametrize("page", [16, 64, 256, 4096])
def test_attention_page_sizes_and_strided_rows(page):
    check([(20, 300), (1, 299), (2, 2)], 4, 2, 128, page, 0, 0, True, seed=page, pad=24)
    check([(20, 300), (1, 299), (2, 2)], 4, 2, 128, page, 50, 9, False, seed=page, pad=12)


@pytest.mark.parametrize("half", [True, False])
def test_attention_large_scores(half):
    """Weights of one and of nothing: the running maximum moves by hundreds."""
    check([(1, 500), (30, 200), (1, 3)], 4, 1, 128, 16, 0, 0, half, seed=1, q_scale=60.0)


@pytest.mark.parametrize("lengths", [[(1, 300), (1, 40)], [(90, 120)], [(300, 300)]])
@pytest.mark.parametrize("magnitude", [1e-12, 1e-4, 1e5, 1e20])
def test_attention_float32_queries_of_any_magnitude(magnitude, lengths):
    """Float32 queries far outside binary16's range, the scale bringing the
    scores back."""
    kc, vc, q, start, lens, table = batch_inputs(lengths, 4, 2, 128, 16, False, 21)
    q = (q * np.float32(magnitude)).astype(np.float32)
    scale = float(np.float32(0.088 / magnitude))
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, 0, 0, scale)
    tk, tv = dev(kc), dev(vc)
    y = q4.attention(q4.kv_cache(tk, tv), dev(q), dev(start), dev(lens), dev(table), scale=scale)
    near(y, ref, attention_tol(ref, absolute, score, 300, 128, False))


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("gap", [3.0, 14.0, 18.0])
def test_attention_many_faint_weights_beside_a_strong_one(gap, half):
    """The first key takes most of the weight, 40000 equal ones share the rest:
    their sum, a known value, has to survive."""
    n, dim = 40001, 64
    page, pages = 256, 160
    kc, vc = (torch.zeros(pages, 1, page, dim, dtype=torch.float16, device=DEV) for _ in range(2))
    kc[0, 0, 0, 0] = 8.0
    vc[:, 0, :, 1] = 1.0
    vc[0, 0, 0, 1] = -1.0
    q = torch.zeros(1, 2, dim, dtype=torch.float16 if half else torch.float32, device=DEV)
    q[:, :, 0] = gap
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    y = q4.attention(q4.kv_cache(kc, vc), q, torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                     torch.tensor([n], dtype=torch.int32, device=DEV), table, scale=0.125)
    faint = (n - 1) * np.exp(-float(q[0, 0, 0]))
    want = (faint - 1.0) / (faint + 1.0)
    # equal weights are off by one rounding, alike: of 2^-11, or 2^-16 where they lie
    # 2^-26 below the strong one; and float32 sums of 40000
    tol = (H16 if half else 2.0 ** -16) * 4 + n * H32 * 2
    assert (y[0, :, 1].double() - want).abs().max() < tol + abs(want) * H16 * half
    assert (y[0, :, 2:] == 0).all()


@pytest.mark.parametrize("half", [True, False])
def test_attention_rows_that_see_nothing(half):
    """More new tokens than cached positions: the first rows see nothing and
    give 0; a conversation without a cache gives only zeros."""
    check([(10, 4), (3, 0), (1, 0), (40, 20), (2, 2)], 4, 2, 64, 16, 0, 0, half, seed=8)
    check([(10, 4), (3, 0), (1, 0), (40, 20), (2, 2)], 4, 2, 64, 16, 3, 2, half, seed=8)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("lengths", [[(1, 2000)], [(1, 1999), (1, 40)], [(4, 1500)], [(70, 1400)]])
def test_attention_long_axis(lengths, half):
    """Few rows and many keys: the key axis is split."""
    check(lengths, 8, 2, 64, 16, 0, 0, half, seed=11)
    check(lengths, 8, 2, 64, 16, 700, 40, half, seed=12)


@pytest.mark.parametrize("count,tokens,longest", [(65, 1, 90), (150, 1, 40), (300, 3, 30),
                                                  (4500, 1, 9), (130, 40, 50)])
def test_attention_many_conversations(count, tokens, longest):
    """More conversations than one look of 64 lanes finds, empty ones among
    them, and leading tokens that none of them holds."""
    rng = np.random.default_rng(count)
    kvs = rng.integers(0, longest + 1, count)
    news = np.minimum(kvs, rng.integers(0, tokens + 1, count))
    lengths = [(int(a), int(b)) for a, b in zip(news, kvs)]
    kc, vc, q, start, lens, table = batch_inputs(lengths, 2, 1, 64, 16, True, 5)
    spare = 3
    q = np.concatenate([q[:spare], q])
    start = start + np.int32(spare)
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, 0, 0, 0.125)
    tk, tv = dev(kc), dev(vc)
    y = torch.full(q.shape, 9.0, dtype=torch.float16, device=DEV)
    q4.attention(q4.kv_cache(tk, tv), dev(q), dev(start), dev(lens), dev(table), y=y)
    assert (y[:spare] == 9.0).all()
    near(y[spare:], ref[spare:], attention_tol(ref[spare:], absolute[spare:], score[spare:],
                                               longest, 64, True))


def test_attention_long_batch_with_split_parts():
    """More than 64 conversations whose key axes are split: the joining kernel
    finds their tokens too."""
    rng = np.random.default_rng(2)
    lengths = [(1, int(n)) for n in rng.integers(1, 60, 70)] + [(1, 2600), (0, 0), (1, 1700)]
    assert q4.q4_0_attention_workspace_size(
        q4.q4_0_kv_cache(0, 0, 500, 1, 16, 64), 2, q4.F16, 72, 163, 73) > 0
    check(lengths, 2, 1, 64, 16, 0, 0, True, seed=6)
    check(lengths, 2, 1, 64, 16, 1500, 33, False, seed=7)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_non_finite_values_in_masked_places(dim, half):
    """A key's or value's infinity or NaN changes the rows that see it and no
    other, though they share its tile."""
    rng = np.random.default_rng(5)
    new, kv, hq, hk, page, window = 50, 90, 4, 2, 16, 30
    kc, vc = (rng.standard_normal((6, hk, page, dim)).astype(np.float16) for _ in range(2))
    table = np.arange(6, dtype=np.int32)[None]
    dt = np.float16 if half else np.float32
    q = rng.standard_normal((new, hq, dim)).astype(dt)
    start, lens = np.array([0, new], np.int32), np.array([kv], np.int32)
    spots = [(vc, 70, 3, np.inf), (vc, 71, 3, np.inf), (vc, 60, 5, -np.inf), (vc, 52, 9, np.nan),
             (kc, 80, 1, np.nan), (vc, 85, 7, np.inf), (vc, 86, 7, -np.inf)]
    for c, j, d, x in spots:
        c[j // page, 1, j % page, d] = x
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, window, 0, dim ** -0.5)
    tk, tv = dev(kc), dev(vc)
    y = q4.attention(q4.kv_cache(tk, tv), dev(q), dev(start), dev(lens), dev(table), window, 0)
    absolute = np.where(np.isfinite(absolute), absolute, 0.0)
    score = np.where(np.isfinite(score), score, 0.0)
    near(y, ref, attention_tol(np.where(np.isfinite(ref), ref, 0.0), absolute, score, kv, dim, half))
    assert np.isfinite(ref[:, :2]).all() and not np.isfinite(ref[:, 2:]).all()


@pytest.mark.parametrize("half", [True, False])
def test_attention_bad_pages_and_tables(half):
    """A row that sees a key on a page outside the cache, or past the table's
    end, is NaN; the rows that do not are untouched.  Rows of no conversation
    keep what y had."""
    kc, vc, q, start, lens, table = batch_inputs([(60, 100), (1, 50), (1, 70)], 4, 2, 64, 16, half, 2)
    table[0, 4] = 99999                                 # keys 64..79 of the first
    table[1, 1] = -1
    lens[2] = 7 * 16 + 5                                # the table ends at 7 pages
    kc, vc = np.nan_to_num(kc), np.nan_to_num(vc)
    table[2, 5:] = 0
    q = np.concatenate([q, q[:3]])
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, 0, 0, 0.125)
    assert np.isnan(ref[24:62]).all() and np.isfinite(ref[:24]).all()
    y = torch.full(q.shape, 5.0, dtype=torch.float16 if half else torch.float32, device=DEV)
    tk, tv = dev(kc), dev(vc)
    q4.attention(q4.kv_cache(tk, tv), dev(q), dev(start), dev(lens), dev(table), y=y)
    assert (y[62:] == 5.0).sum() == 3 * 4 * 64
    near(y[:62], ref[:62], attention_tol(np.nan_to_num(ref[:62]), absolute[:62], score[:62], 120, 64, half))


@pytest.mark.parametrize("window", [0, 20])
def test_attention_impossible_lengths(window):
    """Lengths far past the table, and negative ones, end as rows of NaN and of
    zeros; the conversation beside them is untouched."""
    kc, vc, q, start, lens, table = batch_inputs([(2, 40)] * 3, 4, 2, 64, 16, True, 4)
    lens[0], lens[2] = 2 ** 31 - 1, -2 ** 31
    kc, vc = np.nan_to_num(kc), np.nan_to_num(vc)
    tk, tv = dev(kc), dev(vc)
    y = q4.attention(q4.kv_cache(tk, tv), dev(q), dev(start), dev(lens), dev(table), window, 1)
    lens[0] = lens[2] = 0
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, window, 1, 0.125)
    assert torch.isnan(y[:2]).all() and (y[4:] == 0).all()
    near(y[2:4], ref[2:4], attention_tol(ref[2:4], absolute[2:4], score[2:4], 40, 64, True))


def test_attention_offsets_past_32_bits():
    """Pages whose elements lie past 2^32: the same keys on the cache's first and
    last pages give the same result."""
    pages, hk, page, dim = 140000, 1, 256, 128         # 4.6e9 elements each
    free = torch.cuda.mem_get_info()[0]
    if free < 40 * 2 ** 30:
        pytest.skip("needs 40 GiB of device memory")
    kc = torch.zeros(pages, hk, page, dim, dtype=torch.float16, device=DEV)
    vc = torch.zeros_like(kc)
    k = torch.randn(700, 1, dim, device=DEV)
    cache, inv = q4.kv_cache(kc, vc), torch.ones(8, device=DEV)
    step = torch.arange(700, device=DEV)
    q = torch.randn(1, 4, dim, device=DEV)
    got = []
    for first in (0, pages - 3):
        q4.kv_append(cache, q4.rotary(inv), None, k, -k, step.int(), first * page + step)
        table = torch.arange(first, first + 3, dtype=torch.int32, device=DEV)[None]
        got.append(q4.attention(cache, q, torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                                torch.tensor([700], dtype=torch.int32, device=DEV), table))
    torch.cuda.synchronize()
    assert torch.equal(kc[:3], kc[-3:]) and kc[:3].abs().sum() > 0
    assert torch.equal(got[0], got[1]) and got[0].abs().sum() > 0


# ---- residual norm ----------------------------------------------------------
def norm_check(n, dim, bh, yh, post, gate, pre=True, b=True, pad=0, in_place=False, offset=0.0):
    rng = np.random.default_rng([n, dim, bh, yh])
    h = rng.standard_normal((n, dim + pad)).astype(np.float32)
    x = rng.standard_normal((n, dim + pad)).astype(np.float16 if bh else np.float32)
    shape = {"none": None, "row": (n, 1), "channel": (1, dim), "full": (n, dim)}[gate]
    g = None if shape is None else rng.random(shape).astype(np.float32)
    pw, qw = ((1 + 0.1 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2))
    rh, ry = block.residual_norm(h[:, :dim], x[:, :dim] if b else None, qw if pre else None,
                                 pw if post else None, g, 0.7, 1e-5, offset)
    th = dev(h)[:, :dim]
    out = th if in_place else None
    oh, oy = q4.residual_norm(th, dev(x)[:, :dim] if b else None, dev(qw) if pre else None,
                              dev(pw) if post else None, None if g is None else dev(g), 0.7, 1e-5,
                              offset, h_out=out, y_dtype=torch.float16 if yh else torch.float32)
    torch.cuda.synchronize()
    # the norm's factor: a sum of dim squares and a root, halved by the root
    f = (dim / 2 + 10) * H32
    added = np.abs(rh - h[:, :dim]) if b else 0.0
    tol_h = added * (f + 8 * H32) + np.abs(rh) * 2 * H32 + 1e-30
    if b:
        near(oh, rh, tol_h)
    if pre:
        rms = np.sqrt((rh * rh).mean(-1, keepdims=True) + 1e-5)
        w = np.abs(qw + offset)
        slip = np.sqrt((tol_h * tol_h).mean(-1, keepdims=True)) / rms
        near(oy, ry, np.abs(ry) * (f + slip + (H16 if yh else H32)) + tol_h / rms * w + 2.0 ** -25)
    else:
        assert oy is None


@pytest.mark.parametrize("dim", [1, 2, 63, 64, 65, 255, 512, 1000, 1028, 2560, 4099, 8192, 16384,
                                 20000, 32767, 32768])
def test_residual_norm_widths(dim):
    for bh, yh in itertools.product((False, True), repeat=2):
        norm_check(3, dim, bh, yh, True, "none")


@pytest.mark.parametrize("gate", ["none", "row", "channel", "full"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("n,dim", [(1, 2560), (7, 130), (70, 96), (5, 333)])
def test_residual_norm_gates(n, dim, post, gate):
    norm_check(n, dim, False, True, post, gate, offset=1.0)
    norm_check(n, dim, True, False, post, gate, in_place=True)


@pytest.mark.parametrize("pad", [1, 4, 6])
def test_residual_norm_strides(pad):
    norm_check(6, 132, False, False, True, "full", pad=pad)
    norm_check(6, 132, True, True, True, "row", pad=pad, in_place=True)


def test_residual_norm_parts():
    norm_check(5, 260, False, True, True, "none", pre=False)
    norm_check(5, 260, False, True, False, "none", b=False)
    norm_check(4000, 64, False, False, True, "channel")


def test_residual_norm_zero_and_non_finite_rows():
    h, b = torch.zeros(3, 64, device=DEV), torch.zeros(3, 64, device=DEV)
    b[1, 7], h[2, 9] = float("inf"), float("nan")
    w = torch.ones(64, device=DEV)
    oh, oy = q4.residual_norm(h, b, w, w)
    assert (oh[0] == 0).all() and (oy[0] == 0).all()
    assert torch.isnan(oh[1, 7]) and torch.isnan(oy[2]).all()
    assert (oh[1].nan_to_num() == 0).all()


# ---- streams, graphs --------------------------------------------------------
def test_block_operators_on_another_stream_and_replayed():
    """A decode step (append, attention, residual norm) captured once on a side
    stream and replayed as the conversations grow, against eager calls."""
    torch.manual_seed(0)
    b, hq, hk, dim, page, width = 3, 8, 2, 64, 16, 8
    kc = torch.randn(b * width, hk, page, dim, device=DEV).half()
    vc = torch.randn_like(kc)
    table = torch.randperm(b * width, device=DEV).int().view(b, width)
    start = torch.arange(b + 1, dtype=torch.int32, device=DEV)
    qkv = torch.randn(b, (hq + 2 * hk) * dim, device=DEV)
    lens, pos = (torch.zeros(b, dtype=torch.int32, device=DEV) for _ in range(2))
    slots = torch.zeros(b, dtype=torch.int64, device=DEV)
    inv, w = torch.rand(dim // 2, device=DEV), torch.ones(hq * dim, device=DEV)
    h = torch.randn(b, hq * dim, device=DEV)
    cache, rot = q4.kv_cache(kc, vc), q4.rotary(inv)
    q_out, y = torch.empty(b, hq, dim, device=DEV), torch.empty(b, hq, dim, device=DEV)
    need = q4.q4_0_attention_workspace_size(cache, hq, q4.F32, b, width, b)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    oh, oy = torch.empty_like(h), torch.empty_like(h)

    def step():
        q, k, v = qkv.split([hq * dim, hk * dim, hk * dim], dim=1)
        q4.kv_append(cache, rot, q, k, v, pos, slots, q_out=q_out)
        q4.attention(cache, q_out, start, lens, table, y=y, ws=ws)
        q4.residual_norm(h, y.flatten(1), w, w, h_out=oh, y=oy)

    def place(i):
        base = torch.tensor([5, 40, 100], device=DEV) + i
        pos.copy_(base)
        lens.copy_(base + 1)
        at = table.long().gather(1, (base // page)[:, None])[:, 0]
        slots.copy_(at * page + base % page)
        qkv.normal_()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        place(0)
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, 20):
        place(i)
        before = kc.clone(), vc.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q_out, y, oh, oy, kc, vc)]
        kc.copy_(before[0])
        vc.copy_(before[1])
        for t in (q_out, y, oh, oy):
            t.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        for g, e in zip(got, (q_out, y, oh, oy, kc, vc)):
            assert torch.equal(g, e), i


@pytest.mark.parametrize("handle", [False, True])
def test_conveniences_on_a_given_stream(handle):
    """Outputs and workspaces that a call on another stream allocates are not
    given away before it has run: many calls in flight there, with allocations
    on the current stream in between."""
    torch.manual_seed(3)
    k, v = (torch.randn(300, 2, 16, 64, device=DEV).half() for _ in range(2))
    cache = q4.kv_cache(k, v)
    q = torch.randn(1, 4, 64, device=DEV)
    start = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    lens = torch.tensor([4700], dtype=torch.int32, device=DEV)
    table = torch.arange(300, dtype=torch.int32, device=DEV)[None]
    h, w = torch.randn(3, 256, device=DEV), torch.ones(256, device=DEV)
    assert q4.q4_0_attention_workspace_size(cache, 4, q4.F32, 1, 300, 1) > 0
    want = q4.attention(cache, q, start, lens, table), q4.residual_norm(h, h * 2, w, w)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    got = []
    twice = h * 2
    torch.cuda.synchronize()
    for _ in range(20):
        got.append((q4.attention(cache, q, start, lens, table, stream=stream),
                    q4.residual_norm(h, twice, w, w, stream=stream)))
        for size in (1 << 12, 1 << 16, 1 << 20):
            torch.empty(size, dtype=torch.uint8, device=DEV).fill_(255)
        side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for y, (oh, oy) in got:
        assert torch.equal(y, want[0]) and torch.equal(oy, want[1][1])
        assert torch.equal(oh, want[1][0])


def test_workspace_contents_do_not_matter():
    k, v = (torch.randn(64, 2, 16, 64, device=DEV).half() for _ in range(2))
    cache = q4.kv_cache(k, v)
    q = torch.randn(1, 4, 64, device=DEV)
    start = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    lens = torch.tensor([900], dtype=torch.int32, device=DEV)
    table = torch.arange(64, dtype=torch.int32, device=DEV)[None]
    need = q4.q4_0_attention_workspace_size(cache, 4, q4.F32, 1, 64, 1)
    got = []
    for fill in (0, 255):
        ws = torch.full((max(need, 256),), fill, dtype=torch.uint8, device=DEV)
        got.append(q4.attention(cache, q, start, lens, table, ws=ws))
    assert torch.equal(got[0], got[1]) and torch.isfinite(got[0]).all()


def test_block_operators_allocate_no_device_memory():
    """Free device memory is unchanged by calls with caller-owned buffers (after
    a first round that loads the code)."""
    n, hq, hk, dim = 70, 8, 2, 128
    kc, vc = (torch.zeros(64, hk, 16, dim, dtype=torch.float16, device=DEV) for _ in range(2))
    cache, rot = q4.kv_cache(kc, vc), q4.rotary(torch.ones(64, device=DEV))
    qkv = torch.randn(n, (hq + 2 * hk) * dim, device=DEV)
    parts = qkv.split([hq * dim, hk * dim, hk * dim], dim=1)
    pos, slots = torch.arange(n, device=DEV).int(), torch.arange(n, device=DEV)
    q, y = torch.empty(n, hq, dim, device=DEV), torch.empty(n, hq, dim, device=DEV)
    ws = torch.empty(q4.WORKSPACE_MAX, dtype=torch.uint8, device=DEV)
    table = torch.arange(64, dtype=torch.int32, device=DEV)[None]
    one, all_ = (torch.tensor([0, k], dtype=torch.int32, device=DEV) for k in (1, n))
    lens = torch.tensor([1000], dtype=torch.int32, device=DEV)
    h, w = torch.randn(n, hq * dim, device=DEV), torch.ones(hq * dim, device=DEV)
    oh, oy = torch.empty_like(h), torch.empty_like(h)

    def round_():
        q4.kv_append(cache, rot, *parts, pos, slots, q_out=q)
        q4.attention(cache, q, all_, lens, table, y=y, ws=ws)
        q4.attention(cache, q[:1], one, lens, table, y=y[:1], ws=ws)      # split, joined
        q4.residual_norm(h, y.flatten(1), w, w, h_out=oh, y=oy)

    round_()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    for _ in range(5):
        round_()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == before


def test_example_decodes_what_one_pass_gives():
    """The example's captured decode steps against one pass over the whole text;
    with a window and first tokens, and without.  Decode takes activations in 22
    bits, a pass of more rows in binary16: a dozen roundings of 2^-11 along the
    way, of which the two that norms rescale count most."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for args in ({}, dict(window=0, sinks=0, prompts=(3, 100), steps=6, heads=8, dim=128, seed=4)):
        got, want = example.run(**args)
        assert torch.isfinite(got).all()
        assert float((got - want).norm() / want.norm()) < 12 * H16


def test_calls_refuse_tensors_on_the_host():
    k = torch.zeros(2, 2, 16, 64, dtype=torch.float16, device=DEV)
    c = q4.kv_cache(k, k.clone())
    q = torch.zeros(1, 4, 64, device=DEV)
    start = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    lens = torch.tensor([1], dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        q4.attention(c, q, start, lens, table)
    kv = torch.zeros(1, 2, 64, device=DEV)
    slots = torch.zeros(1, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        q4.kv_append(c, q4.rotary(torch.ones(32)), q, kv, kv, start[:1], slots)
    with pytest.raises(ValueError):
        q4.residual_norm(kv[0], kv[0], torch.ones(64))
    with pytest.raises(ValueError):
        q4.kv_append(c, None, q, kv, kv, None, slots.cpu())


def test_first_calls_of_a_process_capture_into_a_graph():
    import json
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "cold_capture_block.py")],
                       capture_output=True, text=True, timeout=100)
    print(r.stdout[-2000:], r.stderr[-2000:], flush=True)
    assert r.returncode == 0
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(res) == 7 and all(res.values()), res
