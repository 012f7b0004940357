"""A step of drafted tokens on the GPU against the float64 definitions
(oracle/step.py, oracle/block.py): the 8-bit cache's append, reading and
attention, the table's lookup, the drafts' verification, and all of them
together.

Tolerances follow from the roundings a result passes through, in units of half
a step (binary16 2^-11, float32 2^-24), with worst-case sums:
- a float32 sum of N products is off by at most (N + 1) 2^-24 times the sum of
  their absolute values; scales multiply scores and weights once each;
- float32 attention takes q and the weights as two binary16 parts, off by
  2^-22; passes of binary16 rows round each weight once (2^-11);
- a code is within half a step of its element, and the scale, a maximum over
  127, as near as the elements are.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_q4_amd as q4
import oracle
import synth
from oracle import block, step
from test_gpu_block import DEV, H16, H32, append_tol, dev, near

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---- append and reading ------------------------------------------------------
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
def test_append8(case):
    n, hq, hk, dim, rot_dim, page, inter, norm, xh, qh, first = case
    rng = np.random.default_rng(list(case[:6]))
    pages = (n + page - 1) // page + 2
    wide = rng.standard_normal((n, (hq + 2 * hk) * dim + 16)).astype(
        np.float16 if xh else np.float32)
    q, k, v = (wide[:, a:b] for a, b in ((0, hq * dim), (hq * dim, (hq + hk) * dim),
                                         ((hq + hk) * dim, (hq + 2 * hk) * dim)))
    codes = [rng.integers(-128, 128, (pages, hk, page, dim)).astype(np.int8) for _ in range(2)]
    scales = [rng.random((pages, hk, page)).astype(np.float32) for _ in range(2)]
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    if n > 4:
        slots[1], slots[3] = -1, pages * page            # two padded tokens
    pos = (first + np.arange(n)).astype(np.int32)
    inv = (10000.0 ** (-np.arange(0, rot_dim, 2) / max(rot_dim, 1))).astype(np.float32)
    qw, kw = ((1 + 0.1 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2))
    amp, off = (1.0, 0.0) if n % 2 else (1.25, 0.5)
    empty = np.zeros((pages, hk, page, dim))
    rq, rk, rv = block.append(empty, empty, q, k, v, pos, slots, inv_freq=inv, interleaved=inter,
                              amplitude=amp, eps=1e-5, offset=off, q_norm=qw if norm else None,
                              k_norm=kw if norm else None)
    w, t = dev(wide), [dev(a) for a in (*codes, *scales)]
    rot = q4.rotary(inv_freq=dev(inv) if rot_dim else None, interleaved=inter, amplitude=amp,
                    eps=1e-5, weight_offset=off, q_norm=dev(qw) if norm else None,
                    k_norm=dev(kw) if norm else None)
    out = torch.full((n, hq, dim), float("nan"), dtype=torch.float16 if qh else torch.float32,
                     device=DEV)
    cache = q4.kv_cache8(*t)
    q4.kv_append(cache, rot, w[:, :hq * dim], w[:, hq * dim:(hq + hk) * dim],
                 w[:, (hq + hk) * dim:(hq + 2 * hk) * dim], dev(pos), dev(slots), q_out=out)
    torch.cuda.synchronize()
    near(out, rq, append_tol(rq, rq, qh, qw if norm else None, rot_dim > 0))
    kc, vc, ks, vs = (x.cpu().numpy() for x in t)
    written = np.zeros((pages, hk, page), bool)
    for s in slots[(slots >= 0) & (slots < pages * page)]:
        written[s // page, :, s % page] = True
    for got, was in zip((kc, vc, ks, vs), (*codes, *scales)):
        assert np.array_equal(got[~written], was[~written])
    # V enters as it is: the codes and scales of float32 arithmetic, bit for bit
    c, s = step.quantize(rv[written].astype(np.float32))
    assert np.array_equal(vc[written], c) and np.array_equal(vs[written], s)
    # K carries the norm's and the rotation's roundings
    x = rk[written]
    slip = append_tol(x, x, False, kw if norm else None, rot_dim > 0)
    top = np.abs(x).max(-1)
    near(ks[written], top / 127, slip.max(-1) / 127 + top / 127 * 2 * H32)
    half = ks[written].astype(np.float64)[:, None] / 2
    near(kc[written] * ks[written].astype(np.float64)[:, None], x, half * (1 + 1e-4) + slip)
    assert (np.abs(kc[written].astype(int)).max(-1) == 127).all() and kc[written].min() >= -127

    # reading: every row, some twice, some outside
    where = np.concatenate([np.arange(pages * page), [0, 5, -1, pages * page, 2 ** 40]])
    inside = (where >= 0) & (where < pages * page)
    for dt, h in ((torch.float16, H16), (torch.float32, H32)):
        gk, gv = q4.kv_read(cache, dev(where), dtype=dt)
        for got, cc, ss in ((gk, kc, ks), (gv, vc, vs)):
            want = step.numbers(cc, ss).transpose(0, 2, 1, 3).reshape(-1, hk, dim)
            want = np.where(inside[:, None, None], want[np.where(inside, where, 0)], 0.0)
            near(got, want, np.abs(want) * h + (2.0 ** -25 if h == H16 else 0.0))


def test_append8_zero_faint_and_non_finite_rows():
    k = torch.randn(6, 2, 64, device=DEV)
    k[0] = 0.0
    k[1, 0] *= 1e-38                                   # its scale would be subnormal
    k[2, 1, 5], k[3, 0, 7], k[4, 0, 1] = float("inf"), float("nan"), -float("inf")
    k[5] *= 1e37
    codes = [torch.full((1, 2, 16, 64), 9, dtype=torch.int8, device=DEV) for _ in range(2)]
    scales = [torch.full((1, 2, 16), 7.0, device=DEV) for _ in range(2)]
    cache, slots = q4.kv_cache8(*codes, *scales), torch.arange(6, device=DEV)
    q4.kv_append(cache, None, None, k, k, None, slots)
    for c, s in zip(codes, scales):
        c, s = c[0, :, :6].transpose(0, 1).cpu(), s[0, :, :6].transpose(0, 1).cpu()
        assert (s[0] == 0).all() and (c[0] == 0).all() and s[1, 0] == 0 and (c[1, 0] == 0).all()
        assert torch.isnan(s).nonzero().tolist() == [[2, 1], [3, 0], [4, 0]]
        wc, ws = step.quantize(k[5].cpu().numpy())
        assert np.array_equal(c[5].numpy(), wc) and np.array_equal(s[5].numpy(), ws)
        assert (codes[0][0, :, 6:] == 9).all() and (scales[0][0, :, 6:] == 7).all()
    gk, gv = q4.kv_read(cache, slots, dtype=torch.float32)
    assert torch.isnan(gk).all(-1).nonzero().tolist() == [[2, 1], [3, 0], [4, 0]]
    assert torch.equal(torch.isnan(gk), torch.isnan(gv)) and (gk[0] == 0).all()


@pytest.mark.parametrize("only", ["k", "v"])
def test_read8_of_one_side(only):
    codes = torch.randint(-128, 128, (2, 3, 16, 72), dtype=torch.int8, device=DEV)
    other = torch.zeros_like(codes)
    scales, none = torch.rand(2, 3, 16, device=DEV), torch.zeros(2, 3, 16, device=DEV)
    c = q4.q4_0_kv_cache8(*(t.data_ptr() for t in (
        (codes, other, scales, none) if only == "k" else (other, codes, none, scales))), 2, 3, 16, 72)
    slots, out = torch.arange(31, -1, -1, device=DEV), torch.empty(32, 3, 72, device=DEV)
    q4.q4_0_kv_read8(c, slots, 32, out if only == "k" else None, out if only == "v" else None, q4.F32)
    want = (codes.float() * scales[..., None]).transpose(1, 2).reshape(32, 3, 72).flip(0)
    assert torch.equal(out, want)


# ---- attention ---------------------------------------------------------------
def inputs8(lengths, hq, hk, dim, page, half, seed, window=0, sinks=0, q_scale=1.0, spread=0.5):
    """Codes of any value and scales of several magnitudes; NaN scales and other
    codes wherever no token of the call sees, tables with invalid entries there,
    pages in a shuffled order."""
    rng = np.random.default_rng(seed)
    widths = [max(0, (kv + page - 1) // page) for _, kv in lengths]
    width, pages = max(max(widths), 1), sum(widths) + 2
    order = rng.permutation(pages)
    kc, vc = (rng.integers(-128, 128, (pages, hk, page, dim)).astype(np.int8) for _ in range(2))
    ks, vs = (np.full((pages, hk, page), np.nan, np.float32) for _ in range(2))
    table = np.full((len(lengths), width), -7, np.int32)
    at = 0
    for s, (new, kv) in enumerate(lengths):
        for w in range(widths[s]):
            seen = [j for j in range(w * page, min(kv, (w + 1) * page))
                    if any(block.sees(p, j, window, sinks) for p in range(max(0, kv - new), kv))]
            if seen:
                table[s, w] = order[at]
                offs = [j % page for j in seen]
                for c in (ks, vs):
                    c[order[at]][:, offs] = np.exp(
                        spread * rng.standard_normal((hk, len(offs)))) / 70.0
            at += 1
    n = sum(new for new, _ in lengths)
    q = (q_scale * rng.standard_normal((n, hq, dim))).astype(np.float16 if half else np.float32)
    start = np.concatenate([[0], np.cumsum([new for new, _ in lengths])]).astype(np.int32)
    return kc, vc, ks, vs, q, start, np.array([kv for _, kv in lengths], np.int32), table


def tol8(ref, absolute, score, keys, dim, half, least=2.0 ** -25):
    d = score[..., None] * (2.0 ** -22 + (dim + 10) * H32)
    weight = (H16 if half else 0.0) + 2.0 ** -22 + 2 * (keys + 18) * H32
    return absolute * (2.02 * d + weight) + np.abs(ref) * (H16 if half else H32) + least


def attend8(kc, vc, ks, vs, q, start, lens, table, window=0, sinks=0, scale=1.0):
    return block.attend(step.numbers(kc, ks), step.numbers(vc, vs), q, start, lens, table, window,
                        sinks, scale)


def check8(lengths, hq, hk, dim, page, window, sinks, half, seed=0, q_scale=1.0, pad=0, spread=0.5):
    args = inputs8(lengths, hq, hk, dim, page, half, seed, window, sinks, q_scale, spread)
    kc, vc, ks, vs, q, start, lens, table = args
    scale = dim ** -0.5
    ref, absolute, score = attend8(*args, window, sinks, scale)
    tq = dev(q)
    if pad:                                            # rows that are slices of wider ones
        wide = torch.full((q.shape[0], hq * dim + pad), float("nan"), dtype=tq.dtype, device=DEV)
        wide[:, :hq * dim] = tq.flatten(1)
        tq = wide[:, :hq * dim].unflatten(1, (hq, dim))
    y = torch.full(q.shape, 7.0, dtype=tq.dtype, device=DEV)
    call = (q4.kv_cache8(*(dev(a) for a in (kc, vc, ks, vs))), tq, dev(start), dev(lens),
            dev(table), window, sinks, scale)
    q4.attention(*call, y=y)
    torch.cuda.synchronize()
    near(y, ref, tol8(ref, absolute, score, max(kv for _, kv in lengths), dim, half))
    again = q4.attention(*call)                        # no order of arrival in any sum
    assert torch.equal(y, again)


HEADS = [(1, 1), (4, 1), (8, 2), (6, 2), (5, 1), (16, 1), (17, 1), (7, 7), (40, 1)]


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", HEADS)
def test_attention8_decode(heads, dim, half):
    """One token per conversation, lengths around the edges of pages and tiles,
    an empty conversation among them."""
    lengths = [(1, kv) for kv in (1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 200)] + [(0, 0), (0, 5)]
    check8(lengths, *heads, dim, 16, 0, 0, half, seed=dim + heads[0])


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention8_drafts(dim, half):
    """A last token and drafts of it: rows on both sides of sixteen and of 32."""
    check8([(5, 70), (1, 300), (8, 8), (3, 129), (4, 64), (2, 65), (0, 9)], 8, 2, dim, 32, 0, 0,
           half, seed=dim)
    check8([(5, 70), (1, 300), (8, 8), (3, 129)], 12, 2, dim, 16, 40, 3, half, seed=dim)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 0), (63, 70), (64, 4),
                                          (100, 17), (128, 500), (1000, 2)])
def test_attention8_window(window, sinks, dim, half):
    check8([(1, 190), (40, 133), (1, 3), (70, 70), (3, 260)], 4, 2, dim, 32, window, sinks, half,
           seed=window)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(4, 1), (3, 3), (6, 2), (16, 2)])
def test_attention8_prefill(heads, dim, half):
    check8([(150, 150), (1, 1), (33, 290), (65, 66)], *heads, dim, 16, 0, 0, half, seed=3)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 37])
def test_attention8_long_tiles(dim, half, window):
    """Enough rows for 128-row tiles, on a device of any size."""
    lengths, hk = [(1100, 1100), (3, 50), (900, 1000)], 20
    args = q4.q4_0_kv_cache8(0, 0, 0, 0, 1, hk, 64, dim), hk, q4.F16, 2003, 18, 3, window, 2
    assert q4.q4_0_select_attention8(*args) == 128
    rng = np.random.default_rng(dim)
    kc, vc, ks, vs, q, start, lens, table = inputs8([(0, kv) for _, kv in lengths], hk, hk, dim, 64,
                                                    half, 1)
    kc, vc, ks, vs = (t[:, :1].repeat(hk, 1) for t in (kc, vc, ks, vs))
    pages = len(kc)
    ks[:], vs[:] = (np.exp(0.5 * rng.standard_normal((pages, 1, 64))) / 70 for _ in range(2))
    table = np.full((3, 18), -1, np.int32)
    table[0], table[1, :1], table[2, :16] = np.arange(18), 18, np.arange(19, 35)
    new = [a for a, _ in lengths]
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = rng.standard_normal((sum(new), 1, dim)).astype(np.float16 if half else np.float32)
    scale = dim ** -0.5
    some = np.unique(np.concatenate([np.arange(0, sum(new), 61), [1099, 1100, 1102, 1103, 2002]]))
    y = q4.attention(q4.kv_cache8(*(dev(a) for a in (kc, vc, ks, vs))),
                     dev(np.ascontiguousarray(q.repeat(hk, 1))), dev(start), dev(lens), dev(table),
                     window, 2, scale)
    # rows of one head alike in all, and a sample of them against the definition
    assert torch.equal(y[:, :1].expand(-1, hk, -1), y)
    k64, v64 = step.numbers(kc[:, :1], ks[:, :1]), step.numbers(vc[:, :1], vs[:, :1])
    for t in some:
        s = int(np.searchsorted(start, t, "right") - 1)
        p = lens[s] - (start[s + 1] - t)
        ref, absolute, score = block.attend(k64, v64, q[t:t + 1], [0, 1], [p + 1], table[s:s + 1],
                                            window, 2, scale)
        near(y[t:t + 1, :1], ref, tol8(ref, absolute, score, 1100, dim, half))


@pytest.mark.parametrize("page", [16, 64, 256, 4096])
def test_attention8_page_sizes_and_strided_rows(page):
    check8([(20, 300), (1, 299), (2, 2)], 4, 2, 128, page, 0, 0, True, seed=page, pad=24)
    check8([(20, 300), (1, 299), (2, 2)], 4, 2, 128, page, 50, 9, False, seed=page, pad=12)
    check8([(1, 300), (3, 299), (2, 2)], 4, 2, 128, page, 0, 0, False, seed=page, pad=12)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("q_scale", [60.0, 3000.0])
def test_attention8_large_scores(half, q_scale):
    """Weights of one and of nothing: the running maximum moves by hundreds."""
    check8([(1, 500), (3, 300), (1, 3)], 4, 1, 128, 16, 0, 0, half, seed=1, q_scale=q_scale)
    check8([(1, 500), (30, 200), (1, 3)], 4, 1, 128, 16, 0, 0, half, seed=1, q_scale=q_scale)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("lengths", [[(1, 700), (2, 40)], [(90, 120)], [(40, 300)]])
@pytest.mark.parametrize("magnitude", [1e-30, 1e-9, 1e9, 1e30])
def test_attention8_values_of_any_magnitude(magnitude, lengths, half):
    """Value scales far outside binary16's range, and a few far larger or smaller
    than the others."""
    args = list(inputs8(lengths, 4, 2, 128, 16, half, 21))
    vs = args[3] * np.float32(1e-3 if half else magnitude)
    if half and magnitude != 1e9:      # results have to fit binary16
        vs = args[3] * np.float32(min(magnitude * 1e9, 1.0))
    flat = vs.reshape(-1)
    flat[::7] *= np.float32(1e-12)
    flat[3::50] *= np.float32(20.0)
    args[3] = vs
    kc, vc, ks, vs, q, start, lens, table = args
    y = q4.attention(q4.kv_cache8(*(dev(a) for a in (kc, vc, ks, vs))), dev(q), dev(start),
                     dev(lens), dev(table), scale=float(np.float32(0.088)))
    ref, absolute, score = attend8(*args, 0, 0, float(np.float32(0.088)))
    # (2^-25 is half a step of binary16's smallest numbers: float32's are far smaller)
    near(y, ref, tol8(ref, absolute, score, 700, 128, half, 2.0 ** -25 if half else 1e-37))


@pytest.mark.parametrize("lengths", [[(1, 300), (1, 40)], [(90, 120)], [(300, 300)]])
@pytest.mark.parametrize("magnitude", [1e-12, 1e-4, 1e5, 1e20])
def test_attention8_float32_queries_of_any_magnitude(magnitude, lengths):
    """Float32 queries far outside binary16's range, the scale bringing the
    scores back; and key scales as far."""
    kc, vc, ks, vs, q, start, lens, table = inputs8(lengths, 4, 2, 128, 16, False, 21)
    scale = float(np.float32(0.088 / magnitude))
    for kk, qq in ((ks, (q * np.float32(magnitude)).astype(np.float32)),
                   ((ks * np.float32(magnitude)).astype(np.float32), q)):
        ref, absolute, score = attend8(kc, vc, kk, vs, qq, start, lens, table, 0, 0, scale)
        y = q4.attention(q4.kv_cache8(*(dev(a) for a in (kc, vc, kk, vs))), dev(qq), dev(start),
                         dev(lens), dev(table), scale=scale)
        near(y, ref, tol8(ref, absolute, score, 300, 128, False))


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("gap", [3.0, 14.0, 18.0])
def test_attention8_many_faint_weights_beside_a_strong_one(gap, half):
    """The first key takes most of the weight, 40000 equal ones share the rest:
    their sum, a known value, has to survive."""
    n, dim = 40001, 64
    page, pages = 256, 160
    kc, vc = (torch.zeros(pages, 1, page, dim, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, 1, page), x, device=DEV) for x in (8.0 / 127, 1.0 / 64))
    kc[0, 0, 0, 0] = 127
    vc[:, 0, :, 1] = 64
    vc[0, 0, 0, 1] = -64
    q = torch.zeros(1, 2, dim, dtype=torch.float16 if half else torch.float32, device=DEV)
    q[:, :, 0] = gap
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    y = q4.attention(q4.kv_cache8(kc, vc, ks, vs), q, i32(0, 1), i32(n), table, scale=0.125)
    score = float(ks[0, 0, 0]) * 127 * 0.125 * float(q[0, 0, 0])
    faint = (n - 1) * np.exp(-score)
    want = (faint - 1.0) / (faint + 1.0)
    tol = 2.0 ** -16 * 4 + n * H32 * 2
    assert (y[0, :, 1].double() - want).abs().max() < tol + abs(want) * H16 * half
    assert (y[0, :, 2:] == 0).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,heads,rows", [(256, 48, 64), (1024, 32, 128), (1, 4, 32)])
def test_attention8_faint_weights_of_many_keys(new, heads, rows, dim):
    """One strong key of weight 1 and value 1 among 20000 of weight 2^-24.5 and value -1:
    each alone is less than half a step of the sums, all of them are 8e-4."""
    keys, page, gap = 20000, 64, 24.5
    pages = (keys + page - 1) // page
    kc = torch.zeros(pages, heads, page, dim, dtype=torch.int8, device=DEV)
    vc = torch.full_like(kc, -1)
    kc[0, :, 5, 0], vc[0, :, 5] = 127, 1
    one = torch.ones(pages, heads, page, device=DEV)
    q = torch.zeros(new, heads, dim, device=DEV)
    q[:, :, 0] = gap / np.log2(np.e) / 127
    c = q4.kv_cache8(kc, vc, one, one.clone())
    assert q4.q4_0_select_attention8(c, heads, q4.F32, new, pages, 1) == rows
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    y = q4.attention(c, q, i32(0, new), i32(keys),
                     torch.arange(pages, dtype=torch.int32, device=DEV)[None], scale=1.0)
    faint = np.exp(-127 * float(q[0, 0, 0])) * np.arange(keys - new, keys)
    want = ((1 - faint) / (1 + faint))[:, None, None]
    # sums beside the strong key's: at most 96 tiles of 64 keys, each four products of two
    # parts (off by a step, 2^-23, at most) and a sum (2^-24); then a dozen such sums
    near(y, np.broadcast_to(want, y.shape), (96 * (8 * 2 + 1) + 24 + gap * 2) * H32 * np.ones(y.shape))


@pytest.mark.parametrize("half", [True, False])
def test_attention8_rows_that_see_nothing(half):
    check8([(10, 4), (3, 0), (1, 0), (40, 20), (2, 2)], 4, 2, 64, 16, 0, 0, half, seed=8)
    check8([(10, 4), (3, 0), (1, 0), (40, 20), (2, 2)], 4, 2, 64, 16, 3, 2, half, seed=8)
    check8([(4, 2), (3, 0), (1, 0), (2, 2)], 4, 2, 64, 16, 0, 0, half, seed=8)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("lengths", [[(1, 2000)], [(1, 1999), (1, 40)], [(4, 1500)], [(70, 1400)],
                                     [(6, 1300)]])
def test_attention8_long_axis(lengths, half):
    """Few rows and many keys: the key axis is split."""
    check8(lengths, 8, 2, 64, 16, 0, 0, half, seed=11)
    check8(lengths, 8, 2, 64, 16, 700, 40, half, seed=12, spread=2.0)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("count", [1, 2, 63, 64, 65])
def test_attention8_conversations_of_many_lengths(count, half):
    """Few rows to a conversation on average, several tiles of them to some; equal
    lengths, empty conversations, rows that see nothing."""
    rng = np.random.default_rng([13, count])
    kvs = rng.choice([0, 1, 5, 33, 64, 65, 130, 130, 190], count)
    news = [int(rng.choice([0, 1, 1, 2])) for _ in range(count)]
    for s in range(0, count, 7):
        news[s], kvs[s] = (6, 40, 20)[s % 3], max(kvs[s], 1)
    if count > 16:
        news[15], kvs[15] = 33, 12
    assert sum(news) * 4 <= 32 * count or count < 3
    check8([(n, int(kv)) for n, kv in zip(news, kvs)], 8, 2, 64, 16, 0, 0, half, seed=count)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention8_full_device_of_long_contexts(dim, half):
    """More conversations' heads than units and long tables: a workgroup of twice the
    waves to each, the longest first, no parts."""
    heads = 16 if dim > 128 else 8
    lengths = [(1 + i % 2, 40 + (53 * i) % 333) for i in range(45)] + [(1, 2100), (3, 1500)]
    c = q4.q4_0_kv_cache8(0, 0, 0, 0, 1, heads, 64, dim)
    assert q4.q4_0_attention8_workspace_size(c, heads, q4.F16 if half else q4.F32,
                                             sum(n for n, _ in lengths), 33, len(lengths)) == 0
    check8(lengths, heads, heads, dim, 64, 0, 0, half, seed=dim)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention8_parts_of_many_rows(dim, half):
    """Enough rows that a wave joins a row's parts, some of which see none of its
    keys; conversations that are empty or see nothing among them."""
    lengths = [(8, 900 - 31 * i) for i in range(13)] + [(0, 0), (8, 3), (5, 0), (8, 70)]
    hq, hk = 16, 2
    c = q4.q4_0_kv_cache8(0, 0, 0, 0, 1, hk, 16, dim)
    call = (hq, q4.F16 if half else q4.F32, sum(n for n, _ in lengths), 57, len(lengths))
    rows = call[2] * hq
    assert rows >= 1024 and q4.q4_0_select_attention8(c, *call) == 32
    assert 2 <= q4.q4_0_attention8_workspace_size(c, *call) // (rows * (dim + 2) * 4) <= 64
    check8(lengths, hq, hk, dim, 16, 0, 0, half, seed=dim)
    check8(lengths, hq, hk, dim, 16, 300, 20, half, seed=dim + 1, spread=2.0)


@pytest.mark.parametrize("count,tokens,longest", [(65, 1, 90), (150, 1, 40), (300, 3, 30),
                                                  (4500, 1, 9), (130, 40, 50)])
def test_attention8_many_conversations(count, tokens, longest):
    """More conversations than one look of 64 lanes finds, empty ones among
    them, and leading tokens that none of them holds."""
    rng = np.random.default_rng(count)
    kvs = rng.integers(0, longest + 1, count)
    news = np.minimum(kvs, rng.integers(0, tokens + 1, count))
    lengths = [(int(a), int(b)) for a, b in zip(news, kvs)]
    kc, vc, ks, vs, q, start, lens, table = inputs8(lengths, 2, 1, 64, 16, True, 5)
    spare = 3
    q = np.concatenate([q[:spare], q])
    start = start + np.int32(spare)
    ref, absolute, score = attend8(kc, vc, ks, vs, q, start, lens, table, 0, 0, 0.125)
    y = torch.full(q.shape, 9.0, dtype=torch.float16, device=DEV)
    q4.attention(q4.kv_cache8(*(dev(a) for a in (kc, vc, ks, vs))), dev(q), dev(start), dev(lens),
                 dev(table), y=y)
    assert (y[:spare] == 9.0).all()
    near(y[spare:], ref[spare:], tol8(ref[spare:], absolute[spare:], score[spare:], longest, 64,
                                      True))


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [50, 6])
def test_attention8_non_finite_scales_in_masked_places(new, dim, half):
    """A row whose scale is no finite number changes the rows that see it and no
    other, though they share its tile."""
    rng = np.random.default_rng(5)
    kv, hq, hk, page, window = 90, 4, 2, 16, 30
    kc, vc = (rng.integers(-127, 128, (6, hk, page, dim)).astype(np.int8) for _ in range(2))
    ks, vs = (np.full((6, hk, page), 0.02, np.float32) for _ in range(2))
    table = np.arange(6, dtype=np.int32)[None]
    q = rng.standard_normal((new, hq, dim)).astype(np.float16 if half else np.float32)
    start, lens = np.array([0, new], np.int32), np.array([kv], np.int32)
    spots = [(vs, 70, np.nan), (ks, 56, np.inf), (vs, 87, -np.inf)] if new == 50 else [
        (vs, 87, np.inf), (ks, 88, np.nan)]
    for c, j, x in spots:
        c[j // page, 1, j % page] = x
    ref, absolute, score = attend8(kc, vc, ks, vs, q, start, lens, table, window, 0, dim ** -0.5)
    y = q4.attention(q4.kv_cache8(*(dev(a) for a in (kc, vc, ks, vs))), dev(q), dev(start),
                     dev(lens), dev(table), window, 0)
    bad = np.isnan(ref)
    assert not bad[:, :2].any() and bad[:, 2:].any() and not bad[:, 2:].all()
    fine = lambda a: np.where(np.isfinite(a), a, 0.0)
    near(y, ref, tol8(fine(ref), fine(absolute), fine(score), kv, dim, half))


@pytest.mark.parametrize("half", [True, False])
def test_attention8_bad_pages_and_tables(half):
    """A row that sees a key on a page outside the cache, or past the table's
    end, is NaN; the rows that do not are untouched."""
    kc, vc, ks, vs, q, start, lens, table = inputs8([(60, 100), (1, 50), (1, 70)], 4, 2, 64, 16,
                                                    half, 2)
    table[0, 4] = 99999                                 # keys 64..79 of the first
    table[1, 1] = -1
    lens[2] = 7 * 16 + 5                                # the table ends at 7 pages
    ks, vs = np.nan_to_num(ks), np.nan_to_num(vs)
    table[2, 5:] = 0
    q = np.concatenate([q, q[:3]])
    ref, absolute, score = attend8(kc, vc, ks, vs, q, start, lens, table, 0, 0, 0.125)
    assert np.isnan(ref[24:62]).all() and np.isfinite(ref[:24]).all()
    cache = q4.kv_cache8(*(dev(a) for a in (kc, vc, ks, vs)))
    y = torch.full(q.shape, 5.0, dtype=torch.float16 if half else torch.float32, device=DEV)
    q4.attention(cache, dev(q), dev(start), dev(lens), dev(table), y=y)
    assert (y[62:] == 5.0).sum() == 3 * 4 * 64
    near(y[:62], ref[:62], tol8(np.nan_to_num(ref[:62]), absolute[:62], score[:62], 120, 64, half))
    # the same conversations' last tokens alone (few rows)
    rows = [59, 60, 61]
    y = q4.attention(cache, dev(q[rows]), i32(0, 1, 2, 3), dev(lens), dev(table))
    assert torch.isnan(y).all()


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("new", [2, 20])
def test_attention8_impossible_lengths(window, new):
    """Lengths far past the table, and negative ones, end as rows of NaN and of
    zeros; the conversation beside them is untouched."""
    kc, vc, ks, vs, q, start, lens, table = inputs8([(new, 40)] * 3, 4, 2, 64, 16, True, 4)
    lens[0], lens[2] = 2 ** 31 - 1, -2 ** 31
    ks, vs = np.nan_to_num(ks), np.nan_to_num(vs)
    y = q4.attention(q4.kv_cache8(*(dev(a) for a in (kc, vc, ks, vs))), dev(q), dev(start),
                     dev(lens), dev(table), window, 1)
    lens[0] = lens[2] = 0
    ref, absolute, score = attend8(kc, vc, ks, vs, q, start, lens, table, window, 1, 0.125)
    assert torch.isnan(y[:new]).all() and (y[2 * new:] == 0).all()
    mid = slice(new, 2 * new)
    near(y[mid], ref[mid], tol8(ref[mid], absolute[mid], score[mid], 40, 64, True))


def test_attention8_offsets_past_32_bits():
    """Pages whose elements lie past 2^32: the same keys on the cache's first and
    last pages give the same result, appended, read and attended to."""
    pages, hk, page, dim = 140000, 1, 256, 128         # 4.6e9 elements each
    if torch.cuda.mem_get_info()[0] < 24 * 2 ** 30:
        pytest.skip("needs 24 GiB of device memory")
    kc = torch.zeros(pages, hk, page, dim, dtype=torch.int8, device=DEV)
    vc = torch.zeros_like(kc)
    ks = torch.zeros(pages, hk, page, device=DEV)
    vs = torch.zeros_like(ks)
    k = torch.randn(700, 1, dim, device=DEV)
    cache, inv = q4.kv_cache8(kc, vc, ks, vs), torch.ones(8, device=DEV)
    at = torch.arange(700, device=DEV)
    for new in (1, 60):
        q = torch.randn(new, 4, dim, device=DEV)
        got = []
        for first in (0, pages - 3):
            q4.kv_append(cache, q4.rotary(inv), None, k, -k, at.int(), first * page + at)
            table = torch.arange(first, first + 3, dtype=torch.int32, device=DEV)[None]
            got.append((q4.attention(cache, q, i32(0, new), i32(700), table),
                        *q4.kv_read(cache, first * page + at)))
        torch.cuda.synchronize()
        assert torch.equal(kc[:3], kc[-3:]) and torch.equal(vs[:3], vs[-3:])
        assert kc[:3].abs().sum() > 0
        for a, b in zip(*got):
            assert torch.equal(a, b) and a.abs().sum() > 0


def test_attention8_of_a_whole_text_is_that_of_its_steps():
    """Appended and attended to token by token, in steps of drafts and in one pass:
    the same rows, within the roundings of weights."""
    torch.manual_seed(2)
    n, hq, hk, dim = 90, 8, 2, 128
    rows = [torch.randn(n, h, dim, device=DEV) for h in (hq, hk, hk)]
    shape = (6, hk, 16, dim)
    table = i32(3, 1, 5, 0, 4, 2)[None]
    inv = 100.0 ** (-torch.arange(0, dim, 2, device=DEV) / dim)
    outs = []
    for steps in ([n], [60] + [1] * 30, [50] + [5] * 8):
        cache = q4.kv_cache8(*(torch.zeros(shape, dtype=torch.int8, device=DEV) for _ in range(2)),
                             *(torch.zeros(shape[:3], device=DEV) for _ in range(2)))
        ys, at = [], 0
        for m in steps:
            pos = torch.arange(at, at + m, device=DEV)
            slots = table[0, pos // 16].long() * 16 + pos % 16
            q = q4.kv_append(cache, q4.rotary(inv), *(r[at:at + m] for r in rows), pos.int(), slots)
            ys.append(q4.attention(cache, q, i32(0, m), i32(at + m), table))
            at += m
        outs.append(torch.cat(ys))
    for y in outs[1:]:
        assert float((y - outs[0]).norm() / outs[0].norm()) < 2.0 ** -20


# ---- the table's lookup ------------------------------------------------------
@pytest.mark.parametrize("norm,half", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("out,in_,n", [(1, 32, 3), (17, 96, 40), (300, 160, 7), (64, 2560, 5),
                                       (40, 16384, 3), (33, 16416, 4), (20, 32768, 2)])
def test_embed(out, in_, n, norm, half):
    rng = np.random.default_rng(out)
    blocks = synth.make_blocks(out, in_, seed=out)
    table = oracle.dequantize(blocks, out, in_)
    tokens = rng.integers(0, out, n).astype(np.int32)
    tokens[0] = out - 1
    if n > 3:
        tokens[1], tokens[2], tokens[3] = -1, out, tokens[0]
    pre = (1 + 0.1 * rng.standard_normal(in_)).astype(np.float32)
    scale = float(np.float32(in_ ** 0.5))
    packed = q4.repacked(dev(blocks.reshape(-1)), out, in_)
    h, y = q4.embed(packed, dev(tokens), out, in_, scale=scale, pre=dev(pre) if norm else None,
                    eps=1e-5, weight_offset=0.5, y_dtype=torch.float16 if half else torch.float32)
    want = step.rows(table, tokens, scale)
    near(h, want, np.abs(want) * H32)
    if not norm:
        assert y is None
        return
    ref = block.rms_norm(want, pre, 1e-5, 0.5)
    # the norm's factor: a sum of in_ squares and a root, halved by the root
    near(y, ref, np.abs(ref) * ((in_ / 2 + 14) * H32 + (H16 if half else 0.0)) + 2.0 ** -25)


def test_embed_many_tokens_and_given_outputs():
    out, in_, n = 301, 64, 65536
    blocks = synth.make_blocks(out, in_, seed=4)
    table = torch.from_numpy(oracle.dequantize(blocks, out, in_)).to(DEV)
    packed = q4.repacked(dev(blocks.reshape(-1)), out, in_)
    tokens = torch.randint(0, out, (n,), dtype=torch.int32, device=DEV)
    h = torch.empty(n, in_, device=DEV)
    y = torch.empty(n, in_, dtype=torch.float16, device=DEV)
    pre = torch.ones(in_, device=DEV)
    assert q4.embed(packed, tokens, out, in_, scale=-3.0, h=h)[0] is h
    assert torch.equal(h, table[tokens.long()] * -3.0)
    got = q4.embed(packed, tokens, out, in_, pre=pre, y=y)
    assert got[1] is y and torch.equal(got[0], table[tokens.long()])
    assert torch.equal(y, q4.residual_norm(got[0], pre=pre, y_dtype=torch.float16)[1])


# ---- verification ------------------------------------------------------------
def check_verify(logits, tokens, start, uniform, drafted=None, heat=None, pad=0):
    def wide(x):
        if x is None or not pad:
            return None if x is None else dev(x)
        t = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), device=DEV, dtype=dev(x).dtype)
        t[:, :x.shape[1]] = dev(x)
        return t[:, :x.shape[1]]
    want = step.verify(logits, tokens, start, uniform, drafted, heat)
    call = (wide(logits), dev(tokens), dev(start), dev(uniform), wide(drafted),
            None if heat is None else dev(heat))
    got = q4.verify(*call)
    assert got[0].tolist() == want[0].tolist()
    assert got[1].tolist() == want[1].tolist()
    again = q4.verify(*call)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    return want


def drafts(rng, rows, vocab, half, modelled, spread=2.0):
    """Logits whose likely tokens stand out, drafts that are often right."""
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    n, dt = int(start[-1]), np.float16 if half else np.float32
    logits = (spread * rng.standard_normal((n, vocab))).astype(dt)
    drafted = (logits + 0.7 * rng.standard_normal((n, vocab))).astype(dt)
    source = (drafted if modelled else logits).astype(float)
    tokens = np.zeros(n, np.int32)
    tokens[1:] = (source + rng.gumbel(size=source.shape) * 0.7).argmax(-1)[:-1]
    uniform = rng.random((n, 2)).astype(np.float32)
    return logits, tokens, start, uniform, drafted if modelled else None


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("modelled", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 3, 63, 1000, 8191, 8192, 8193, 32003, 70000])
def test_verify(vocab, modelled, half):
    rng = np.random.default_rng([vocab, modelled, half])
    rows = [1, 5, 0, 3, 9, 2, 0, 17, 4]
    logits, tokens, start, uniform, drafted = drafts(rng, rows, vocab, half, modelled)
    heat = np.array([1.0, 0.7, 1.0, 0.0, 1.5, 0.05, 1.0, 0.9, -1.0], np.float32)
    a, _ = check_verify(logits, tokens, start, uniform, drafted, heat, pad=3)
    # (picks among many tokens of like weight are hardly ever taken)
    assert vocab < 3 or not modelled or 0 < a.sum() < sum(rows)
    check_verify(logits, tokens, start, uniform, drafted)


@pytest.mark.parametrize("modelled", [False, True])
def test_verify_many_conversations(modelled):
    """More conversations than one look of 64 lanes finds, and more conversations
    than rows; leading and trailing rows that none of them holds."""
    rng = np.random.default_rng(7)
    for count in (65, 300):
        rows = rng.integers(0, 4, count)
        rows[0] = 2
        logits, tokens, start, uniform, drafted = drafts(rng, [3, *rows, 2], 50, False, modelled)
        check_verify(logits, tokens, start[1:-1], uniform, drafted,
                     rng.choice([0.0, 0.5, 1.0], count).astype(np.float32))
    empty = np.zeros(400, np.int32)
    logits, tokens, start, uniform, drafted = drafts(rng, [3], 50, False, modelled)
    empty[200:] = 3
    check_verify(logits, tokens, empty, uniform, drafted)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("modelled", [False, True])
def test_verify_many_parts(modelled, half):
    """More than 2048 parts, a wave to each: conversations that draw, that take the
    greatest, and whose rows are no distribution."""
    rng = np.random.default_rng([11, modelled, half])
    rows = [4, 1, 7, 3] * (5 if modelled else 9)
    logits, tokens, start, uniform, drafted = drafts(rng, rows, 33001, half, modelled)
    assert logits.shape[0] * (2 if modelled else 1) * 17 > 2048
    heat = np.tile(np.array([1.0, 0.8, 0.0, 1.2, 0.6, 0.9], np.float32), 6)[:len(rows)]
    check_verify(logits, tokens, start, uniform, drafted, heat, pad=5)
    for s in range(0, len(rows), 3):
        logits[start[s], rng.integers(0, 33001)] = [np.nan, np.inf][s % 2]
    logits[start[7]] = -np.inf
    logits[start[8], 100:] = -np.inf
    _, t = check_verify(logits, tokens, start, uniform, drafted, heat)
    assert (t == -1).sum() > len(rows) // 3


@pytest.mark.parametrize("modelled", [False, True])
def test_verify_more_parts_than_lanes_hold(modelled):
    """Vocabularies past 262144 tokens; what is drawn lies in the last parts too."""
    rng = np.random.default_rng([12, modelled])
    for heat in (1.0, 3.0, 0.0):
        logits, tokens, start, uniform, drafted = drafts(rng, [3, 1, 4], 300007, False, modelled)
        logits[:, 290000:] += 1.5
        check_verify(logits, tokens, start, uniform, drafted, np.full(3, heat, np.float32))


def test_verify_borders():
    """Equal weights, whose cumulative sums are whole numbers: a number that
    falls on a border takes the token after it; 0, numbers from 1 on, below 0
    and NaN."""
    vocab = 16
    us = [k / 16 for k in range(17)] + [1.0 - 2.0 ** -24, 2.0, -1.0, float("nan")]
    n = len(us)
    logits = np.full((n, vocab), -3.5, np.float32)
    uniform = np.zeros((n, 2), np.float32)
    uniform[:, 1] = us
    a, t = check_verify(logits, np.zeros(n, np.int32), np.arange(n + 1, dtype=np.int32), uniform)
    assert t.tolist() == list(range(16)) + [15, 15, 15, 0, 15]
    # excluded tokens are never drawn, whatever the number
    logits[:, [0, 5, 15]] = -np.inf
    uniform[:, 1] = [0.0] * 10 + [2.0] * (n - 10)
    a, t = check_verify(logits, np.zeros(n, np.int32), np.arange(n + 1, dtype=np.int32), uniform)
    assert set(t.tolist()) == {1, 14}


def test_verify_acceptance_borders():
    """u q(d) < p(d) with p(d) a quarter: at a quarter the draft is refused, and it is
    never drawn again; a certain draft is always taken."""
    n = 2 * 4
    logits = np.zeros((n, 4), np.float32)
    start = np.arange(0, n + 1, 2, dtype=np.int32)
    tokens = np.tile([0, 2], 4).astype(np.int32)
    uniform = np.zeros((n, 2), np.float32)
    uniform[::2, 0] = [0.0, 0.25 - 2.0 ** -26, 0.25, 0.9]
    uniform[::2, 1] = 0.5
    a, t = check_verify(logits, tokens, start, uniform)
    assert a.tolist() == [1, 1, 0, 0] and t.tolist() == [0, 0, 1, 1]
    logits[:] = -np.inf
    logits[:, 2] = 1.0
    uniform[::2, 0] = [0.0, 0.5, 1.0 - 2.0 ** -24, 0.9]
    a, t = check_verify(logits, tokens, start, uniform)
    assert a.tolist() == [1] * 4 and t.tolist() == [2] * 4
    # refused all the same (a number above 1): there is nothing else to draw
    uniform[::2, 0] = 1.5
    assert check_verify(logits, tokens, start, uniform)[1].tolist() == [2] * 4


@pytest.mark.parametrize("modelled", [False, True])
def test_verify_equal_distributions_and_strange_drafts(modelled):
    """A draft model equal to the target is taken whatever the numbers below 1;
    drafts outside the vocabulary are refused and nothing is taken from p."""
    rng = np.random.default_rng(1)
    logits, tokens, start, uniform, _ = drafts(rng, [5, 4], 300, False, modelled)
    drafted = logits.copy() if modelled else None
    a, _ = check_verify(logits, tokens, start, uniform, drafted)
    assert not modelled or a.tolist() == [4, 3]
    for bad in (-1, 300, 2 ** 31 - 1, -2 ** 31):
        tokens[2], tokens[6] = bad, bad
        a, _ = check_verify(logits, tokens, start, uniform, drafted)
        assert a.tolist()[0] <= 1
        check_verify(logits, tokens, start, uniform, drafted, np.zeros(2, np.float32))


@pytest.mark.parametrize("modelled", [False, True])
@pytest.mark.parametrize("bad", [np.nan, np.inf, "empty"])
def test_verify_rows_that_are_no_distribution(bad, modelled):
    """They end the step when they are reached, and only then."""
    rng = np.random.default_rng(4)
    logits, tokens, start, uniform, drafted = drafts(rng, [4] * 30, 9000, False, modelled)
    for s in range(30):
        for x in (logits, drafted)[:1 + (modelled and s % 3 == 0)]:
            row = start[s] + s % 4
            if bad == "empty":
                x[row] = -np.inf
            else:
                x[row, rng.integers(0, 9000)] = bad
    for heat in (None, np.zeros(30, np.float32)):
        a, t = check_verify(logits, tokens, start, uniform, drafted, heat)
        assert (t == -1).any() and (t >= 0).any()


def test_verify_greedy_ties():
    """The lowest of equal greatest logits, within a part and across parts."""
    n, vocab = 6, 20000
    logits = np.zeros((n, vocab), np.float16)
    for t, at in enumerate([(5, 9), (8191, 8192), (19999,), (100, 16384), (0, 19999), (8192, 8193)]):
        logits[t, list(at)] = 3.0
    first = np.arange(n + 1, dtype=np.int32)
    zero = np.zeros(n, np.float32)
    _, t = check_verify(logits, np.zeros(n, np.int32), first, np.zeros((n, 2), np.float32), None, zero)
    assert t.tolist() == [5, 8191, 19999, 100, 0, 8192]
    tokens = np.array([1, 5, 8191, 19999, 100, 1], np.int32)
    a, t = check_verify(logits, tokens, np.array([0, n], np.int32), np.ones((n, 2), np.float32), None,
                        zero[:1])
    assert a.tolist() == [4] and t.tolist() == [0]


@pytest.mark.parametrize("heat", [1e-30, 1e-3, 30.0, 1e6])
@pytest.mark.parametrize("modelled", [False, True])
def test_verify_extreme_temperatures_and_logits(heat, modelled):
    rng = np.random.default_rng(8)
    for spread in (1e-3, 1e4):
        args = list(drafts(rng, [3] * 20, 5000, False, modelled, spread))
        args[0][::3] += np.float32(1e6)
        check_verify(*args, np.full(20, heat, np.float32))


def test_verify_draws_follow_the_weights():
    """Every token's share of many evenly spaced numbers, over several parts."""
    rng = np.random.default_rng(6)
    vocab, n = 20011, 4096
    row = (3.0 * rng.standard_normal(vocab)).astype(np.float32)
    u = torch.zeros(n, 2, device=DEV)
    u[:, 1] = (torch.arange(n, device=DEV) + 0.5) / n
    logits = dev(row)[None].expand(n, vocab)
    _, t = q4.verify(logits.contiguous(), torch.zeros(n, dtype=torch.int32, device=DEV),
                     torch.arange(n + 1, dtype=torch.int32, device=DEV), u)
    p = np.exp(row.astype(np.float64) - row.max())
    below = np.cumsum(p) / p.sum()
    want = np.searchsorted(below, (np.arange(n) + 0.5) / n, side="right")
    assert np.array_equal(t.cpu().numpy(), want)


# ---- together, streams, graphs -----------------------------------------------
def load_example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 2)])
def test_drafted_steps_of_a_served_block(window, sinks):
    """Ids in, ids out: lookup, a block over an 8-bit cache, the tied logit head,
    verification; a captured step of 1 + 4 tokens a conversation, replayed.
    Greedily, right drafts are taken up to the first wrong one, and the tokens are
    those that one token a step draws."""
    example = load_example()
    torch.manual_seed(5)
    vocab, width, page, batch, m = 500, 256, 16, 3, 5
    blk = example.Block(width, 4, 2, 64, 512, seed=3, window=window, sinks=sinks)
    blocks = synth.make_blocks(vocab, width, seed=77)
    head = q4.repacked(dev(blocks.reshape(-1)), vocab, width)
    pages, lens0 = 8, [21, 3, 40]
    table = torch.randperm(batch * pages, device=DEV).int().view(batch, pages)
    shape = (batch * pages, 2, page, 64)

    def new_cache():
        return q4.kv_cache8(*(torch.zeros(shape, dtype=torch.int8, device=DEV) for _ in range(2)),
                            *(torch.zeros(shape[:3], device=DEV) for _ in range(2)))

    def logits_of(tokens, cache, place):
        h, x = q4.embed(head, tokens, vocab, width, scale=width ** 0.5, pre=blk.norms["next"])
        _, x = blk(h, x, cache, place)
        return q4.matmul(head, x, vocab)

    def prefill(cache):
        n = sum(lens0)
        place = example.new_batch(n, table)
        example.place(place, lens0, lens0, page)
        tokens = torch.arange(n, device=DEV).int() * 7 % vocab
        logits = logits_of(tokens, cache, place)
        ends = torch.tensor(lens0).cumsum(0) - 1
        return logits[ends.to(DEV)].argmax(-1).tolist()

    uniform = torch.rand(batch * m, 2, device=DEV)
    cold = torch.zeros(batch, device=DEV)

    # one token a step
    cache = new_cache()
    drawn = [[t] for t in prefill(cache)]
    place = example.new_batch(batch, table)
    for i in range(14):
        example.place(place, [1] * batch, [n + i + 1 for n in lens0], page)
        last = i32(*(d[-1] for d in drawn))
        logits = logits_of(last, cache, place)
        a, t = q4.verify(logits, last, place["q_start"], uniform[:batch], temperature=cold)
        assert a.tolist() == [0] * batch
        top = logits.topk(2).values
        # a near tie might be drawn differently on tiles of other shapes
        assert ((top[:, 0] - top[:, 1]) > 1e-3 * top[:, 0].abs()).all()
        for d, x in zip(drawn, t.tolist()):
            d.append(x)

    # drafted, captured and replayed
    cache = new_cache()
    assert [d[0] for d in drawn] == prefill(cache)
    place = example.new_batch(batch * m, table)
    tokens = torch.zeros(batch * m, dtype=torch.int32, device=DEV)
    out = {}

    def one():
        out["logits"] = logits_of(tokens, cache, place)
        out["a"], out["t"] = q4.verify(out["logits"], tokens, place["q_start"], uniform,
                                       temperature=cold)

    have = [1] * batch
    wrong = [[4, 2, 1], [0, 4, 3], [4, 1, 4]]          # the first wrong draft of each step
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    example.place(place, [m] * batch, [n + m for n in lens0], page)
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    captured = dict(out)
    for first in wrong:
        new = []
        for s in range(batch):
            d = drawn[s][have[s] - 1:have[s] - 1 + m]
            if first[s] < m - 1:
                d[1 + first[s]] = (d[1 + first[s]] + 1) % vocab
            new += d
        tokens.copy_(i32(*new))
        example.place(place, [m] * batch, [n + h - 1 + m for n, h in zip(lens0, have)], page)
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in captured.items()}
        one()                                          # the same rows once more, eagerly
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], out[k]), k
        want = [min(f, m - 1) for f in first]
        assert got["a"].tolist() == want
        for s in range(batch):
            assert got["t"][s].item() == drawn[s][have[s] + want[s]]
            have[s] += want[s] + 1


def step_calls():
    """A run of all of them on caller-owned buffers: (call, its outputs)."""
    torch.manual_seed(1)
    n, hq, hk, dim, width, vocab = 6, 8, 2, 128, 40, 9001
    kc, vc = (torch.randint(-127, 128, (3 * width, hk, 16, dim), dtype=torch.int8, device=DEV)
              for _ in range(2))
    ks, vs = (0.01 + 0.02 * torch.rand(3 * width, hk, 16, device=DEV) for _ in range(2))
    cache, rot = q4.kv_cache8(kc, vc, ks, vs), q4.rotary(torch.rand(dim // 2, device=DEV))
    table = torch.randperm(3 * width, device=DEV).int().view(3, width)
    start, lens = i32(0, 1, 4, 6), i32(600, 17, 301)
    pos = i32(599, 14, 15, 16, 299, 300)
    owner = torch.tensor([0, 1, 1, 1, 2, 2], device=DEV)
    slots = table[owner, (pos // 16).long()].long() * 16 + pos % 16
    tokens = torch.randint(0, vocab, (n,), dtype=torch.int32, device=DEV)
    packed = q4.repacked(dev(synth.make_blocks(vocab, 256, seed=1).reshape(-1)), vocab, 256)
    qkv = torch.randn(n, (hq + 2 * hk) * dim, device=DEV)
    q16 = torch.randn(n, hq, dim, device=DEV).half()
    logits, drafted = (2 * torch.randn(n, vocab, device=DEV) for _ in range(2))
    uniform, heat = torch.rand(n, 2, device=DEV), torch.tensor([1.0, 0.5, 0.0], device=DEV)
    pre = torch.ones(256, device=DEV)
    out = {"h": torch.empty(n, 256, device=DEV), "x": torch.empty(n, 256, device=DEV),
           "q": torch.empty(n, hq, dim, device=DEV), "y": torch.empty(n, hq, dim, device=DEV),
           "y16": torch.empty(n, hq, dim, device=DEV).half(),
           "k": torch.empty(n, hk, dim, device=DEV), "v": torch.empty(n, hk, dim, device=DEV),
           "a": torch.empty(3, dtype=torch.int32, device=DEV),
           "t": torch.empty(3, dtype=torch.int32, device=DEV),
           "a1": torch.empty(3, dtype=torch.int32, device=DEV),
           "t1": torch.empty(3, dtype=torch.int32, device=DEV)}

    def call(ws, o=out, **kw):
        q4.embed(packed, tokens, vocab, 256, scale=2.0, pre=pre, h=o["h"], y=o["x"], **kw)
        q4.kv_append(cache, rot, *qkv.split([hq * dim, hk * dim, hk * dim], dim=1), pos, slots,
                     q_out=o["q"], **kw)
        q4.kv_read(cache, slots, k=o["k"], v=o["v"], **kw)
        q4.attention(cache, o["q"], start, lens, table, y=o["y"], ws=ws, **kw)
        q4.attention(cache, q16, start, lens, table, window=200, sinks=4, y=o["y16"], ws=ws, **kw)
        q4.verify(logits, tokens, start, uniform, draft_logits=drafted, temperature=heat,
                  accepted=o["a"], following=o["t"], ws=ws, **kw)
        q4.verify(logits, tokens, start, uniform, accepted=o["a1"], following=o["t1"], ws=ws, **kw)

    return call, out


def new_ws(fill=0):
    return torch.full((q4.WORKSPACE_MAX,), fill, dtype=torch.uint8, device=DEV)


def test_step_operators_allocate_nothing_and_take_any_workspace():
    call, out = step_calls()
    ws = new_ws()
    call(ws)
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in out.items()}
    before = torch.cuda.mem_get_info()[0]
    for fill in (255, 127):
        ws.fill_(fill)
        for o in out.values():
            o.zero_()
        call(ws)
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], want[k]), k
    assert torch.cuda.mem_get_info()[0] == before


@pytest.mark.parametrize("handle", [False, True])
def test_step_operators_on_two_streams_at_once(handle):
    """Two streams with their own outputs and workspaces, many calls in flight."""
    call, out = step_calls()
    call(new_ws())
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    sets = [({k: torch.zeros_like(v) for k, v in out.items()}, new_ws()) for _ in sides]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (o, ws) in zip(sides, sets):
            call(ws, o, stream=s.cuda_stream if handle else s)
    torch.cuda.synchronize()
    for o, _ in sets:
        for k in out:
            assert torch.equal(o[k], out[k]), k


def test_conveniences_allocate_on_a_given_stream():
    """Outputs and workspaces that a call on another stream allocates are not
    given away before it has run."""
    torch.manual_seed(3)
    kc, vc = (torch.randint(-9, 9, (300, 2, 16, 64), dtype=torch.int8, device=DEV) for _ in range(2))
    cache = q4.kv_cache8(kc, vc, *(torch.rand(300, 2, 16, device=DEV) for _ in range(2)))
    q, table = torch.randn(1, 4, 64, device=DEV), torch.arange(300, device=DEV).int()[None]
    logits, tokens, uni = torch.randn(3, 30000, device=DEV), i32(1, 2, 3), torch.rand(3, 2, device=DEV)
    start, slots, lens, one = i32(0, 3), torch.arange(9, device=DEV), i32(4700), i32(0, 1)
    packed = q4.repacked(dev(synth.make_blocks(20, 64, seed=1).reshape(-1)), 20, 64)
    pre = torch.ones(64, device=DEV)

    def calls(**kw):
        return (q4.attention(cache, q, one, lens, table, **kw), *q4.kv_read(cache, slots, **kw),
                *q4.verify(logits, tokens, start, uni, draft_logits=logits, **kw),
                *q4.embed(packed, tokens, 20, 64, pre=pre, **kw))
    want = calls()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append(calls(stream=side))
        for size in (1 << 12, 1 << 16, 1 << 20):
            torch.empty(size, dtype=torch.uint8, device=DEV).fill_(255)
        side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_step_calls_refuse_tensors_on_the_host():
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.int8, device=DEV)
    s = torch.zeros(2, 2, 16, device=DEV)
    with pytest.raises(ValueError, match="different devices"):
        q4.kv_cache8(kc, kc.clone(), s, s.cpu())
    c = q4.kv_cache8(kc, kc.clone(), s, s.clone())
    with pytest.raises(ValueError):
        q4.kv_read(c, torch.zeros(3, dtype=torch.int64))
    q = torch.zeros(1, 4, 64, device=DEV)
    with pytest.raises(ValueError):
        q4.attention(c, q, i32(0, 1), torch.tensor([1], dtype=torch.int32),
                     torch.zeros(1, 2, dtype=torch.int32, device=DEV))
    packed = torch.zeros(q4.q4_0_packed_bytes(20, 64), dtype=torch.uint8)
    with pytest.raises(ValueError):
        q4.embed(packed, i32(1), 20, 64)
    with pytest.raises(ValueError):
        q4.verify(torch.zeros(1, 9, device=DEV), i32(1), i32(0, 1), torch.zeros(1, 2))


def test_first_calls_of_a_process_capture_into_a_graph():
    import json
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "cold_capture_step.py")],
                       capture_output=True, text=True, timeout=100)
    print(r.stdout[-2000:], r.stderr[-2000:], flush=True)
    assert r.returncode == 0
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(res) == 11 and all(res.values()), res
