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
from test_gpu_block import DEV, H16, H32, append_tol, attention_tol, batch_inputs, dev, near

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
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, 0, 0,
                                        float(np.float32(scale)))
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


# ---- attention: 128-row tiles -------------------------------------------------
HEADS_128 = 64      # key/value heads, one query head each: a few hundred tokens fill the device


def by_128(lengths, dim, half, window=0, sinks=0, seed=0, change=None, q_scale=1.0):
    """A call on 128-row tiles against the oracle.  change(kc, vc, table, lens)
    plants what the call has to bear."""
    kc, vc, q, start, lens, table = batch_inputs(lengths, HEADS_128, HEADS_128, dim, 16, half, seed,
                                                 window, sinks, q_scale)
    n, scale = q.shape[0], dim ** -0.5
    if change:
        change(kc, vc, table, lens)
    assert q4.q4_0_select_attention(q4.q4_0_kv_cache(0, 0, len(kc), HEADS_128, 16, dim), HEADS_128,
                                    q4.F16 if half else q4.F32, n, table.shape[1], len(lengths),
                                    window, sinks) == 128
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, window, sinks, scale)
    y = attend(kc, vc, q, start, lens, table, window, sinks, scale)
    keys = max(kv for _, kv in lengths)
    clean = lambda a: np.where(np.isfinite(a), a, 0.0)
    near(y, ref, attention_tol(clean(ref), clean(absolute), clean(score), keys, dim, half))
    assert torch.equal(y.nan_to_num(), attend(kc, vc, q, start, lens, table, window, sinks,
                                              scale).nan_to_num())
    return ref


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_128_row_tiles(dim, half):
    """Long passes: conversations that start and end inside a tile, one of one
    token, one behind a cache, and rows that see nothing."""
    by_128([(200, 200), (1, 77), (130, 150), (61, 64), (0, 9), (9, 4)], dim, half, seed=dim)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(70, 5), (17, 130)])
def test_attention_128_row_tiles_window(window, sinks, dim, half):
    by_128([(140, 290), (150, 150), (3, 2), (110, 112)], dim, half, window, sinks, seed=window)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_128_row_tiles_bad_pages(dim, half):
    """A page outside the cache and a table that ends too early: the rows that
    see such keys are NaN, the others are not touched."""
    def change(kc, vc, table, lens):
        kc[np.isnan(kc)], vc[np.isnan(vc)] = 0, 0
        table[0, 6] = len(kc)                             # keys 96..111
        table[1] = 0
        lens[1] = 16 * table.shape[1] + 40
    ref = by_128([(190, 190), (140, 140), (20, 20)], dim, half, seed=5, change=change)
    assert np.isfinite(ref[:96]).all() and np.isnan(ref[96:190]).all()
    assert np.isnan(ref[329]).all() and np.isfinite(ref[330:]).all()


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_128_row_tiles_non_finite(dim, half):
    """Infinities and NaN of keys and values stay with the rows that see them,
    though a tile's other rows share the product."""
    spots = [(1, 150, 3, np.inf), (1, 151, 3, np.inf), (1, 100, 5, -np.inf), (1, 60, 9, np.nan),
             (0, 170, 1, np.nan), (1, 175, 7, np.inf), (1, 176, 7, -np.inf)]

    def change(kc, vc, table, lens):
        for which, j, d, x in spots:
            (kc, vc)[which][table[0, j // 16], 1, j % 16, d] = x
    ref = by_128([(200, 200), (140, 160), (50, 50)], dim, half, window=60, seed=6, change=change)
    assert np.isfinite(ref[:, [0, 2]]).all() and not np.isfinite(ref[:200, 1]).all()


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_128_row_tiles_far_scores(dim, half):
    """One head's scores near 2^40: exact ones, so the highest level a row sees
    decides alone."""
    lengths = [(200, 200), (140, 160), (50, 50)]
    rng, kc, vc, start, lens, table = plain(lengths, dim, 9, pages=100)
    assert q4.q4_0_select_attention(q4.q4_0_kv_cache(0, 0, 100, HEADS_128, 16, dim), HEADS_128,
                                    q4.F32, start[-1], table.shape[1], 3) == 128
    level = rng.permutation(1600).reshape(100, 16) - 800.0
    kc, vc = (np.repeat(c[:, :1], HEADS_128, 1) for c in (kc, vc))
    kc[:, 5] = 0
    kc[:, 5, :, 2] = level
    table = np.stack([rng.permutation(100)[:table.shape[1]] for _ in lengths]).astype(np.int32)
    q = rng.standard_normal((start[-1], HEADS_128, dim)).astype(np.float16 if half else np.float32)
    q[:, 5] = 0
    q[:, 5, 2] = 2.0 ** 14
    q[:, :5] = q[:, 6:] = 0
    ref, absolute, _ = block.attend(kc, vc, q, start, lens, table, 0, 0, 2.0 ** 20)
    y = attend(kc, vc, q, start, lens, table, 0, 0, 2.0 ** 20)
    # elsewhere equal weights: each rounded alike, and sums of up to 200 terms
    near(y, ref, np.abs(ref) * (H16 if half else H32) + absolute * 2 * 216 * H32 + 2.0 ** -25)


def test_attention_more_tiles_than_one_launch_takes():
    """More tiles than a grid's third axis: the last ones go in a second launch.
    Few rows to a conversation (most hold none), and one conversation of very
    many rows."""
    batch, width = 65536, 2
    rng, kc, vc, _, _, _ = plain([(1, 1)], 64, 2, pages=40)
    news = np.zeros(batch, np.int64)
    news[[0, 5000, 40000, 65533, 65534, 65535]] = [2, 1, 3, 1, 2, 1]
    lens = np.where(news > 0, 17 + np.arange(batch) % 14, 0).astype(np.int32)
    start = np.concatenate([[0], news.cumsum()]).astype(np.int32)
    table = rng.integers(0, 40, (batch, width)).astype(np.int32)
    q = rng.standard_normal((start[-1], 4, 64)).astype(np.float16)
    y = attend(kc, vc, q, start, lens, table, scale=0.125)
    used = np.flatnonzero(news)
    ref, absolute, score = block.attend(kc, vc, q, np.concatenate([start[used], start[-1:]]),
                                        lens[used], table[used], 0, 0, 0.125)
    near(y, ref, attention_tol(ref, absolute, score, 31, 64, True))

    n, heads, window = 65536, 128, 4
    assert q4.q4_0_select_attention(q4.q4_0_kv_cache(0, 0, 64, 1, 1024, 64), heads, q4.F16, n, 64,
                                    1, window, 0) == 128
    g = torch.Generator(device=DEV).manual_seed(3)
    tk, tv = (torch.randn(64, 1, 1024, 64, device=DEV, generator=g).half() for _ in range(2))
    tq = torch.randn(n, heads, 64, device=DEV, generator=g).half()
    order = torch.randperm(64, device=DEV, generator=g)
    y = q4.attention(q4.kv_cache(tk, tv), tq, torch.tensor([0, n], dtype=torch.int32, device=DEV),
                     torch.tensor([n], dtype=torch.int32, device=DEV), order.int()[None], window)
    pick = torch.cat([torch.tensor([0, 1, 2, 3, n - 2, n - 1]),
                      torch.from_numpy(rng.integers(4, n, 60))])
    k, v = (t[order, 0].reshape(n, 64).double().cpu().numpy() for t in (tk, tv))
    want, absolute, score = (np.zeros((len(pick), heads, 64)), np.zeros((len(pick), heads, 64)),
                             np.zeros((len(pick), heads)))
    qs = tq[pick.to(DEV)].double().cpu().numpy()
    for i, t in enumerate(pick.tolist()):
        js = np.arange(max(0, t - window + 1), t + 1)
        z = qs[i] @ k[js].T / 8
        w = np.exp(z - z.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        want[i], absolute[i] = w @ v[js], w @ np.abs(v[js])
        score[i] = (np.abs(qs[i]) @ np.abs(k[js]).T / 8).max(1)
    near(y[pick.to(DEV)], want, attention_tol(want, absolute, score, window, 64, True))


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("tokens", [1, 40])
@pytest.mark.parametrize("gap", [3.0, 14.0, 18.0])
def test_attention_faint_weights_count(gap, tokens, half):
    """One strong key and 40000 faint equal ones: a row's result is known from
    the faint ones' share f of the strong one's weight.  An error of the faint
    sum, e of it, moves the result (f - 1) / (f + 1) by 2 f e / (f + 1)^2; e is a
    faint weight's rounding (relative, or half of binary16's last step where a
    weight of 2^7 (float32: 2^14) exp(-gap) lies that low), float32 sums of
    40000, and the power's own rounding.  Without the faint keys it would be -1,
    which has to be out of reach."""
    n, dim, page, pages = 40001, 64, 256, 160
    kc, vc = (torch.zeros(pages, 1, page, dim, dtype=torch.float16, device=DEV) for _ in range(2))
    kc[0, 0, 0, 0] = 8.0
    vc[:, 0, :, 1] = 1.0
    vc[0, 0, 0, 1] = -1.0
    q = torch.zeros(tokens, 2, dim, dtype=torch.float16 if half else torch.float32, device=DEV)
    q[:, :, 0] = gap
    i32 = dict(dtype=torch.int32, device=DEV)
    y = q4.attention(q4.kv_cache(kc, vc), q, torch.tensor([0, tokens], **i32),
                     torch.tensor([n], **i32), torch.arange(pages, **i32)[None], scale=0.125)
    f = (n - tokens + np.arange(tokens)) * np.exp(-gap)
    want = (f - 1) / (f + 1)
    weight = 2.0 ** (7 if half else 14) * np.exp(-gap)
    e = max(H16 if half else 2.0 ** -22, 2.0 ** -25 / weight) + 2 * n * H32 + 64 * gap * H32
    tol = 2 * f * e / (f + 1) ** 2 + np.abs(want) * (H16 if half else 4 * H32)
    assert (np.abs(want + 1) > 2 * tol).all()
    got = y[:, :, 1].double().cpu().numpy()
    assert (np.abs(got - want[:, None]) <= tol[:, None]).all(), np.abs(got - want[:, None]).max()
    assert (y[:, :, 0] == 0).all() and (y[:, :, 2:] == 0).all()


# ---- residual norm ------------------------------------------------------------
@pytest.mark.parametrize("dim", [8, 130])
def test_residual_norm_columns_of_one_buffer(dim):
    """h, b, h_out, y and the gate as columns of one buffer: they share its rows
    and no element."""
    n, rng = 5, np.random.default_rng(dim)
    x = rng.standard_normal((n, 5 * dim)).astype(np.float32)
    wide = dev(x)
    h, b, gate, out, y = (wide[:, i * dim:(i + 1) * dim] for i in range(5))
    pre, post = (dev((1 + rng.random(dim)).astype(np.float32)) for _ in range(2))
    got = q4.residual_norm(h, b, pre, post, gate, 0.5, h_out=out, y=y)
    torch.cuda.synchronize()
    rh, ry = block.residual_norm(x[:, :dim], x[:, dim:2 * dim], pre.double().cpu().numpy(),
                                 post.double().cpu().numpy(), x[:, 2 * dim:3 * dim], 0.5)
    # norms and sums of dim terms, a few roundings of each element, all below 32
    tol = (dim + 20) * H32 * 32
    near(got[0], rh, tol)
    near(got[1], ry, tol)
    assert got[0] is out and got[1] is y
    assert torch.equal(wide[:, :3 * dim], dev(x[:, :3 * dim]))


# ---- attention: what a result of few rows is off by ----------------------------
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lengths,window", [([(1, 20), (1, 37), (1, 3)], 0), ([(8, 30)], 0),
                                            ([(3, 200), (5, 24)], 20)])
def test_attention_of_few_binary16_rows_is_off_by_its_rounding(lengths, window, dim):
    """Up to 32 rows to a conversation a binary16 result carries the rounding of
    its own type, and of float32 weights and sums besides.  (Few keys and small
    scores keep those far below a binary16 weight's rounding.)"""
    kc, vc, q, start, lens, table = batch_inputs(lengths, 8, 2, dim, 16, True, dim, window, 4,
                                                 q_scale=0.25)
    assert q4.q4_0_select_attention(q4.q4_0_kv_cache(0, 0, len(kc), 2, 16, dim), 8, q4.F16,
                                    len(q), table.shape[1], len(lengths), window, 4) == 32
    ref, absolute, score = block.attend(kc, vc, q, start, lens, table, window, 4, dim ** -0.5)
    y = attend(kc, vc, q, start, lens, table, window, 4, dim ** -0.5)
    near(y, ref, attention_tol(ref, absolute, score, 40, dim, False) + np.abs(ref) * H16
         + 2.0 ** -25)


def clean(a):
    return np.where(np.isfinite(a), a, 0.0)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_attention_infinite_keys(lengths, dim, half):
    """A key whose score is minus infinity has the weight 0, whatever the type of
    the queries; a score of plus infinity is NaN throughout."""
    rng, kc, vc, start, lens, table = plain(lengths, dim, 13)
    table[:] = np.arange(table.shape[1])
    kc[0, :, 3, 0], kc[1, 1, 9, 1], kc[2, 0, 5, 1] = np.inf, -np.inf, -np.inf
    q = rng.standard_normal((start[-1], 4, dim)).astype(np.float16 if half else np.float32)
    q[:, :, 0], q[:, :, 1] = -np.abs(q[:, :, 0]) - 1, np.abs(q[:, :, 1]) + 1
    q[::-5, 3, 0] *= -1
    with np.errstate(invalid="ignore"):
        ref, absolute, score = block.attend(kc, vc, q, start, lens, table, 0, 0, dim ** -0.5)
    y = attend(kc, vc, q, start, lens, table, scale=dim ** -0.5)
    assert np.isfinite(ref[-1, :3]).all() and np.isnan(ref[-1, 3]).all()
    near(y, ref, attention_tol(clean(ref), clean(absolute), clean(score), 300, dim, half))


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_attention_infinite_keys_with_infinite_values(lengths, dim, half):
    """A key whose score is minus infinity has the weight 0, and 0 times its
    value's infinity is NaN in that column; finite values beside it count
    nothing, and a score of plus infinity is NaN throughout."""
    rng, kc, vc, start, lens, table = plain(lengths, dim, 12)
    table[:] = np.arange(table.shape[1])
    kc[0, :, 3, 0] = np.inf
    vc[0, :, 3, 7], vc[0, 1, 3, 9] = np.inf, -np.inf
    kc[2, 0, 5, 1], vc[2, 0, 5, 11] = -np.inf, np.nan
    q = rng.standard_normal((start[-1], 4, dim)).astype(np.float16 if half else np.float32)
    q[:, :, 0] = -np.abs(q[:, :, 0]) - np.finfo(q.dtype).tiny
    q[::-5, 3, 0] *= -1
    q[:, :, 1] = np.abs(q[:, :, 1]) + np.finfo(q.dtype).tiny
    with np.errstate(invalid="ignore"):
        ref, absolute, score = block.attend(kc, vc, q, start, lens, table, 0, 0, dim ** -0.5)
    y = attend(kc, vc, q, start, lens, table, scale=dim ** -0.5)
    assert np.isnan(ref[-1, 0, 7]) and np.isfinite(ref[-1, 0, 8]) and np.isnan(ref[-1, 3]).all()
    near(y, ref, attention_tol(clean(ref), clean(absolute), clean(score), 300, dim, half))
