"""The operators between a block's products without a GPU: every invalid call
is refused before anything touches HIP, workspace sizes, and the float64
definitions on hand-worked cases."""
import math

import numpy as np
import pytest
import torch

import gemm_q4_amd as q4
from oracle import block

A, B, C, D, E, F, G, H = ((i + 1) << 36 for i in range(8))   # fake device addresses, far apart


def status_of(fn, *args):
    try:
        fn(*args)
    except q4.Q4Error as e:
        return e.status
    return q4.OK


def cache(**kw):
    f = dict(k=A, v=B, pages=4, heads=2, page_size=16, dim=64)
    f.update(kw)
    return q4.q4_0_kv_cache(*(f[n] for n in ("k", "v", "pages", "heads", "page_size", "dim")))


def rot(**kw):
    f = dict(inv_freq=C, rot_dim=64, interleaved=0, amplitude=1.0, q_norm=0, k_norm=0, eps=1e-6,
             weight_offset=0.0)
    f.update(kw)
    return q4.q4_0_rotary(*f.values())


BAD_CACHES = [
    (dict(k=0), q4.ENULL), (dict(v=0), q4.ENULL), (dict(k=A + 8), q4.EALIGN),
    (dict(v=B + 2), q4.EALIGN), (dict(v=A + 64), q4.EALIAS), (dict(pages=0), q4.ESHAPE),
    (dict(pages=1 << 31), q4.ESHAPE), (dict(heads=0), q4.ESHAPE), (dict(heads=1025), q4.ESHAPE),
    (dict(page_size=8), q4.ESHAPE), (dict(page_size=48), q4.ESHAPE),
    (dict(page_size=131072), q4.ESHAPE), (dict(page_size=-16), q4.ESHAPE),
    (dict(dim=0), q4.ESHAPE), (dict(dim=60), q4.ESHAPE), (dict(dim=520), q4.ESHAPE),
    (dict(pages=(1 << 31) - 1, heads=1024, page_size=65536, dim=512), q4.ESHAPE),
]


def append_args(**kw):
    f = dict(cache=cache(), rot=rot(), q=D, q_stride=256, k=E, k_stride=128, v=F, v_stride=128,
             x_dtype=q4.F32, q_out=G, q_dtype=q4.F16, q_heads=4, positions=H, slots=H + (1 << 30),
             n=3)
    f.update(kw)
    return tuple(f.values())


@pytest.mark.parametrize("bad,expect", BAD_CACHES)
def test_append_refuses_bad_caches(bad, expect):
    assert status_of(q4.q4_0_kv_append, *append_args(cache=cache(**bad))) == expect


@pytest.mark.parametrize("bad,expect", [
    (dict(cache=None), q4.ENULL), (dict(n=0), q4.ESHAPE), (dict(n=q4.MAX_N + 1), q4.ESHAPE),
    (dict(x_dtype=2), q4.EINVAL), (dict(q_dtype=-1), q4.EINVAL), (dict(q_heads=0), q4.ESHAPE),
    (dict(q_heads=1025), q4.ESHAPE), (dict(rot=rot(rot_dim=-8)), q4.ESHAPE),
    (dict(rot=rot(rot_dim=72)), q4.ESHAPE), (dict(rot=rot(rot_dim=20)), q4.ESHAPE),
    (dict(k_stride=127), q4.ESHAPE), (dict(v_stride=0), q4.ESHAPE),
    (dict(q_stride=255), q4.ESHAPE), (dict(q_stride=1 << 60), q4.ESHAPE),
    (dict(k=0), q4.ENULL), (dict(v=0), q4.ENULL), (dict(slots=0), q4.ENULL),
    (dict(q_out=0), q4.ENULL), (dict(positions=0), q4.ENULL), (dict(rot=rot(inv_freq=0)), q4.ENULL),
    (dict(k=E + 8), q4.EALIGN), (dict(q=D + 4), q4.EALIGN), (dict(k_stride=129), q4.EALIGN),
    (dict(x_dtype=q4.F16, v_stride=132), q4.EALIGN), (dict(slots=H + 4), q4.EALIGN),
    (dict(positions=H + 2), q4.EALIGN), (dict(q_out=G + 8), q4.EALIGN),
    (dict(rot=rot(q_norm=C + 260)), q4.EALIGN), (dict(rot=rot(inv_freq=C + 1)), q4.EALIGN),
    (dict(q_out=D + 64), q4.EALIAS), (dict(q_out=A + 64), q4.EALIAS), (dict(k=A), q4.EALIAS),
    (dict(slots=B + 8), q4.EALIAS), (dict(positions=G), q4.EALIAS),
    (dict(rot=rot(k_norm=B)), q4.EALIAS), (dict(rot=rot(inv_freq=G)), q4.EALIAS),
])
def test_append_refusals(bad, expect):
    assert status_of(q4.q4_0_kv_append, *append_args(**bad)) == expect


def attention_args(**kw):
    f = dict(cache=cache(), q=D, q_stride=256, x_dtype=q4.F16, q_heads=4, y=E, n=3, q_start=F,
             kv_len=G, table=H, table_stride=4, batch=2, window=0, sinks=0, scale=0.125)
    f.update(kw)
    return tuple(f.values())


@pytest.mark.parametrize("bad,expect", BAD_CACHES)
def test_attention_refuses_bad_caches(bad, expect):
    assert status_of(q4.q4_0_attention, *attention_args(cache=cache(**bad))) == expect


@pytest.mark.parametrize("bad,expect", [
    (dict(cache=None), q4.ENULL), (dict(n=0), q4.ESHAPE), (dict(batch=0), q4.ESHAPE),
    (dict(n=q4.MAX_N + 1), q4.ESHAPE), (dict(batch=q4.MAX_N + 1), q4.ESHAPE),
    (dict(q_heads=3), q4.ESHAPE), (dict(q_heads=0), q4.ESHAPE), (dict(table_stride=0), q4.ESHAPE),
    (dict(table_stride=(1 << 26) + 1), q4.ESHAPE), (dict(window=-1), q4.EINVAL),
    (dict(window=1 << 31), q4.EINVAL), (dict(sinks=-1), q4.EINVAL), (dict(x_dtype=2), q4.EINVAL),
    (dict(cache=cache(dim=96)), q4.EUNSUPPORTED), (dict(cache=cache(dim=512)), q4.EUNSUPPORTED),
    (dict(scale=0.0), q4.EINVAL), (dict(scale=-1.0), q4.EINVAL),
    (dict(scale=float("inf")), q4.EINVAL), (dict(scale=float("nan")), q4.EINVAL),
    (dict(q_stride=255), q4.ESHAPE), (dict(q=0), q4.ENULL), (dict(y=0), q4.ENULL),
    (dict(q_start=0), q4.ENULL), (dict(kv_len=0), q4.ENULL), (dict(table=0), q4.ENULL),
    (dict(q=D + 8), q4.EALIGN), (dict(q_stride=260), q4.EALIGN), (dict(y=E + 8), q4.EALIGN),
    (dict(q_start=F + 2), q4.EALIGN), (dict(table=H + 1), q4.EALIGN), (dict(y=D + 64), q4.EALIAS),
    (dict(y=A + 16), q4.EALIAS), (dict(y=H), q4.EALIAS),
])
def test_attention_refusals(bad, expect):
    assert status_of(q4.q4_0_attention, *attention_args(**bad)) == expect


def test_attention_workspace():
    """A call that splits the key axis needs a workspace and refuses one that is
    missing, small, misaligned or overlapping; sizes stay within the limit."""
    size = q4.q4_0_attention_workspace_size
    for n, batch, width in [(1, 1, 1), (1, 1, 8192), (64, 64, 512), (5000, 2, 400),
                            (65536, 65536, 4), (65536, 1, 100000)]:
        for dim in (64, 128, 256):
            c = cache(k=0, v=0, heads=8, dim=dim, pages=1 << 20)
            assert 0 <= size(c, 32, q4.F16, n, width, batch) <= q4.WORKSPACE_MAX
    c = cache(heads=8, dim=128, pages=1 << 14)
    args = dict(cache=c, q_stride=4096, q_heads=32, n=1, batch=1, table_stride=8192)
    need = size(c, 32, q4.F16, 1, 8192, 1)
    if need:
        ws = 9 << 36
        call = lambda *w: status_of(q4.q4_0_attention, *attention_args(**args), *w)
        assert call() == q4.EWORKSPACE
        assert call(ws, need - 1) == q4.EWORKSPACE
        assert call(ws + 64, need) == q4.EALIGN
        assert call(D, need) == q4.EALIAS
    assert status_of(size, cache(dim=96), 4, q4.F16, 1, 1, 1) == q4.EUNSUPPORTED
    assert status_of(size, cache(), 3, q4.F16, 1, 1, 1) == q4.ESHAPE


def norm_args(**kw):
    f = dict(b=A, b_dtype=q4.F32, b_stride=64, post=B, gate=C, gate_row=64, gate_col=1, alpha=1.0,
             h=D, h_out=D, h_stride=64, pre=E, weight_offset=0.0, eps=1e-6, y=F, y_dtype=q4.F16,
             y_stride=64, n=3, dim=64)
    f.update(kw)
    return tuple(f.values())


@pytest.mark.parametrize("bad,expect", [
    (dict(n=0), q4.ESHAPE), (dict(dim=0), q4.ESHAPE), (dict(n=q4.MAX_N + 1), q4.ESHAPE),
    (dict(dim=32769, b_stride=40000, h_stride=40000, y_stride=40000), q4.EUNSUPPORTED),
    (dict(b=0, y=0), q4.ENULL), (dict(b_dtype=2), q4.EINVAL), (dict(y_dtype=-1), q4.EINVAL),
    (dict(gate_col=2), q4.EINVAL), (dict(gate_row=-1), q4.EINVAL), (dict(b_stride=63), q4.ESHAPE),
    (dict(h_stride=63), q4.ESHAPE), (dict(y_stride=63), q4.ESHAPE), (dict(h=0), q4.ENULL),
    (dict(h_out=0), q4.ENULL), (dict(pre=0), q4.ENULL), (dict(h=D + 2), q4.EALIGN),
    (dict(b=A + 2), q4.EALIGN), (dict(y=F + 1), q4.EALIGN), (dict(h_out=D + 64), q4.EALIAS),
    (dict(h_out=A), q4.EALIAS), (dict(y=D), q4.EALIAS), (dict(y=E), q4.EALIAS),
    (dict(h_out=C), q4.EALIAS), (dict(y=A + 16), q4.EALIAS),
])
def test_residual_norm_refusals(bad, expect):
    assert status_of(q4.q4_0_residual_norm, *norm_args(**bad)) == expect


def test_conveniences_refuse_what_does_not_fit():
    """Types, shapes and strides that the addresses alone would not show."""
    k = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    c = q4.kv_cache(k, k.clone())
    q, kv = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    pos, slots = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        q4.kv_cache(k.float(), k)
    with pytest.raises(ValueError):
        q4.kv_cache(k, k[:1])
    with pytest.raises(ValueError):
        q4.kv_cache(k.transpose(1, 2), k.transpose(1, 2))
    with pytest.raises(TypeError):
        q4.kv_append(c, None, q, kv, kv.half(), pos, slots)
    with pytest.raises(TypeError):
        q4.kv_append(c, None, q, kv, kv, pos, slots.int())
    with pytest.raises(TypeError):
        q4.kv_append(c, None, q, kv, kv, pos.long(), slots)
    with pytest.raises(ValueError):
        q4.kv_append(c, None, q, kv[:, :1], kv, pos, slots)
    with pytest.raises(ValueError):
        q4.kv_append(c, None, q, kv.transpose(1, 2).contiguous().transpose(1, 2), kv, pos, slots)
    with pytest.raises(ValueError):
        q4.kv_append(c, None, q, kv, kv, pos, slots[:2])
    with pytest.raises(ValueError):
        q4.kv_append(c, q4.rotary(q_norm=torch.ones(32)), q, kv, kv, pos, slots)
    start, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        q4.attention(c, q[..., :32], start, lens, table)
    with pytest.raises(TypeError):
        q4.attention(c, q.bfloat16(), start, lens, table)
    with pytest.raises(TypeError):
        q4.attention(c, q, start, lens.long(), table)
    with pytest.raises(ValueError):
        q4.attention(c, q, start[:1], lens, table)
    with pytest.raises(TypeError):
        q4.attention(c, q, start, lens, table, y=q.half())
    h = torch.zeros(3, 64)
    with pytest.raises(TypeError):
        q4.residual_norm(h.half(), h)
    with pytest.raises(ValueError):
        q4.residual_norm(h, h[:2])
    with pytest.raises(ValueError):
        q4.residual_norm(h, h.clone(), gate=torch.zeros(3, 2))
    with pytest.raises(ValueError):
        q4.residual_norm(h, h.clone(), pre=torch.zeros(63))


# ---- the definitions, by hand ------------------------------------------------
def test_oracle_rotation_by_hand():
    x = [1.0, 2.0, 3.0, 4.0, 9.0]
    quarter = [math.pi / 2, math.pi]          # position 1: a quarter and a half turn
    assert np.allclose(block.rotate(x, 1, quarter), [-3.0, -2.0, 1.0, -4.0, 9.0])
    assert np.allclose(block.rotate(x, 1, quarter, interleaved=True),
                       [-2.0, 1.0, -3.0, -4.0, 9.0])
    assert np.allclose(block.rotate(x, 0, quarter, amplitude=2.0), [2.0, 4.0, 6.0, 8.0, 9.0])


def test_oracle_norm_by_hand():
    assert np.allclose(block.rms_norm([3.0, 4.0], [1.0, 2.0], 0.0),
                       [3 / math.sqrt(12.5), 8 / math.sqrt(12.5)])
    h, y = block.residual_norm([[1.0, 1.0]], b=[[3.0, 4.0]], pre=[1.0, 1.0], gate=[[2.0]],
                               alpha=0.5, eps=0.0)
    assert np.allclose(h, [[4.0, 5.0]]) and np.allclose(y, np.array([[4.0, 5.0]]) / math.sqrt(20.5))


def test_oracle_visibility_by_hand():
    see = lambda p, w, s: [j for j in range(10) if block.sees(p, j, w, s)]
    assert see(3, 0, 0) == [0, 1, 2, 3]
    assert see(5, 2, 0) == [4, 5]
    assert see(5, 2, 1) == [0, 4, 5]
    assert see(1, 4, 3) == [0, 1]
    assert see(-1, 2, 2) == []


def test_oracle_attention_by_hand():
    k = np.zeros((2, 1, 2, 2))
    v = np.arange(8.0).reshape(2, 1, 2, 2)
    k[1, 0, 0] = [math.log(3.0), 0.0]
    q = np.ones((2, 1, 2))
    # table [1, 0]: key 0 on page 1 offset 0 (weight 3), key 1 on page 1 offset 1 (weight 1)
    y, absolute, score = block.attend(k, v, q, [0, 2], [2], [[1, 0]])
    assert np.allclose(y[0, 0], [4.0, 5.0]) and np.allclose(y[1, 0], [4.5, 5.5])
    assert np.allclose(absolute, y) and np.isclose(score[1, 0], math.log(3.0))
    y, _, _ = block.attend(k, v, q, [0, 2], [1], [[1, 0]])     # position -1 sees nothing
    assert np.allclose(y[0], 0.0) and np.allclose(y[1, 0], [4.0, 5.0])
    y, _, _ = block.attend(k, v, q, [0, 1], [2], [[-1, 0]])
    assert np.isnan(y).all()


def test_oracle_append_by_hand():
    kc, vc = np.zeros((2, 1, 2, 4)), np.zeros((2, 1, 2, 4))
    rows = np.arange(8.0).reshape(2, 4)
    q, k, v = block.append(kc, vc, rows, rows, rows, [0, 0], [3, -1])
    assert np.allclose(k[1, 0, 1], rows[0]) and np.allclose(v[1, 0, 1], rows[0])
    assert k[0].sum() == 0 and k[1, 0, 0].sum() == 0 and np.allclose(q[1, 0], rows[1])
