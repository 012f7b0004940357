"""The operators of a step of drafted tokens without a GPU: every invalid call
is refused before anything touches HIP, workspace sizes, what the conveniences
refuse, and the float64 definitions on hand-worked cases."""
import itertools

import numpy as np
import pytest
import torch

import gemm_q4_amd as q4
from oracle import step

A, B, C, D, E, F, G, H, I, J = ((i + 1) << 36 for i in range(10))   # fake addresses, far apart


def status_of(fn, *args):
    try:
        fn(*args)
    except q4.Q4Error as e:
        return e.status
    return q4.OK


def cache(**kw):
    f = dict(k=A, v=B, k_scale=I, v_scale=J, pages=4, heads=2, page_size=16, dim=64)
    f.update(kw)
    return q4.q4_0_kv_cache8(*f.values())


BAD_CACHES = [
    (dict(k=0), q4.ENULL), (dict(v=0), q4.ENULL), (dict(k_scale=0), q4.ENULL),
    (dict(v_scale=0), q4.ENULL), (dict(k=A + 8), q4.EALIGN), (dict(v=B + 2), q4.EALIGN),
    (dict(k_scale=I + 2), q4.EALIGN), (dict(v_scale=J + 1), q4.EALIGN),
    (dict(v=A + 64), q4.EALIAS), (dict(k_scale=B + 64), q4.EALIAS),
    (dict(v_scale=I + 8), q4.EALIAS), (dict(pages=0), q4.ESHAPE), (dict(pages=1 << 31), q4.ESHAPE),
    (dict(heads=0), q4.ESHAPE), (dict(heads=1025), q4.ESHAPE), (dict(page_size=8), q4.ESHAPE),
    (dict(page_size=48), q4.ESHAPE), (dict(page_size=131072), q4.ESHAPE),
    (dict(dim=0), q4.ESHAPE), (dict(dim=60), q4.ESHAPE), (dict(dim=520), q4.ESHAPE),
    (dict(pages=(1 << 31) - 1, heads=1024, page_size=65536, dim=512), q4.ESHAPE),
]


def append_args(**kw):
    f = dict(cache=cache(), rot=q4.q4_0_rotary(C, 64, 0, 1.0, 0, 0, 1e-6, 0.0), q=D, q_stride=256,
             k=E, k_stride=128, v=F, v_stride=128, x_dtype=q4.F32, q_out=G, q_dtype=q4.F16,
             q_heads=4, positions=H, slots=H + (1 << 30), n=3)
    f.update(kw)
    return tuple(f.values())


def attention_args(**kw):
    f = dict(cache=cache(), q=D, q_stride=256, x_dtype=q4.F16, q_heads=4, y=E, n=3, q_start=F,
             kv_len=G, table=H, table_stride=4, batch=2, window=0, sinks=0, scale=0.125)
    f.update(kw)
    return tuple(f.values())


def read_args(**kw):
    f = dict(cache=cache(), slots=C, n=5, k=D, v=E, y_dtype=q4.F16)
    f.update(kw)
    return tuple(f.values())


@pytest.mark.parametrize("bad,expect", BAD_CACHES)
def test_bad_caches(bad, expect):
    assert status_of(q4.q4_0_kv_append8, *append_args(cache=cache(**bad))) == expect
    assert status_of(q4.q4_0_attention8, *attention_args(cache=cache(**bad))) == expect
    assert status_of(q4.q4_0_kv_read8, *read_args(cache=cache(**bad))) == expect


@pytest.mark.parametrize("bad,expect", [
    (dict(cache=None), q4.ENULL), (dict(n=0), q4.ESHAPE), (dict(n=q4.MAX_N + 1), q4.ESHAPE),
    (dict(x_dtype=2), q4.EINVAL), (dict(q_heads=0), q4.ESHAPE), (dict(k_stride=127), q4.ESHAPE),
    (dict(k=0), q4.ENULL), (dict(slots=0), q4.ENULL), (dict(positions=0), q4.ENULL),
    (dict(k=E + 8), q4.EALIGN), (dict(slots=H + 4), q4.EALIGN), (dict(q_out=D + 64), q4.EALIAS),
    (dict(q_out=A + 64), q4.EALIAS), (dict(q_out=I + 16), q4.EALIAS), (dict(k=A), q4.EALIAS),
    (dict(v=J), q4.EALIAS), (dict(slots=B + 8), q4.EALIAS), (dict(positions=I + 4), q4.EALIAS),
])
def test_append_refusals(bad, expect):
    assert status_of(q4.q4_0_kv_append8, *append_args(**bad)) == expect


@pytest.mark.parametrize("bad,expect", [
    (dict(cache=None), q4.ENULL), (dict(n=0), q4.ESHAPE), (dict(n=q4.MAX_N + 1), q4.ESHAPE),
    (dict(slots=0), q4.ENULL), (dict(k=0, v=0), q4.ENULL), (dict(y_dtype=2), q4.EINVAL),
    (dict(slots=C + 4), q4.EALIGN), (dict(k=D + 8), q4.EALIGN), (dict(v=E + 4), q4.EALIGN),
    (dict(v=D + 64), q4.EALIAS), (dict(k=A), q4.EALIAS), (dict(v=I), q4.EALIAS),
    (dict(k=C), q4.EALIAS),
])
def test_read_refusals(bad, expect):
    assert status_of(q4.q4_0_kv_read8, *read_args(**bad)) == expect


@pytest.mark.parametrize("bad,expect", [
    (dict(cache=None), q4.ENULL), (dict(n=0), q4.ESHAPE), (dict(batch=0), q4.ESHAPE),
    (dict(q_heads=3), q4.ESHAPE), (dict(table_stride=0), q4.ESHAPE),
    (dict(table_stride=(1 << 26) + 1), q4.ESHAPE), (dict(window=-1), q4.EINVAL),
    (dict(sinks=1 << 31), q4.EINVAL), (dict(x_dtype=2), q4.EINVAL),
    (dict(cache=cache(dim=96)), q4.EUNSUPPORTED), (dict(cache=cache(dim=512)), q4.EUNSUPPORTED),
    (dict(scale=0.0), q4.EINVAL), (dict(scale=float("nan")), q4.EINVAL),
    (dict(q_stride=255), q4.ESHAPE), (dict(q=0), q4.ENULL), (dict(table=0), q4.ENULL),
    (dict(q=D + 8), q4.EALIGN), (dict(y=D + 64), q4.EALIAS), (dict(y=A + 16), q4.EALIAS),
    (dict(y=I), q4.EALIAS), (dict(y=J + 16), q4.EALIAS), (dict(y=H), q4.EALIAS),
])
def test_attention_refusals(bad, expect):
    assert status_of(q4.q4_0_attention8, *attention_args(**bad)) == expect


def test_attention_workspace():
    size = q4.q4_0_attention8_workspace_size
    for n, batch, width in [(1, 1, 1), (1, 1, 8192), (64, 64, 512), (5000, 2, 400),
                            (65536, 65536, 4), (65536, 1, 100000)]:
        for dim in (64, 128, 256):
            c = cache(k=0, v=0, k_scale=0, v_scale=0, heads=8, dim=dim, pages=1 << 20)
            assert 0 <= size(c, 32, q4.F16, n, width, batch) <= q4.WORKSPACE_MAX
    args = dict(cache=cache(heads=8, dim=128, pages=1 << 12), q_stride=4096, q_heads=32, n=1,
                batch=1, table_stride=8192)
    need = size(args["cache"], 32, q4.F16, 1, 8192, 1)
    assert need > 0
    call = lambda *w: status_of(q4.q4_0_attention8, *attention_args(**args), *w)
    ws = 11 << 36
    assert call() == q4.EWORKSPACE and call(ws, need - 1) == q4.EWORKSPACE
    assert call(ws + 64, need) == q4.EALIGN
    assert call(D, need) == q4.EALIAS and call(I, need) == q4.EALIAS
    assert status_of(size, cache(dim=96), 4, q4.F16, 1, 1, 1) == q4.EUNSUPPORTED
    assert q4.q4_0_select_attention8(cache(), 4, q4.F16, 1, 4, 1) == 32
    assert status_of(q4.q4_0_select_attention8, cache(), 3, q4.F16, 1, 4, 1) == q4.ESHAPE


def embed_args(**kw):
    f = dict(packed=A, tokens=B, n=3, out=300, in_=64, scale=2.0, h=C, pre=D, weight_offset=0.0,
             eps=1e-6, y=E, y_dtype=q4.F16)
    f.update(kw)
    return tuple(f.values())


@pytest.mark.parametrize("bad,expect", [
    (dict(n=0), q4.ESHAPE), (dict(n=q4.MAX_N + 1), q4.ESHAPE), (dict(out=0), q4.ESHAPE),
    (dict(in_=33), q4.ESHAPE), (dict(in_=32800), q4.EUNSUPPORTED), (dict(y_dtype=2), q4.EINVAL),
    (dict(scale=float("inf")), q4.EINVAL), (dict(scale=float("nan")), q4.EINVAL),
    (dict(packed=0), q4.ENULL), (dict(tokens=0), q4.ENULL), (dict(h=0), q4.ENULL),
    (dict(pre=0), q4.ENULL), (dict(packed=A + 8), q4.EALIGN), (dict(tokens=B + 2), q4.EALIGN),
    (dict(h=C + 4), q4.EALIGN), (dict(y=E + 2), q4.EALIGN), (dict(pre=D + 4), q4.EALIGN),
    (dict(h=A + 64), q4.EALIAS), (dict(y=C + 64), q4.EALIAS), (dict(h=B), q4.EALIAS),
    (dict(y=D), q4.EALIAS),
])
def test_embed_refusals(bad, expect):
    assert status_of(q4.q4_0_embed, *embed_args(**bad)) == expect


def verify_args(**kw):
    f = dict(logits=A, stride=1000, drafted=B, drafted_stride=1000, x_dtype=q4.F32, vocab=1000,
             tokens=C, q_start=D, n=6, batch=2, temperature=E, uniform=F, accepted=G, next_=H,
             workspace=I, workspace_bytes=1 << 20)
    f.update(kw)
    return tuple(f.values())


@pytest.mark.parametrize("bad,expect", [
    (dict(n=0), q4.ESHAPE), (dict(n=q4.MAX_N + 1), q4.ESHAPE), (dict(batch=0), q4.ESHAPE),
    (dict(batch=q4.MAX_N + 1), q4.ESHAPE), (dict(vocab=0), q4.ESHAPE),
    (dict(vocab=q4.MAX_OUT + 1, stride=1 << 30, drafted_stride=1 << 30), q4.ESHAPE),
    (dict(vocab=q4.MAX_OUT, n=65536, stride=1 << 30, drafted_stride=1 << 30), q4.EUNSUPPORTED),
    (dict(x_dtype=2), q4.EINVAL), (dict(stride=999), q4.ESHAPE),
    (dict(drafted_stride=999), q4.ESHAPE), (dict(stride=1 << 60), q4.ESHAPE),
    (dict(logits=0), q4.ENULL), (dict(tokens=0), q4.ENULL), (dict(q_start=0), q4.ENULL),
    (dict(uniform=0), q4.ENULL), (dict(accepted=0), q4.ENULL), (dict(next_=0), q4.ENULL),
    (dict(logits=A + 2), q4.EALIGN), (dict(drafted=B + 2), q4.EALIGN),
    (dict(tokens=C + 2), q4.EALIGN), (dict(temperature=E + 1), q4.EALIGN),
    (dict(uniform=F + 2), q4.EALIGN), (dict(next_=H + 2), q4.EALIGN),
    (dict(accepted=A + 16), q4.EALIAS), (dict(next_=G + 4), q4.EALIAS), (dict(next_=F), q4.EALIAS),
    (dict(accepted=C), q4.EALIAS), (dict(workspace=0, workspace_bytes=0), q4.EWORKSPACE),
    (dict(workspace_bytes=100), q4.EWORKSPACE), (dict(workspace=I + 16), q4.EALIGN),
    (dict(workspace=B + 256), q4.EALIAS), (dict(workspace=G), q4.EALIAS),
])
def test_verify_refusals(bad, expect):
    assert status_of(q4.q4_0_verify, *verify_args(**bad)) == expect


def test_verify_workspace():
    size = q4.q4_0_verify_workspace_size
    need = size(6, 2, 1000, True)
    assert size(6, 2, 1000) < need < 4096
    assert status_of(q4.q4_0_verify, *verify_args(workspace_bytes=need - 1)) == q4.EWORKSPACE
    assert size(600, 64, 200000, True) <= q4.WORKSPACE_MAX
    assert status_of(size, 0, 1, 10) == q4.ESHAPE
    assert status_of(size, 65536, 1, q4.MAX_OUT) == q4.EUNSUPPORTED


def test_verify_draft_logits_without_their_last_row():
    """The last row judges nothing: what lies where it would be is no overlap."""
    last = B + 5 * 1000 * 4
    near = dict(workspace=0, workspace_bytes=0)        # refused, but after the overlaps
    assert status_of(q4.q4_0_verify, *verify_args(accepted=last, **near)) == q4.EWORKSPACE
    assert status_of(q4.q4_0_verify, *verify_args(accepted=last - 4, **near)) == q4.EALIAS
    one = dict(n=1, batch=1, **near)
    assert status_of(q4.q4_0_verify, *verify_args(accepted=B, **one)) == q4.EWORKSPACE
    assert status_of(q4.q4_0_verify, *verify_args(accepted=A, **one)) == q4.EALIAS


# ---- the conveniences --------------------------------------------------------
def host_cache(pages=2, heads=2, page=16, dim=64):
    k = torch.zeros(pages, heads, page, dim, dtype=torch.int8)
    s = torch.zeros(pages, heads, page)
    return k, k.clone(), s, s.clone()


def test_cache_descriptors_refuse_what_does_not_fit():
    k, v, ks, vs = host_cache()
    with pytest.raises(TypeError, match="k must be Char"):
        q4.kv_cache8(k.half(), v, ks, vs)
    with pytest.raises(ValueError, match="v must have shape"):
        q4.kv_cache8(k, v[:1], ks, vs)
    with pytest.raises(TypeError, match="k_scale must be Float"):
        q4.kv_cache8(k, v, ks.half(), vs)
    with pytest.raises(ValueError, match="v_scale must have shape"):
        q4.kv_cache8(k, v, ks, vs[..., None])
    with pytest.raises(ValueError, match="k must be contiguous"):
        q4.kv_cache8(k.transpose(1, 2).contiguous().transpose(1, 2), v, ks, vs)
    with pytest.raises(ValueError, match="no empty dimension"):
        q4.kv_cache8(k[:0], v[:0], ks[:0], vs[:0])
    with pytest.raises(TypeError, match="v_scale must be a tensor"):
        q4.kv_cache8(k, v, ks, None)
    with pytest.raises(TypeError):
        type(q4.kv_cache8(k, v, ks, vs))()


def test_cache_descriptor_follows_its_tensors():
    k, v, ks, vs = host_cache()
    c = q4.kv_cache8(k, v, ks, vs)
    at = lambda: q4.q4_0_kv_cache8.from_address(c.address)
    assert (at().k, at().v, at().k_scale, at().v_scale) == tuple(
        t.data_ptr() for t in (k, v, ks, vs))
    assert (c.pages, c.heads, c.page_size, c.dim) == (2, 2, 16, 64)
    new = host_cache(3, 1, 32, 128)
    for t, n in zip((k, v, ks, vs), new):
        t.data = n
    assert (at().k, at().v_scale) == (k.data_ptr(), vs.data_ptr())
    assert (c.pages, c.heads, c.page_size, c.dim) == (3, 1, 32, 128)
    vs.data = torch.zeros(3, 1, 16)
    with pytest.raises(ValueError, match="v_scale must have shape"):
        c.dim


def test_conveniences_refuse_what_does_not_fit():
    c = q4.kv_cache8(*host_cache())
    q, kv = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError, match="cache must come from kv_cache"):
        q4.kv_append(object(), None, q, kv, kv, None, slots, q_out=q.clone())
    with pytest.raises(TypeError, match="one type"):
        q4.kv_append(c, None, q, kv, kv.half(), None, slots)
    with pytest.raises(ValueError, match="on a GPU"):
        q4.kv_append(c, None, q, kv, kv, None, slots)
    half = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="kv_cache8"):
        q4.kv_read(q4.kv_cache(half, half.clone()), slots)
    with pytest.raises(TypeError, match="slots must be Long"):
        q4.kv_read(c, slots.int())
    with pytest.raises(TypeError, match="v must be Float"):
        q4.kv_read(c, slots, k=kv.clone(), v=kv.half())
    with pytest.raises(ValueError, match="k must have shape"):
        q4.kv_read(c, slots, k=kv[:2].clone())
    with pytest.raises(ValueError, match="on a GPU"):
        q4.kv_read(c, slots)
    start, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be"):
        q4.attention(c, q[..., :32], start, lens, torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="on a GPU"):
        q4.attention(c, q, start, lens, torch.zeros(1, 2, dtype=torch.int32))

    packed, tokens = torch.zeros(q4.q4_0_packed_bytes(20, 64), dtype=torch.uint8), start
    with pytest.raises(ValueError, match="fewer than"):
        q4.embed(packed, tokens, 33, 64)
    with pytest.raises(TypeError, match="dense bytes"):
        q4.embed(packed.float(), tokens, 20, 64)
    with pytest.raises(TypeError, match="tokens must be Int"):
        q4.embed(packed, tokens.long(), 20, 64)
    with pytest.raises(ValueError, match="pre must have shape"):
        q4.embed(packed, tokens, 20, 64, pre=torch.ones(32))
    with pytest.raises(ValueError, match="h must have shape"):
        q4.embed(packed, tokens, 20, 64, h=torch.ones(2, 32))
    with pytest.raises(ValueError, match="on a GPU"):
        q4.embed(packed, tokens, 20, 64)

    logits, tok, uni = torch.zeros(3, 50), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(ValueError, match="logits must be"):
        q4.verify(logits[None], tok, start, uni, ws=packed)
    with pytest.raises(TypeError, match="one type"):
        q4.verify(logits, tok, start, uni, draft_logits=logits.half())
    with pytest.raises(ValueError, match="does not fit"):
        q4.verify(logits, tok, start, uni, draft_logits=logits[:, :49])
    with pytest.raises(TypeError, match="tokens must be Int"):
        q4.verify(logits, tok.long(), start, uni)
    with pytest.raises(ValueError, match="uniform must have shape"):
        q4.verify(logits, tok, start, uni[:, :1])
    with pytest.raises(ValueError, match="temperature must have shape"):
        q4.verify(logits, tok, start, uni, temperature=torch.ones(2))
    with pytest.raises(TypeError, match="accepted must be Int"):
        q4.verify(logits, tok, start, uni, accepted=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="on a GPU"):
        q4.verify(logits, tok, start, uni)
    with pytest.raises(q4.Q4Error):
        q4.verify(logits, tok, start[:1], uni)


# ---- the definitions, by hand ------------------------------------------------
def test_oracle_quantize_by_hand():
    c, s = step.quantize([[127.0, -63.5, 0.5, 1.5], [0.0] * 4, [1.0, np.inf, 0.0, 0.0]])
    assert c[0].tolist() == [127, -64, 0, 2] and s[0] == 1.0
    assert c[1].tolist() == [0] * 4 and s[1] == 0.0 and np.isnan(s[2])
    c, s = step.quantize([[-2.54, 1.0]])
    assert c.tolist() == [[-127, 50]] and np.isclose(s[0], 0.02)
    assert step.quantize([[1e-37, 0.0]])[1][0] == 0.0          # the scale would lose bits
    x = step.numbers([[2, -3], [1, 1]], [0.5, np.inf])
    assert x[0].tolist() == [1.0, -1.5] and np.isnan(x[1]).all()


def test_oracle_rows_by_hand():
    y = step.rows([[1.0, 2.0], [3.0, -4.0]], [1, 2, -1, 0], 0.5)
    assert y.tolist() == [[1.5, -2.0], [0.0, 0.0], [0.0, 0.0], [0.5, 1.0]]


def test_oracle_verify_by_hand():
    # p = (1/2, 1/4, 1/4), three rows of one conversation: two drafts
    l = np.log([[0.5, 0.25, 0.25]] * 3)
    u = lambda *x: np.array(x, float).reshape(3, 2)
    run = lambda tokens, uni, **kw: tuple(int(x[0]) for x in step.verify(
        l, tokens, [0, 3], uni, **kw))
    # drafts 0 and 1 are taken below 1/2 and 1/4; the draw is from p
    assert run([9, 0, 1], u(0.49, 0, 0.24, 0, 0, 0.74)) == (2, 1)
    assert run([9, 0, 1], u(0.49, 0, 0.24, 0, 0, 0.76)) == (2, 2)
    # the second is refused: what is left is (1/2, -, 1/4)
    assert run([9, 0, 1], u(0.49, 0, 0.26, 0.66, 0, 0)) == (1, 0)
    assert run([9, 0, 1], u(0.49, 0, 0.26, 0.67, 0, 0)) == (1, 2)
    # drawn from q = (1/4, 1/2, 1/4): u q(1) < 1/4 takes it; refused: only token 0 is above
    q = np.log([[0.25, 0.5, 0.25]] * 3)
    assert run([9, 1, 1], u(0.49, 0, 0.51, 0.99, 0, 0), drafted=q) == (1, 0)
    # greedy: token 0 wins
    assert run([9, 0, 0], u(1, 0, 1, 0, 0, 0.9), temperature=[0.0]) == (2, 0)
    assert run([9, 0, 1], u(0, 0, 0, 0, 0, 0.9), temperature=[0.0]) == (1, 0)
    # outside the vocabulary: refused, all of p is left
    assert run([9, 3, 0], u(0, 0.8, 0, 0, 0, 0)) == (0, 2)
    l[1, 2] = np.nan
    assert run([9, 0, 1], u(0.49, 0, 0.24, 0, 0, 0.74)) == (1, -1)
    a, b = step.verify(l, [9, 0, 1], [0, 0, 1, 3], u(0, 0.1, 0.3, 0.3, 0, 0))
    assert a.tolist() == [0, 0, 0] and b.tolist() == [-1, 0, -1]


@pytest.mark.parametrize("drawn", [False, True])
def test_oracle_verify_draws_from_the_target(drawn):
    """The token after the last accepted position is distributed as the target's
    own, whatever the draft: over a grid of uniform numbers, drafts drawn from q
    (or picked)."""
    rng = np.random.default_rng(3)
    l, g = rng.standard_normal((2, 2, 5))
    p = np.exp(l[0]) / np.exp(l[0]).sum()
    q = np.exp(g[0]) / np.exp(g[0]).sum()
    grid = (np.arange(100) + 0.5) / 100
    got = np.zeros(5)
    for d in range(5) if drawn else [2]:
        share = q[d] if drawn else 1.0
        for u, v in itertools.product(grid, grid):
            a, t = step.verify(l, [0, d], [0, 2], [[u, v], [0, 0.5]], drafted=g if drawn else None)
            got[d if a[0] else t[0]] += share / 10000
    assert np.abs(got - p).max() < 0.03           # steps of the two grids
