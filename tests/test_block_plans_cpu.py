"""How attention calls are cut into work, as the host queries show it, without a
GPU."""
import pytest

import gemm_q4_amd as q4


def cache(heads=8, dim=128):
    return q4.q4_0_kv_cache(0, 0, 1 << 14, heads, 16, dim)


@pytest.mark.parametrize("dtype", [q4.F32, q4.F16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_tiles_by_rows(dim, dtype):
    """Up to 32 rows to a conversation 32-row tiles; above, 128 rows where that
    gives every compute unit a tile, else 64."""
    rows = lambda n, batch, heads=8, group=4: q4.q4_0_select_attention(
        cache(heads, dim), heads * group, dtype, n, 512, batch)
    assert rows(1, 1) == rows(8, 1) == rows(64, 64) == rows(512, 64) == 32
    assert rows(9, 1) == rows(512, 1) == rows(900, 1) == rows(40, 3) == 64
    assert rows(1100, 1) == rows(65536, 1) == rows(8000, 2) == rows(513, 64) == 128
    assert rows(512, 1, heads=64, group=1) == 128


def test_tile_query_refuses_what_the_call_refuses():
    def status(*a):
        with pytest.raises(q4.Q4Error) as e:
            q4.q4_0_select_attention(*a)
        return e.value.status
    assert status(None, 8, q4.F16, 1, 1, 1) == q4.ENULL
    assert status(cache(dim=96), 8, q4.F16, 1, 1, 1) == q4.EUNSUPPORTED
    assert status(cache(), 9, q4.F16, 1, 1, 1) == q4.ESHAPE
    assert status(cache(), 8, q4.F16, 0, 1, 1) == q4.ESHAPE
    assert status(cache(), 8, 5, 1, 1, 1) == q4.EINVAL


def test_split_calls_refuse_bad_workspaces():
    """One token over a long axis is split: it needs a workspace, and refuses one
    that is missing, small, misaligned or overlapping."""
    at = [(i + 1) << 36 for i in range(8)]
    c = q4.q4_0_kv_cache(at[0], at[1], 1 << 14, 8, 16, 128)
    need = q4.q4_0_attention_workspace_size(c, 32, q4.F16, 1, 8192, 1)
    assert 0 < need <= q4.WORKSPACE_MAX

    def status(*workspace):
        with pytest.raises(q4.Q4Error) as e:
            q4.q4_0_attention(c, at[2], 4096, q4.F16, 32, at[3], 1, at[4], at[5], at[6], 8192, 1, 0,
                              0, 0.125, *workspace)
        return e.value.status
    assert status() == q4.EWORKSPACE
    assert status(at[7], need - 1) == q4.EWORKSPACE
    assert status(at[7] + 64, need) == q4.EALIGN
    assert status(at[2], need) == q4.EALIAS
    assert status(at[3] + 4096 - 256, need) == q4.EALIAS


@pytest.mark.parametrize("moved", [
    dict(y=63), dict(y=65), dict(y=128), dict(y=300), dict(h_out=1), dict(h_out=129),
    dict(y=64, y_stride=321), dict(y=64, y_dtype=q4.F16), dict(gate=255, gate_col=0)])
def test_residual_norm_refuses_columns_that_meet(moved):
    """Columns of one wide buffer (rows of 320: h from 0 on, b from 128, h_out from
    192, y from 256) that share an element, or rows of different strides."""
    f = dict(h=0, b=128, h_out=192, y=256, gate=None, gate_col=1, y_dtype=q4.F32, y_stride=320)
    f.update(moved)
    at = {name: 0 if f[name] is None else (1 << 36) + 4 * f[name]
          for name in ("h", "b", "h_out", "y", "gate")}
    with pytest.raises(q4.Q4Error) as e:
        q4.q4_0_residual_norm(at["b"], q4.F32, 320, 0, at["gate"], 320, f["gate_col"], 1.0, at["h"],
                              at["h_out"], 320, 2 << 36, 0.0, 1e-6, at["y"], f["y_dtype"],
                              f["y_stride"], 3, 64)
    assert e.value.status == q4.EALIAS
