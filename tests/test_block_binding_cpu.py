"""The block operators' conveniences without a GPU: what they refuse and with
which message, descriptors whose tensors change, and the package where their
extension module is missing."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import gemm_q4_amd as q4


@pytest.mark.parametrize("shape", [(1, 1, 16, 0), (1, 1, 0, 64), (1, 0, 16, 64), (0, 1, 16, 64)])
def test_caches_without_elements_are_refused(shape):
    """A head of no elements would be divided by in the calls that follow."""
    k = torch.zeros(shape, dtype=torch.float16)
    with pytest.raises(ValueError, match="no empty dimension"):
        q4.kv_cache(k, k.clone())


def test_descriptors_follow_their_tensors():
    """A parameter moved or cast holds other memory afterwards: the descriptor
    gives the new memory, or refuses it, and never the old one's address."""
    k, v = (torch.zeros(2, 2, 16, 64, dtype=torch.float16) for _ in range(2))
    cache = q4.kv_cache(k, v)
    at = lambda: q4.q4_0_kv_cache.from_address(cache.address)
    assert (at().k, at().v) == (k.data_ptr(), v.data_ptr())
    k.data = torch.ones(2, 2, 16, 64, dtype=torch.float16)
    assert (at().k, at().v) == (k.data_ptr(), v.data_ptr())
    k.data, v.data = (torch.zeros(3, 1, 32, 128, dtype=torch.float16) for _ in range(2))
    assert (at().k, at().v) == (k.data_ptr(), v.data_ptr())
    assert (cache.pages, cache.heads, cache.page_size, cache.dim) == (3, 1, 32, 128)
    v.data = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="v must have shape"):
        cache.address
    with pytest.raises(ValueError, match="v must have shape"):
        cache.dim
    v.data = torch.zeros(3, 1, 32, 128)
    with pytest.raises(TypeError, match="v must be Half"):
        cache.address

    inv, norm = torch.ones(32), torch.nn.Parameter(torch.ones(64), requires_grad=False)
    rot = q4.rotary(inv, interleaved=True, amplitude=0.5, q_norm=norm, eps=1e-3, weight_offset=1.0)
    at = lambda: q4.q4_0_rotary.from_address(rot.address)
    assert (at().inv_freq, at().q_norm, at().k_norm) == (inv.data_ptr(), norm.data_ptr(), None)
    norm.data = torch.full((128,), 2.0)
    inv.data = torch.ones(16)
    assert (at().inv_freq, at().q_norm, at().rot_dim) == (inv.data_ptr(), norm.data_ptr(), 32)
    assert (at().interleaved, at().amplitude, at().weight_offset) == (1, 0.5, 1.0)
    assert abs(at().eps - 1e-3) < 1e-9
    norm.data = norm.data.double()
    with pytest.raises(TypeError, match="q_norm must be Float"):
        rot.address


def test_calls_read_a_descriptor_whose_tensors_changed():
    """A call sees the tensors as they are now, before anything else of it."""
    k, v = (torch.zeros(2, 2, 16, 64, dtype=torch.float16) for _ in range(2))
    cache, norm = q4.kv_cache(k, v), torch.ones(64)
    rot = q4.rotary(q_norm=norm)
    q, kv = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64)
    norm.data = torch.ones(32)
    with pytest.raises(ValueError, match="norm weights of 32 do not fit heads of 64"):
        q4.kv_append(cache, rot, q, kv, kv, None, slots)
    v.data = torch.zeros(2, 2, 16, 64)
    with pytest.raises(TypeError, match="v must be Half"):
        q4.kv_append(cache, None, q, kv, kv, None, slots, q_out=q.clone())


class Wrapper:
    """Device memory that is no tensor, as a storage or another library's array is."""
    is_cuda, device = True, torch.device("cuda", 0)

    def data_ptr(self):
        return 1 << 36


def test_device_memory_that_is_no_tensor_goes_to_the_current_stream(monkeypatch):
    """Any argument that says it is on a GPU brings torch's current stream of its
    device, not the null stream."""
    class Stream:
        cuda_stream = 0x5150
    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: asked.append(d) or Stream)
    assert q4._stream(None, 1 << 36, Wrapper()) == 0x5150
    assert asked == [torch.device("cuda", 0)]
    assert q4._stream(None, 1 << 36, torch.zeros(1), None) is None
    assert q4._stream(7, Wrapper()) == 7


USE = """
import ctypes, sys
sys.path.insert(0, {root!r})
import torch
import gemm_q4_amd as q4
assert q4.__file__.startswith({root!r})
assert q4.q4_0_blocks_bytes(2, 64) == 72
assert q4.q4_0_select_kernel(1, 64, 64, q4.F32) > 0
c = q4.q4_0_kv_cache(0, 0, 500, 1, 16, 64)
assert q4.q4_0_attention_workspace_size(c, 2, q4.F16, 72, 163, 73) >= 0
k = torch.zeros(1, 1, 16, 64, dtype=torch.float16)
h = torch.zeros(1, 64)
for call in (lambda: q4.kv_cache(k, k.clone()), lambda: q4.rotary(),
             lambda: q4.residual_norm(h, h, h[0])):
    try:
        call()
    except ImportError as e:
        print(e)
    else:
        raise SystemExit("not refused")
"""


@pytest.mark.parametrize("extension,reason", [
    (None, "_bind"),
    ("raise ImportError('undefined symbol: x')", "undefined symbol"),
    ("torch_version = '0.1'", "built with torch 0.1, this is torch " + torch.__version__),
])
def test_products_do_not_need_the_extension_module(tmp_path, extension, reason):
    """Where the conveniences' module is missing, does not load or was built with
    another torch, the package imports and its products and C calls are there;
    the conveniences say what is wrong."""
    package = tmp_path / "gemm_q4_amd"
    package.mkdir()
    shutil.copy(q4.__file__, package / "__init__.py")
    if extension:
        (package / "_bind.py").write_text(extension)
    r = subprocess.run([sys.executable, "-c", USE.format(root=str(tmp_path))], cwd=tmp_path,
                       env={**os.environ, "Q4_0_LIBRARY": q4.LIB_PATH, "PYTHONPATH": ""},
                       capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr
    lines = r.stdout.strip().splitlines()
    assert len(lines) == 3 and all(reason in line and "build it again" in line for line in lines)


def refused(kind, message, call, *args, **kw):
    with pytest.raises(kind, match=message):
        call(*args, **kw)


def test_append_says_what_does_not_fit():
    """Each check by its own message: on the host every call is refused in the
    end, so the type of the error alone would show nothing."""
    k = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    c = q4.kv_cache(k, k.clone())
    q, kv = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    pos, slots = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    call = q4.kv_append
    refused(ValueError, "every tensor of the call must be on a GPU", call, c, None, q, kv, kv, pos,
            slots)
    refused(TypeError, "cache must come from kv_cache", call, k, None, None, kv, kv, pos, slots)
    refused(TypeError, "rot must come from rotary", call, c, k, q, kv, kv, pos, slots)
    refused(TypeError, "k must be a tensor", call, c, None, q, None, kv, pos, slots)
    refused(TypeError, "k must be float32 or float16", call, c, None, q, kv.double(), kv, pos,
            slots)
    refused(TypeError, "q, k and v must have one type", call, c, None, q, kv, kv.half(), pos, slots)
    refused(TypeError, "q, k and v must have one type", call, c, None, q.half(), kv, kv, pos, slots)
    refused(ValueError, "k has shape .* which does not fit", call, c, None, q, kv[:, :1], kv, pos,
            slots)
    refused(ValueError, "v has shape .* which does not fit", call, c, None, q, kv, kv[:2], pos,
            slots)
    refused(ValueError, "k must have two or three dimensions", call, c, None, q, kv[0, 0], kv, pos,
            slots)
    apart = torch.zeros(3, 2, 128)[..., ::2]
    refused(ValueError, "k's rows must be dense", call, c, None, q, apart, kv, pos, slots)
    refused(ValueError, "k's rows must be dense", call, c, None, q,
            kv.transpose(1, 2).contiguous().transpose(1, 2), kv, pos, slots)
    refused(ValueError, "q has shape .* which does not fit", call, c, None, q[:2], kv, kv, pos,
            slots, q_out=q)
    refused(ValueError, "q_out must have shape", call, c, None, q, kv, kv, pos, slots, q_out=q[:2])
    refused(TypeError, "q_out must be float32 or float16", call, c, None, q, kv, kv, pos, slots,
            q_out=q.bfloat16())
    refused(ValueError, "q_out must be contiguous", call, c, None, q, kv, kv, pos, slots,
            q_out=torch.zeros(3, 4, 128)[..., :64])
    refused(TypeError, "positions must be Int", call, c, None, q, kv, kv, pos.long(), slots)
    refused(ValueError, "positions must have shape", call, c, None, q, kv, kv, pos[:2], slots)
    refused(TypeError, "slots must be Long", call, c, None, q, kv, kv, pos, slots.int())
    refused(ValueError, "slots must have shape", call, c, None, q, kv, kv, pos, slots[:2])
    refused(ValueError, "slots must be contiguous", call, c, None, q, kv, kv, pos,
            torch.zeros(6, dtype=torch.int64)[::2])
    refused(ValueError, "norm weights of 32 do not fit heads of 64", call, c,
            q4.rotary(q_norm=torch.ones(32)), q, kv, kv, pos, slots)


def test_descriptors_say_what_does_not_fit():
    k = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    refused(TypeError, "k must be Half", q4.kv_cache, k.float(), k)
    refused(TypeError, "v must be Half", q4.kv_cache, k, k.float())
    refused(TypeError, "v must be a tensor", q4.kv_cache, k, None)
    refused(ValueError, "v must have shape", q4.kv_cache, k, k[:1])
    refused(ValueError, "k must be .pages, heads, page_size, dim.", q4.kv_cache, k[0], k[0])
    refused(ValueError, "k must be contiguous", q4.kv_cache, k.transpose(1, 2), k.transpose(1, 2))
    refused(TypeError, "inv_freq must be Float", q4.rotary, torch.ones(4).double())
    refused(ValueError, "inv_freq must have one dimension", q4.rotary, torch.ones(2, 4))
    refused(ValueError, "inv_freq must be contiguous", q4.rotary, torch.ones(8)[::2])
    refused(TypeError, "k_norm must be a tensor", q4.rotary, k_norm=[1.0])
    refused(ValueError, "q_norm and k_norm have different lengths", q4.rotary,
            q_norm=torch.ones(64), k_norm=torch.ones(32))


def test_attention_says_what_does_not_fit():
    k = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    c, q = q4.kv_cache(k, k.clone()), torch.zeros(3, 4, 64)
    start, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    call = q4.attention
    refused(ValueError, "every tensor of the call must be on a GPU", call, c, q, start, lens, table)
    refused(ValueError, "q must be .n, heads, 64.", call, c, q[..., :32], start, lens, table)
    refused(TypeError, "must be float32 or float16", call, c, q.bfloat16(), start, lens, table)
    refused(ValueError, "q's rows must be dense", call, c, torch.zeros(3, 4, 128)[..., :64], start,
            lens, table)
    refused(TypeError, "kv_len must be Int", call, c, q, start, lens.long(), table)
    refused(TypeError, "q_start must be Int", call, c, q, start.long(), lens, table)
    refused(ValueError, "q_start must have shape", call, c, q, start[:1], lens, table)
    refused(TypeError, "table must be Int", call, c, q, start, lens, table.long())
    refused(ValueError, "table must have shape", call, c, q, start, lens, table.expand(2, 2))
    refused(ValueError, "table must be contiguous", call, c, q, start, lens,
            torch.zeros(1, 4, dtype=torch.int32)[:, ::2])
    refused(TypeError, "y must be Float", call, c, q, start, lens, table, y=q.half())
    refused(ValueError, "y must have shape", call, c, q, start, lens, table, y=q[:2])
    refused(ValueError, "ws must be contiguous", call, c, q, start, lens, table,
            ws=torch.zeros(8, dtype=torch.uint8)[::2])


def test_residual_norm_says_what_does_not_fit():
    h, w, call = torch.zeros(3, 64), torch.ones(64), q4.residual_norm
    refused(ValueError, "every tensor of the call must be on a GPU", call, h, h.clone(), w, w)
    refused(TypeError, "h must be float32", call, h.half(), h)
    refused(ValueError, "h must be .n, dim.", call, h[0], h[0])
    refused(ValueError, "h's rows must be dense", call, torch.zeros(3, 128)[:, ::2], None, w)
    refused(ValueError, "b has shape .* which does not fit", call, h, h[:2])
    refused(TypeError, "b must be float32 or float16", call, h, h.bfloat16())
    refused(TypeError, "h_out must be float32", call, h, h, h_out=h.half())
    refused(ValueError, "h_out must have h's row stride", call, h, h,
            h_out=torch.zeros(3, 128)[:, :64])
    refused(TypeError, "gate must be float32", call, h, h, gate=h.half())
    refused(ValueError, "gate must be .n, dim., .n, 1. or .1, dim.", call, h, h,
            gate=torch.zeros(3, 2))
    refused(ValueError, "gate must be", call, h, h, gate=w)
    refused(ValueError, "pre must have shape", call, h, h, pre=w[:63])
    refused(TypeError, "pre must be Float", call, h, h, pre=w.half())
    refused(ValueError, "post must have shape", call, h, h, post=w[:63])
    refused(ValueError, "y has shape .* which does not fit", call, h, h, pre=w, y=h[:2])
    refused(TypeError, "y must be float32 or float16", call, h, h, pre=w, y=h.double())
