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
