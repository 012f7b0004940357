"""Python binding of libq4_0, the MI355X Q4_0 matmul library (include/q4_0.h).

Argument marshalling only: every q4_0_* function calls the C entry point of
the same name in ``libq4_0.so`` (built in this directory by
``gemm_q4_amd.build``), with the same arguments in the same order.  Pointer
arguments accept torch tensors (their ``data_ptr()``) or integers;
``stream`` accepts a ``torch.cuda.Stream``, an integer hipStream_t, or None
(torch's current stream on the tensors' device, else the null stream).
A negative status raises ``Q4Error``; the *_workspace_size queries return
the byte count.  There is no CPU fallback: importing this package fails if
the HIP library has not been built.

The library allocates nothing: calls that need scratch memory take a
caller-owned workspace.  The torch conveniences at the end of this file
(``matmul``, ``matmul_argmax``, ``matmul_routed``, ...) query the size and
allocate the workspace through torch's allocator, as they do their outputs.

torch is imported before the library is loaded: torch ships its own HIP
runtime under the same soname, and loading ours first would put two HIP
runtimes in one process, whose streams and contexts do not mix.  With torch
loaded first, libq4_0.so binds to torch's runtime; the import checks that
only one copy of the HIP runtime is mapped.
"""
from __future__ import annotations

import ctypes
import os

import torch  # must precede the CDLL below

_HERE = os.path.dirname(os.path.abspath(__file__))
# Q4_0_LIBRARY names another build of the same library (a tuning variant)
LIB_PATH = os.environ.get("Q4_0_LIBRARY") or os.path.join(_HERE, "libq4_0.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python -c 'import __graft_entry__ as g; g.build()')")

_lib = ctypes.CDLL(LIB_PATH)


def _mapped_runtimes():
    paths = {}
    try:
        with open("/proc/self/maps") as fh:
            for line in fh:
                parts = line.split()
                if len(parts) >= 6:
                    base = os.path.basename(parts[5])
                    for lib in ("libamdhip64.so",):
                        if base.startswith(lib):
                            paths.setdefault(lib, set()).add(os.path.realpath(parts[5]))
    except OSError:
        pass
    return paths


for _libname, _paths in _mapped_runtimes().items():
    if len(_paths) > 1:
        raise ImportError(f"two copies of {_libname} are loaded ({sorted(_paths)}); "
                          "import torch before anything that loads a HIP runtime")

# constants of include/q4_0.h
OK, EINVAL, ESHAPE, ENULL, EALIGN, EALIAS, EUNSUPPORTED, EHIP, EWORKSPACE = \
    0, -1, -2, -3, -4, -5, -6, -7, -8
F32, F16 = 0, 1
KERNEL_AUTO, KERNEL_GEMV_DPP, KERNEL_GEMV_MFMA, KERNEL_GEMM = 0, 1, 2, 3
KERNEL_NAMES = {KERNEL_AUTO: "auto", KERNEL_GEMV_DPP: "gemv_dpp",
                KERNEL_GEMV_MFMA: "gemv_mfma", KERNEL_GEMM: "gemm"}
MAX_IN, MAX_OUT, MAX_N = 1048576, 16777216, 65536
MAX_EXPERTS, MAX_ROUTED = 4096, 64
WORKSPACE_MAX, WORKSPACE_ALIGN = 134217728, 256
STATIC_SCRATCH_BYTES = 16777216
ROUTE_AUTO, ROUTE_BY_COLUMN, ROUTE_BY_EXPERT = 0, 1, 2

_i64, _vp, _int, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_f32 = ctypes.c_float
_szp = ctypes.POINTER(_sz)
_SIGS = {
    "q4_0_blocks_bytes": (_sz, [_i64, _i64]),
    "q4_0_packed_bytes": (_sz, [_i64, _i64]),
    "q4_0_repack": (_int, [_vp, _vp, _i64, _i64, _vp]),
    "q4_0_unpack": (_int, [_vp, _vp, _i64, _i64, _vp]),
    "q4_0_matmul": (_int, [_vp, _vp, _int, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "q4_0_matmul_ex": (_int, [_vp, _vp, _int, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "q4_0_matmul_workspace_size": (_int, [_i64, _i64, _i64, _int, _int, _szp]),
    "q4_0_matmul_static": (_int, [_vp, _vp, _int, _vp, _i64, _i64, _i64, _vp]),
    "q4_0_select_kernel": (_int, [_i64, _i64, _i64, _int]),
    "q4_0_kernel_supports": (_int, [_int, _i64, _i64, _i64, _int]),
    "q4_0_strerror": (ctypes.c_char_p, [_int]),
    "q4_0_version": (_int, []),
    "q4_0_matmul_grouped": (_int, [_vp, _int, _int, _i64, _vp, _sz, _vp]),
    "q4_0_grouped_workspace_size": (_int, [_vp, _int, _int, _i64, _szp]),
    "q4_0_matmul_argmax": (_int, [_vp, _vp, _int, _vp, _i64, _i64, _i64, _vp, _vp,
                                  _vp, _sz, _vp]),
    "q4_0_argmax_workspace_size": (_int, [_i64, _i64, _i64, _int, _szp]),
    "q4_0_quantize_x8": (_int, [_vp, _int, _vp, _vp, _i64, _i64, _vp]),
    "q4_0_matmul_w4a8": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "q4_0_w4a8_workspace_size": (_int, [_i64, _i64, _i64, _szp]),
    "q4_0_mfma_loop": (_int, [_vp, _i64, _i64, ctypes.POINTER(_i64), _vp]),
    "q4_0_stream_read": (_int, [_vp, _i64, _vp, _i64, _vp]),
    "q4_0_matmul_routed": (_int, [_vp, _i64, _vp, _int, _vp, _i64, _vp, _i64, _i64, _i64,
                                  _vp, _sz, _vp]),
    "q4_0_matmul_routed_ex": (_int, [_vp, _i64, _vp, _int, _vp, _i64, _vp, _i64, _i64, _i64,
                                     _int, _vp, _sz, _vp]),
    "q4_0_select_route": (_int, [_i64, _i64, _i64, _i64, _i64]),
    "q4_0_routed_workspace_size": (_int, [_i64, _i64, _i64, _i64, _i64, _int, _szp]),
    "q4_0_kv_append": (_int, [_vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _int, _i64,
                              _vp, _vp, _i64, _vp]),
    "q4_0_attention": (_int, [_vp, _vp, _i64, _int, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64,
                              _i64, _i64, _f32, _vp, _sz, _vp]),
    "q4_0_attention_workspace_size": (_int, [_vp, _i64, _int, _i64, _i64, _i64, _i64, _i64,
                                             _szp]),
    "q4_0_select_attention": (_int, [_vp, _i64, _int, _i64, _i64, _i64, _i64, _i64]),
    "q4_0_kv_append8": (_int, [_vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _int, _i64,
                               _vp, _vp, _i64, _vp]),
    "q4_0_kv_read8": (_int, [_vp, _vp, _i64, _vp, _vp, _int, _vp]),
    "q4_0_attention8": (_int, [_vp, _vp, _i64, _int, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64,
                               _i64, _i64, _f32, _vp, _sz, _vp]),
    "q4_0_attention8_workspace_size": (_int, [_vp, _i64, _int, _i64, _i64, _i64, _i64, _i64,
                                              _szp]),
    "q4_0_select_attention8": (_int, [_vp, _i64, _int, _i64, _i64, _i64, _i64, _i64]),
    "q4_0_embed": (_int, [_vp, _vp, _i64, _i64, _i64, _f32, _vp, _vp, _f32, _f32, _vp, _int,
                          _vp]),
    "q4_0_verify": (_int, [_vp, _i64, _vp, _i64, _int, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp,
                           _vp, _vp, _sz, _vp]),
    "q4_0_verify_workspace_size": (_int, [_i64, _i64, _i64, _int, _szp]),
    "q4_0_residual_norm": (_int, [_vp, _int, _i64, _vp, _vp, _i64, _i64, _f32, _vp, _vp, _i64,
                                  _vp, _f32, _f32, _vp, _int, _i64, _i64, _i64, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


class Q4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {q4_0_strerror(status)} (status {status})")


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _nbytes(ws, workspace_bytes):
    """Workspace size argument: as given, else the tensor's size, else 0."""
    if workspace_bytes is not None:
        return workspace_bytes
    if ws is None or isinstance(ws, int):
        return 0
    return ws.numel() * ws.element_size()


# torch's current stream as a bare handle where torch offers that (0.1 us
# against 2 us through a Stream object, as much as a small call's marshalling)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


class _Unusable:
    """Stands for the extension module where it cannot be used: every use of it
    says why.  The products and the C calls need libq4_0.so alone."""

    def __init__(self, reason):
        self._reason = reason

    def __getattr__(self, name):
        raise ImportError(f"the block operators' conveniences need gemm_q4_amd/_bind.so: "
                          f"{self._reason}; build it again "
                          "(python -c 'import __graft_entry__ as g; g.build()')")


def _load_bind():
    """The conveniences' extension module.  It is built against one torch, whose
    C++ interface another does not keep."""
    try:
        from . import _bind
    except ImportError as e:
        return _Unusable(str(e))
    if _bind.torch_version != torch.__version__:
        return _Unusable(f"it was built with torch {_bind.torch_version}, this is torch "
                         f"{torch.__version__}")
    _bind.setup(*(ctypes.cast(getattr(_lib, name), _vp).value
                  for name in ("q4_0_kv_append", "q4_0_attention", "q4_0_residual_norm",
                               "q4_0_kv_append8", "q4_0_attention8", "q4_0_kv_read8",
                               "q4_0_embed", "q4_0_verify")),
                _raw_stream)
    return _bind


_bind = _load_bind()


def _stream(stream, *tensors):
    if stream is None:
        for t in tensors:
            if isinstance(t, torch.Tensor):
                if t.is_cuda:
                    return _raw_stream(t.get_device())
            elif getattr(t, "is_cuda", False):      # a storage, a wrapper
                return torch.cuda.current_stream(t.device).cuda_stream
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> int:
    if status < 0:
        raise Q4Error(status, where)
    return status


def _size(fn, where, *args) -> int:
    out = _sz(0)
    _check(fn(*args, ctypes.byref(out)), where)
    return out.value


def q4_0_strerror(status: int) -> str:
    return _lib.q4_0_strerror(status).decode()


def q4_0_version() -> int:
    return _lib.q4_0_version()


def q4_0_blocks_bytes(out: int, in_: int) -> int:
    return _lib.q4_0_blocks_bytes(out, in_)


def q4_0_packed_bytes(out: int, in_: int) -> int:
    return _lib.q4_0_packed_bytes(out, in_)


def q4_0_repack(blocks, packed, out: int, in_: int, stream=None) -> None:
    _check(_lib.q4_0_repack(_ptr(blocks), _ptr(packed), out, in_,
                            _stream(stream, blocks, packed)), "q4_0_repack")


def q4_0_unpack(packed, blocks, out: int, in_: int, stream=None) -> None:
    _check(_lib.q4_0_unpack(_ptr(packed), _ptr(blocks), out, in_,
                            _stream(stream, packed, blocks)), "q4_0_unpack")


def q4_0_matmul(packed, x, x_dtype: int, y, n: int, out: int, in_: int,
                workspace=None, workspace_bytes=None, stream=None) -> None:
    _check(_lib.q4_0_matmul(_ptr(packed), _ptr(x), x_dtype, _ptr(y), n, out, in_,
                            _ptr(workspace), _nbytes(workspace, workspace_bytes),
                            _stream(stream, packed, x, y)), "q4_0_matmul")


def q4_0_matmul_ex(packed, x, x_dtype: int, y, n: int, out: int, in_: int,
                   kernel: int, workspace=None, workspace_bytes=None, stream=None) -> None:
    _check(_lib.q4_0_matmul_ex(_ptr(packed), _ptr(x), x_dtype, _ptr(y), n, out,
                               in_, kernel, _ptr(workspace),
                               _nbytes(workspace, workspace_bytes),
                               _stream(stream, packed, x, y)), "q4_0_matmul_ex")


def q4_0_matmul_static(packed, x, x_dtype: int, y, n: int, out: int, in_: int,
                       stream=None) -> None:
    _check(_lib.q4_0_matmul_static(_ptr(packed), _ptr(x), x_dtype, _ptr(y), n, out, in_,
                                   _stream(stream, packed, x, y)), "q4_0_matmul_static")


def q4_0_matmul_workspace_size(n: int, out: int, in_: int, x_dtype: int = F32,
                               kernel: int = KERNEL_AUTO) -> int:
    return _size(_lib.q4_0_matmul_workspace_size, "q4_0_matmul_workspace_size",
                 n, out, in_, x_dtype, kernel)


class q4_0_linear(ctypes.Structure):
    """One linear of q4_0_matmul_grouped (struct q4_0_linear of include/q4_0.h)."""
    _fields_ = [("packed", _vp), ("x", _vp), ("y", _vp), ("out", _i64), ("in_", _i64)]


MAX_GROUP = 8


def _linears(linears):
    arr = (q4_0_linear * max(1, len(linears)))()
    tensors = []
    for i, (packed, x, y, out, in_) in enumerate(linears):
        arr[i] = q4_0_linear(_ptr(packed), _ptr(x), _ptr(y), out, in_)
        tensors += [packed, x, y]
    return arr, tensors


def q4_0_matmul_grouped(linears, x_dtype: int, n: int, workspace=None, workspace_bytes=None,
                        stream=None) -> None:
    """linears: sequence of (packed, x, y, out, in) with tensors or pointers."""
    arr, tensors = _linears(linears)
    _check(_lib.q4_0_matmul_grouped(ctypes.cast(arr, _vp), len(linears), x_dtype, n,
                                    _ptr(workspace), _nbytes(workspace, workspace_bytes),
                                    _stream(stream, *tensors)), "q4_0_matmul_grouped")


def q4_0_grouped_workspace_size(linears, x_dtype: int, n: int) -> int:
    arr, _ = _linears(linears)
    return _size(_lib.q4_0_grouped_workspace_size, "q4_0_grouped_workspace_size",
                 ctypes.cast(arr, _vp), len(linears), x_dtype, n)


def q4_0_matmul_argmax(packed, x, x_dtype: int, y, n: int, out: int, in_: int,
                       max_val, max_idx, workspace=None, workspace_bytes=None,
                       stream=None) -> None:
    _check(_lib.q4_0_matmul_argmax(_ptr(packed), _ptr(x), x_dtype, _ptr(y), n, out, in_,
                                   _ptr(max_val), _ptr(max_idx), _ptr(workspace),
                                   _nbytes(workspace, workspace_bytes),
                                   _stream(stream, packed, x, max_val)), "q4_0_matmul_argmax")


def q4_0_argmax_workspace_size(n: int, out: int, in_: int, x_dtype: int = F32) -> int:
    return _size(_lib.q4_0_argmax_workspace_size, "q4_0_argmax_workspace_size",
                 n, out, in_, x_dtype)


def q4_0_quantize_x8(x, x_dtype: int, q, d, n: int, in_: int, stream=None) -> None:
    _check(_lib.q4_0_quantize_x8(_ptr(x), x_dtype, _ptr(q), _ptr(d), n, in_,
                                 _stream(stream, x, q, d)), "q4_0_quantize_x8")


def q4_0_matmul_w4a8(packed, q, d, y, n: int, out: int, in_: int, workspace=None,
                     workspace_bytes=None, stream=None) -> None:
    _check(_lib.q4_0_matmul_w4a8(_ptr(packed), _ptr(q), _ptr(d), _ptr(y), n, out, in_,
                                 _ptr(workspace), _nbytes(workspace, workspace_bytes),
                                 _stream(stream, packed, q, y)), "q4_0_matmul_w4a8")


def q4_0_w4a8_workspace_size(n: int, out: int, in_: int) -> int:
    return _size(_lib.q4_0_w4a8_workspace_size, "q4_0_w4a8_workspace_size", n, out, in_)


def q4_0_select_kernel(n: int, out: int, in_: int, x_dtype: int = F32) -> int:
    return _check(_lib.q4_0_select_kernel(n, out, in_, x_dtype), "q4_0_select_kernel")


def q4_0_kernel_supports(kernel: int, n: int, out: int, in_: int,
                         x_dtype: int = F32) -> bool:
    st = _lib.q4_0_kernel_supports(kernel, n, out, in_, x_dtype)
    if st == EUNSUPPORTED:
        return False
    _check(st, "q4_0_kernel_supports")
    return True


def q4_0_matmul_routed(experts, n_experts: int, x, x_dtype: int, route, k: int, y, n: int,
                       out: int, in_: int, workspace=None, workspace_bytes=None,
                       stream=None) -> None:
    _check(_lib.q4_0_matmul_routed(_ptr(experts), n_experts, _ptr(x), x_dtype, _ptr(route), k,
                                   _ptr(y), n, out, in_, _ptr(workspace),
                                   _nbytes(workspace, workspace_bytes),
                                   _stream(stream, y, x)), "q4_0_matmul_routed")


def q4_0_matmul_routed_ex(experts, n_experts: int, x, x_dtype: int, route, k: int, y, n: int,
                          out: int, in_: int, route_kernel: int, workspace=None,
                          workspace_bytes=None, stream=None) -> None:
    _check(_lib.q4_0_matmul_routed_ex(_ptr(experts), n_experts, _ptr(x), x_dtype, _ptr(route),
                                      k, _ptr(y), n, out, in_, route_kernel, _ptr(workspace),
                                      _nbytes(workspace, workspace_bytes),
                                      _stream(stream, y, x)), "q4_0_matmul_routed_ex")


def q4_0_select_route(n: int, k: int, n_experts: int, out: int, in_: int) -> int:
    return _check(_lib.q4_0_select_route(n, k, n_experts, out, in_), "q4_0_select_route")


def q4_0_routed_workspace_size(n: int, k: int, n_experts: int, out: int, in_: int,
                               route_kernel: int = ROUTE_AUTO) -> int:
    return _size(_lib.q4_0_routed_workspace_size, "q4_0_routed_workspace_size",
                 n, k, n_experts, out, in_, route_kernel)


def q4_0_mfma_loop(sink, workgroups: int, iters: int, stream=None) -> int:
    """Enqueue the MFMA loop measurement aid; returns the launch's flops."""
    flops = _i64(0)
    _check(_lib.q4_0_mfma_loop(_ptr(sink), workgroups, iters, ctypes.byref(flops),
                               _stream(stream, sink)), "q4_0_mfma_loop")
    return flops.value


def q4_0_stream_read(src, nbytes: int, sink, workgroups: int, stream=None) -> None:
    """Enqueue the streaming-read measurement aid (nbytes == 0: an empty launch)."""
    _check(_lib.q4_0_stream_read(_ptr(src), nbytes, _ptr(sink), workgroups,
                                 _stream(stream, sink)), "q4_0_stream_read")


class q4_0_kv_cache(ctypes.Structure):
    """A paged cache's descriptor (struct q4_0_kv_cache of include/q4_0.h)."""
    _fields_ = [("k", _vp), ("v", _vp), ("pages", _i64), ("heads", _i64), ("page_size", _i64),
                ("dim", _i64)]


class q4_0_kv_cache8(ctypes.Structure):
    """An 8-bit paged cache's descriptor (struct q4_0_kv_cache8 of include/q4_0.h)."""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("pages", _i64),
                ("heads", _i64), ("page_size", _i64), ("dim", _i64)]


class q4_0_rotary(ctypes.Structure):
    """Position rotation and per-head norms (struct q4_0_rotary of include/q4_0.h)."""
    _fields_ = [("inv_freq", _vp), ("rot_dim", _i64), ("interleaved", _int),
                ("amplitude", _f32), ("q_norm", _vp), ("k_norm", _vp), ("eps", _f32),
                ("weight_offset", _f32)]


def _ref(struct):
    """Address of a descriptor: a ctypes structure, or kv_cache()'s, kv_cache8()'s or
    rotary()'s."""
    if struct is None:
        return None
    return ctypes.addressof(struct) if isinstance(struct, ctypes.Structure) else struct.address


def q4_0_kv_append(cache, rot, q, q_stride: int, k, k_stride: int, v, v_stride: int,
                   x_dtype: int, q_out, q_dtype: int, q_heads: int, positions, slots, n: int,
                   stream=None) -> None:
    """cache: q4_0_kv_cache; rot: q4_0_rotary or None."""
    _check(_lib.q4_0_kv_append(_ref(cache), _ref(rot), _ptr(q), q_stride, _ptr(k), k_stride,
                               _ptr(v), v_stride, x_dtype, _ptr(q_out), q_dtype, q_heads,
                               _ptr(positions), _ptr(slots), n, _stream(stream, k, v)),
           "q4_0_kv_append")


def q4_0_attention(cache, q, q_stride: int, x_dtype: int, q_heads: int, y, n: int, q_start,
                   kv_len, table, table_stride: int, batch: int, window: int, sinks: int,
                   scale: float, workspace=None, workspace_bytes=None, stream=None) -> None:
    """cache: q4_0_kv_cache."""
    _check(_lib.q4_0_attention(_ref(cache), _ptr(q), q_stride, x_dtype, q_heads, _ptr(y), n,
                               _ptr(q_start), _ptr(kv_len), _ptr(table), table_stride, batch,
                               window, sinks, scale, _ptr(workspace),
                               _nbytes(workspace, workspace_bytes), _stream(stream, q, y)),
           "q4_0_attention")


def q4_0_attention_workspace_size(cache, q_heads: int, x_dtype: int, n: int, table_stride: int,
                                  batch: int, window: int = 0, sinks: int = 0) -> int:
    return _size(_lib.q4_0_attention_workspace_size, "q4_0_attention_workspace_size",
                 _ref(cache), q_heads, x_dtype, n, table_stride, batch, window, sinks)


def q4_0_select_attention(cache, q_heads: int, x_dtype: int, n: int, table_stride: int,
                          batch: int, window: int = 0, sinks: int = 0) -> int:
    return _check(_lib.q4_0_select_attention(_ref(cache), q_heads, x_dtype, n, table_stride, batch,
                                             window, sinks), "q4_0_select_attention")


def q4_0_kv_append8(cache, rot, q, q_stride: int, k, k_stride: int, v, v_stride: int,
                    x_dtype: int, q_out, q_dtype: int, q_heads: int, positions, slots, n: int,
                    stream=None) -> None:
    """cache: q4_0_kv_cache8; rot: q4_0_rotary or None."""
    _check(_lib.q4_0_kv_append8(_ref(cache), _ref(rot), _ptr(q), q_stride, _ptr(k), k_stride,
                                _ptr(v), v_stride, x_dtype, _ptr(q_out), q_dtype, q_heads,
                                _ptr(positions), _ptr(slots), n, _stream(stream, k, v)),
           "q4_0_kv_append8")


def q4_0_kv_read8(cache, slots, n: int, k, v, y_dtype: int, stream=None) -> None:
    """cache: q4_0_kv_cache8."""
    _check(_lib.q4_0_kv_read8(_ref(cache), _ptr(slots), n, _ptr(k), _ptr(v), y_dtype,
                              _stream(stream, slots, k, v)), "q4_0_kv_read8")


def q4_0_attention8(cache, q, q_stride: int, x_dtype: int, q_heads: int, y, n: int, q_start,
                    kv_len, table, table_stride: int, batch: int, window: int, sinks: int,
                    scale: float, workspace=None, workspace_bytes=None, stream=None) -> None:
    """cache: q4_0_kv_cache8."""
    _check(_lib.q4_0_attention8(_ref(cache), _ptr(q), q_stride, x_dtype, q_heads, _ptr(y), n,
                                _ptr(q_start), _ptr(kv_len), _ptr(table), table_stride, batch,
                                window, sinks, scale, _ptr(workspace),
                                _nbytes(workspace, workspace_bytes), _stream(stream, q, y)),
           "q4_0_attention8")


def q4_0_attention8_workspace_size(cache, q_heads: int, x_dtype: int, n: int, table_stride: int,
                                   batch: int, window: int = 0, sinks: int = 0) -> int:
    return _size(_lib.q4_0_attention8_workspace_size, "q4_0_attention8_workspace_size",
                 _ref(cache), q_heads, x_dtype, n, table_stride, batch, window, sinks)


def q4_0_select_attention8(cache, q_heads: int, x_dtype: int, n: int, table_stride: int,
                           batch: int, window: int = 0, sinks: int = 0) -> int:
    return _check(_lib.q4_0_select_attention8(_ref(cache), q_heads, x_dtype, n, table_stride,
                                              batch, window, sinks), "q4_0_select_attention8")


def q4_0_embed(packed, tokens, n: int, out: int, in_: int, scale: float, h, pre,
               weight_offset: float, eps: float, y, y_dtype: int, stream=None) -> None:
    _check(_lib.q4_0_embed(_ptr(packed), _ptr(tokens), n, out, in_, scale, _ptr(h), _ptr(pre),
                           weight_offset, eps, _ptr(y), y_dtype, _stream(stream, h, tokens)),
           "q4_0_embed")


def q4_0_verify(logits, stride: int, drafted, drafted_stride: int, x_dtype: int, vocab: int,
                tokens, q_start, n: int, batch: int, temperature, uniform, accepted, next_,
                workspace=None, workspace_bytes=None, stream=None) -> None:
    _check(_lib.q4_0_verify(_ptr(logits), stride, _ptr(drafted), drafted_stride, x_dtype, vocab,
                            _ptr(tokens), _ptr(q_start), n, batch, _ptr(temperature),
                            _ptr(uniform), _ptr(accepted), _ptr(next_), _ptr(workspace),
                            _nbytes(workspace, workspace_bytes),
                            _stream(stream, logits, accepted)), "q4_0_verify")


def q4_0_verify_workspace_size(n: int, batch: int, vocab: int, drafted: bool = False) -> int:
    return _size(_lib.q4_0_verify_workspace_size, "q4_0_verify_workspace_size", n, batch, vocab,
                 int(bool(drafted)))


def q4_0_residual_norm(b, b_dtype: int, b_stride: int, post, gate, gate_row: int, gate_col: int,
                       alpha: float, h, h_out, h_stride: int, pre, weight_offset: float,
                       eps: float, y, y_dtype: int, y_stride: int, n: int, dim: int,
                       stream=None) -> None:
    _check(_lib.q4_0_residual_norm(_ptr(b), b_dtype, b_stride, _ptr(post), _ptr(gate), gate_row,
                                   gate_col, alpha, _ptr(h), _ptr(h_out), h_stride, _ptr(pre),
                                   weight_offset, eps, _ptr(y), y_dtype, y_stride, n, dim,
                                   _stream(stream, h, y)), "q4_0_residual_norm")


# ---- torch conveniences (allocation through torch, then the C calls above) --
_DTYPE_CODES = {torch.float32: F32, torch.float16: F16}


def dtype_code(x) -> int:
    """Q4_0_F32 or Q4_0_F16 for a torch tensor's dtype."""
    code = _DTYPE_CODES.get(x.dtype)
    if code is not None:
        return code
    raise TypeError(f"x must be float32 or float16, not {x.dtype}")


def workspace(nbytes: int, device):
    """A workspace of nbytes on `device` (torch's allocator aligns to at least
    512 bytes), or None when nothing is needed."""
    import torch
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def repacked(blocks, out: int, in_: int, stream=None):
    """Repack a uint8 CUDA tensor of GGUF blocks into a new packed tensor."""
    import torch
    packed = torch.empty(q4_0_packed_bytes(out, in_), dtype=torch.uint8,
                         device=blocks.device)
    q4_0_repack(blocks, packed, out, in_, stream)
    return packed


def matmul(packed, x, out: int, y=None, kernel: int = KERNEL_AUTO, stream=None, ws=None):
    """y[n x out] = x . W^T for a 2-D CUDA tensor x (float32 or float16)."""
    import torch
    n, in_ = x.shape
    if y is None:
        y = torch.empty((n, out), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(q4_0_matmul_workspace_size(n, out, in_, dtype_code(x), kernel), x.device)
    q4_0_matmul_ex(packed, x, dtype_code(x), y, n, out, in_, kernel, ws, None, stream)
    return y


def matmul_grouped(linears, x_dtype: int, n: int, stream=None, ws=None):
    """q4_0_matmul_grouped with its workspace allocated through torch."""
    if ws is None and linears:
        dev = next(t.device for t in linears[0][:3] if hasattr(t, "device"))
        ws = workspace(q4_0_grouped_workspace_size(linears, x_dtype, n), dev)
    q4_0_matmul_grouped(linears, x_dtype, n, ws, None, stream)


def matmul_argmax(packed, x, out: int, y=None, stream=None, ws=None):
    """(max value [n] float32, max index [n] int32) of y = x . W^T per row;
    y is written when given."""
    import torch
    n, in_ = x.shape
    mv = torch.empty(n, dtype=torch.float32, device=x.device)
    mi = torch.empty(n, dtype=torch.int32, device=x.device)
    if ws is None:
        ws = workspace(q4_0_argmax_workspace_size(n, out, in_, dtype_code(x)), x.device)
    q4_0_matmul_argmax(packed, x, dtype_code(x), y, n, out, in_, mv, mi, ws, None, stream)
    return mv, mi


def quantize_x8(x, stream=None):
    """(q int8 [n x in], d float32 [n x in/32]) of a 2-D CUDA tensor x."""
    import torch
    n, in_ = x.shape
    q = torch.empty((n, in_), dtype=torch.int8, device=x.device)
    d = torch.empty((n, in_ // 32), dtype=torch.float32, device=x.device)
    q4_0_quantize_x8(x, dtype_code(x), q, d, n, in_, stream)
    return q, d


def matmul_w4a8(packed, q, d, out: int, y=None, stream=None, ws=None):
    """y [n x out] of the W4A8 product on quantized activations (q, d)."""
    import torch
    n, in_ = q.shape
    if y is None:
        y = torch.empty((n, out), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(q4_0_w4a8_workspace_size(n, out, in_), q.device)
    q4_0_matmul_w4a8(packed, q, d, y, n, out, in_, ws, None, stream)
    return y


def matmul_routed(experts, n_experts: int, x, route, out: int, y=None, stream=None,
                  route_kernel: int = ROUTE_AUTO, ws=None):
    """y[t*k + j] = x[t] . W_{route[t, j]}^T for a stack of repacked experts
    (one flat uint8 tensor, n_experts matrices of q4_0_packed_bytes apart) and
    route an int32 [n x k] device tensor.  Returns y [n*k x out]."""
    import torch
    n, in_ = x.shape
    k = route.shape[1]
    if y is None:
        y = torch.empty((n * k, out), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(q4_0_routed_workspace_size(n, k, n_experts, out, in_, route_kernel),
                       x.device)
    q4_0_matmul_routed_ex(experts, n_experts, x, dtype_code(x), route, k, y, n, out, in_,
                          route_kernel, ws, None, stream)
    return y


# The checks of the block operators' conveniences are made by the extension
# module (csrc/q4_0_bind.cpp): here they would cost more than a small kernel.
def _handle(stream):
    """A stream argument as an integer, None for torch's current stream."""
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _new(stream, *args, **kw):
    """torch.empty for a call on `stream`: what the call alone holds goes back to
    that stream's pool, where its next owner is ordered after the call."""
    if stream is None:
        return torch.empty(*args, **kw)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=kw["device"])
    with torch.cuda.stream(stream):
        return torch.empty(*args, **kw)


def kv_cache(k, v):
    """Descriptor of a paged cache: k and v float16 [pages, heads, page_size,
    dim] CUDA tensors, which it keeps alive and reads anew at every use, so
    that one whose data was replaced is followed.  Any call here that takes a
    q4_0_kv_cache takes it too."""
    return _bind.kv_cache(k, v)


def kv_cache8(k, v, k_scale, v_scale):
    """Descriptor of an 8-bit paged cache: k and v int8 [pages, heads, page_size, dim]
    and their scales float32 [pages, heads, page_size], CUDA tensors, held and read
    anew as by kv_cache().  kv_append, kv_read and attention take it."""
    return _bind.kv_cache8(k, v, k_scale, v_scale)


def rotary(inv_freq=None, interleaved: bool = False, amplitude: float = 1.0, q_norm=None,
           k_norm=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """Descriptor of a rotation (inv_freq: float32 [rot_dim / 2], or None) and of
    per-head norms (float32 [dim] weights, or None); it keeps the tensors alive
    and reads them anew at every use, as kv_cache() does."""
    return _bind.rotary(inv_freq, interleaved, amplitude, q_norm, k_norm, eps, weight_offset)


def kv_append(cache, rot, q, k, v, positions, slots, q_out=None, stream=None):
    """Append k and v to `cache` (kv_cache()'s; kv_cache8()'s: in 8 bits) and rotate
    q: q [n, q_heads * dim] (or None), k and v [n, heads * dim], or the same with
    the heads as a dimension; rows may be slices of wider ones.  positions int32 [n],
    slots int64 [n].  Returns the rotated q [n, q_heads, dim]: q_out, or a new tensor
    of q's type."""
    if q is not None and q_out is None:
        heads = q.shape[1] if q.dim() == 3 else q.shape[1] // cache.dim
        q_out = _new(stream, (q.shape[0], heads, cache.dim), dtype=q.dtype, device=q.device)
    _check(_bind.kv_append(cache, rot, q, k, v, positions, slots, q_out, _handle(stream)),
           "q4_0_kv_append")
    return None if q is None else q_out


def kv_read(cache, slots, k=None, v=None, dtype=None, stream=None):
    """(k, v): rows of an 8-bit cache (kv_cache8()'s) as numbers, [n, heads, dim] of
    `dtype` (float16 unless given): as given, or new tensors.  slots int64 [n]."""
    shape = (slots.shape[0], cache.heads, cache.dim)
    if dtype is None:
        given = k if k is not None else v
        dtype = torch.float16 if given is None else given.dtype
    if k is None:
        k = _new(stream, shape, dtype=dtype, device=slots.device)
    if v is None:
        v = _new(stream, shape, dtype=dtype, device=slots.device)
    _check(_bind.kv_read(cache, slots, k, v, _handle(stream)), "q4_0_kv_read8")
    return k, v


def attention(cache, q, q_start, kv_len, table, window: int = 0, sinks: int = 0, scale=None,
              y=None, stream=None, ws=None):
    """Attention of q [n, q_heads, dim] over `cache` (q4_0_attention; kv_cache8()'s:
    q4_0_attention8): q_start int32 [batch + 1], kv_len int32 [batch], table int32
    [batch, pages of the longest].  scale: dim ** -0.5 unless given.  Returns y, like q."""
    if y is None:
        y = _new(stream, q.shape, dtype=q.dtype, device=q.device)
    if ws is None:
        size = (q4_0_attention8_workspace_size if _bind.is_cache8(cache)
                else q4_0_attention_workspace_size)
        need = size(cache, q.shape[1], dtype_code(q), q.shape[0], table.shape[-1],
                    kv_len.shape[0], window, sinks)
        ws = _new(stream, need, dtype=torch.uint8, device=q.device) if need else None
    if scale is None:
        scale = cache.dim ** -0.5
    _check(_bind.attention(cache, q, q_start, kv_len, table, window, sinks, scale, y, ws,
                           _handle(stream)), "q4_0_attention")
    return y


def residual_norm(h, b=None, pre=None, post=None, gate=None, alpha: float = 1.0,
                  eps: float = 1e-6, weight_offset: float = 0.0, h_out=None, y=None,
                  y_dtype=None, stream=None):
    """h_out = h + alpha * gate * N(b; post) and y = N(h_out; pre)
    (q4_0_residual_norm) for h float32 [n, dim] and b [n, dim] float32 or
    float16.  gate float32 [n, dim], [n, 1] or [1, dim]; post, pre float32
    [dim] or None (no norm).  Without b, y = N(h; pre).  Returns (h_out, y):
    as given, or new tensors (y of y_dtype, float32 unless given; None without
    pre).  h_out may be h."""
    if b is None:
        h_out = h
    elif h_out is None:
        if h.is_contiguous():
            h_out = _new(stream, h.shape, dtype=h.dtype, device=h.device)
        else:           # rows as far apart as h's
            n, dim = h.shape
            h_out = _new(stream, (n, max(h.stride(0), dim)), dtype=h.dtype,
                         device=h.device)[:, :dim]
    if pre is None:
        y = None
    elif y is None:
        y = _new(stream, h.shape, dtype=y_dtype or torch.float32, device=h.device)
    _check(_bind.residual_norm(h, b, pre, post, gate, alpha, eps, weight_offset, h_out, y,
                               _handle(stream)), "q4_0_residual_norm")
    return h_out, y


def embed(packed, tokens, out: int, in_: int, scale: float = 1.0, pre=None, eps: float = 1e-6,
          weight_offset: float = 0.0, h=None, y=None, y_dtype=None, stream=None):
    """(h, y): h [n, in_] float32 the rows `tokens` (int32 [n]) of a repacked table,
    times scale, and y = N(h; pre) (q4_0_embed): as given, or new tensors (y of
    y_dtype, float32 unless given; None without pre)."""
    shape = (tokens.shape[0], in_)
    if h is None:
        h = _new(stream, shape, dtype=torch.float32, device=tokens.device)
    if pre is None:
        y = None
    elif y is None:
        y = _new(stream, shape, dtype=y_dtype or torch.float32, device=tokens.device)
    _check(_bind.embed(packed, tokens, out, in_, scale, pre, eps, weight_offset, h, y,
                       _handle(stream)), "q4_0_embed")
    return h, y


def verify(logits, tokens, q_start, uniform, draft_logits=None, temperature=None, accepted=None,
           following=None, stream=None, ws=None):
    """(accepted, following), int32 [batch]: how many of each conversation's drafted
    tokens the target's logits [n, vocab] take, and the token that follows them
    (q4_0_verify).  tokens int32 [n] (the step's tokens: row t judges tokens[t + 1]),
    q_start int32 [batch + 1], uniform float32 [n, 2], draft_logits like logits or
    None (drafts that were picked), temperature float32 [batch] or None (1)."""
    batch = q_start.shape[0] - 1
    if accepted is None:
        accepted = _new(stream, batch, dtype=torch.int32, device=logits.device)
    if following is None:
        following = _new(stream, batch, dtype=torch.int32, device=logits.device)
    if ws is None:
        need = q4_0_verify_workspace_size(logits.shape[0], batch, logits.shape[-1],
                                          draft_logits is not None)
        ws = _new(stream, need, dtype=torch.uint8, device=logits.device)
    _check(_bind.verify(logits, tokens, q_start, uniform, draft_logits, temperature, accepted,
                        following, ws, _handle(stream)), "q4_0_verify")
    return accepted, following
