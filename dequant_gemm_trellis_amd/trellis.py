"""ctypes binding over libtrellis.so (include/trellis.h, trellis_grouped.h, trellis_mlp.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI. PyTorch supplies device memory and the stream.
Importing this module raises ImportError when the library is not built; there
is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os
from typing import NamedTuple

import torch

from .synth import Shape

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtrellis.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
        "(hipcc --offload-arch=gfx950)")
_lib = C.CDLL(LIB_PATH)

OK = 0
ERR_NULL = -1
ERR_GEOMETRY = -2
ERR_ALIGN = -3
ERR_LUT = -4
ERR_WORKSPACE = -5
ERR_HIP = -6
ERR_OVERLAP = -7
OP_GEMV = 0
OP_GEMV_SCATTER = 1
OP_PREFILL = 2
MAX_M = 32

# Every function the headers under include/ declare, for the export check.
EXPORTED = ("trellis_lut_upload", "trellis_gemv", "trellis_gemv_dual", "trellis_gemv_scatter",
            "trellis_prefill", "trellis_prefill_dual", "trellis_gate_up_swiglu",
            "trellis_gemv_scatter_static", "trellis_static_scratch_bytes", "trellis_workspace_bytes",
            "trellis_expand", "trellis_repack", "trellis_strerror", "trellis_gather_probe",
            "trellis_gather_probe_values", "trellis_gather_probe_out_floats", "trellis_route",
            "trellis_route_workspace_bytes", "trellis_dispatch", "trellis_combine",
            "trellis_combine_backward", "trellis_adapters", "trellis_adapters_backward",
            "trellis_adapters_workspace_bytes", "trellis_experts",
            "trellis_experts_workspace_bytes", "trellis_experts_mlp",
            "trellis_experts_mlp_workspace_bytes", "trellis_keep", "trellis_restore",
            "trellis_swiglu", "trellis_swiglu_backward", "trellis_adapters_backward_kept")
PROBE_PAIR_B64, PROBE_COPIES8_B32, PROBE_SINGLE_B32 = 0, 1, 2


class Geometry(C.Structure):
    _fields_ = [("axis", C.c_int32), ("T", C.c_int32), ("L", C.c_int32), ("k", C.c_int32),
                ("in_features", C.c_int32), ("out_features", C.c_int32),
                ("block_interleave", C.c_int32)]

    @classmethod
    def of(cls, shape: Shape) -> "Geometry":
        return cls(shape.axis, shape.T, shape.L, shape.k, shape.in_features, shape.out_features,
                   shape.block_interleave)


_vp = C.c_void_p
_GP = C.POINTER(Geometry)
_lib.trellis_lut_upload.argtypes = [_vp, C.c_int32, _vp, _vp]
_lib.trellis_gemv.argtypes = [_vp, _vp, _vp, _vp, _GP, _vp, _vp]
_lib.trellis_gemv_dual.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _GP, _vp]
_lib.trellis_gemv_scatter.argtypes = [_vp, _vp, _vp, _vp, _GP, _vp, C.c_size_t, _vp, _vp]
_lib.trellis_prefill.argtypes = [_vp, C.c_int32, _vp, _vp, _vp, _GP, _vp, C.c_size_t, _vp, _vp]
_lib.trellis_prefill_dual.argtypes = [_vp, C.c_int32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _GP,
                                      _vp]
_lib.trellis_gate_up_swiglu.argtypes = [_vp, C.c_int32, _vp, _vp, _vp, _vp, _vp, _vp, _GP, _vp,
                                        _vp]
_lib.trellis_gemv_scatter_static.argtypes = [_vp, _vp, _vp, _vp, _GP, _vp, _vp]
_lib.trellis_static_scratch_bytes.argtypes = []
_lib.trellis_static_scratch_bytes.restype = C.c_size_t
_lib.trellis_workspace_bytes.argtypes = [_GP, C.c_int32, C.c_int32]
_lib.trellis_workspace_bytes.restype = C.c_size_t
_lib.trellis_expand.argtypes = [_vp, _vp, _vp, _GP, _vp, _vp]
_lib.trellis_repack.argtypes = [_vp, _vp, _GP, C.c_int32, _vp]
_lib.trellis_strerror.argtypes = [C.c_int]
_lib.trellis_strerror.restype = C.c_char_p
_lib.trellis_gather_probe.argtypes = [C.c_int32, C.c_int32, _vp, C.c_size_t, _vp]
_lib.trellis_gather_probe.restype = C.c_int
_lib.trellis_gather_probe_values.argtypes = [C.c_int32, C.c_int32]
_lib.trellis_gather_probe_values.restype = C.c_uint64
_lib.trellis_gather_probe_out_floats.argtypes = []
_lib.trellis_gather_probe_out_floats.restype = C.c_size_t
class AdapterSet(C.Structure):
    _fields_ = [("a", C.c_void_p), ("b", C.c_void_p), ("scales", C.c_void_p),
                ("count", C.c_int32), ("rank", C.c_int32), ("in_features", C.c_int32),
                ("out_features", C.c_int32)]


class ExpertSet(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("lut", C.c_void_p), ("g", Geometry)]


class _KeptRows(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("exponents", C.c_void_p)]


_AP = C.POINTER(AdapterSet)
_EP = C.POINTER(ExpertSet)
_KP = C.POINTER(_KeptRows)
_i32 = C.c_int32
_lib.trellis_adapters.argtypes = [_vp, _vp, _i32, _AP, _vp, _vp, _vp, _vp, C.c_size_t, _vp]
_lib.trellis_adapters_backward.argtypes = [_vp, _vp, _vp, _vp, _i32, _AP, _vp, _vp, _vp, _vp, _vp,
                                           C.c_size_t, _vp]
_lib.trellis_adapters_workspace_bytes.argtypes = [_AP, _i32, _i32]
_lib.trellis_adapters_workspace_bytes.restype = C.c_size_t
_lib.trellis_experts.argtypes = [_vp, _i32, _vp, _i32, _vp, _vp, _vp, _GP, _vp, _vp, C.c_size_t, _vp]
_lib.trellis_experts_workspace_bytes.argtypes = [_GP, _i32, _i32]
_lib.trellis_experts_workspace_bytes.restype = C.c_size_t
_lib.trellis_route.argtypes = [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, C.c_size_t, _vp]
_lib.trellis_route_workspace_bytes.argtypes = [_i32, _i32, _i32]
_lib.trellis_route_workspace_bytes.restype = C.c_size_t
_lib.trellis_dispatch.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp, _vp]
_lib.trellis_combine.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp]
_lib.trellis_combine_backward.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]
_lib.trellis_experts_mlp.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _EP, _EP, _vp, _vp, C.c_size_t, _vp]
_lib.trellis_experts_mlp_workspace_bytes.argtypes = [_i32, _i32, _i32, _EP, _EP]
_lib.trellis_experts_mlp_workspace_bytes.restype = C.c_size_t
_lib.trellis_keep.argtypes = [_vp, _i32, _i32, _KP, _vp]
_lib.trellis_restore.argtypes = [_KP, _i32, _i32, _vp, _vp]
_lib.trellis_swiglu.argtypes = [_vp, _i32, _i32, _vp, _KP, _vp]
_lib.trellis_swiglu_backward.argtypes = [_vp, _vp, _KP, _i32, _i32, _vp, _vp, _vp]
_lib.trellis_adapters_backward_kept.argtypes = [_vp, _KP, _vp, _vp, _i32, _AP, _vp, _vp, _vp, _vp, _vp,
                                                C.c_size_t, _vp]
for _f in ("trellis_lut_upload", "trellis_gemv", "trellis_gemv_dual", "trellis_gemv_scatter",
           "trellis_prefill", "trellis_prefill_dual", "trellis_gate_up_swiglu", "trellis_expand",
           "trellis_repack", "trellis_gemv_scatter_static", "trellis_route", "trellis_dispatch",
           "trellis_combine", "trellis_combine_backward", "trellis_adapters",
           "trellis_adapters_backward", "trellis_experts", "trellis_experts_mlp", "trellis_keep",
           "trellis_restore", "trellis_swiglu", "trellis_swiglu_backward",
           "trellis_adapters_backward_kept"):
    getattr(_lib, _f).restype = C.c_int


class TrellisError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {strerror(status)} (status {status})")
        self.status = status


def strerror(status: int) -> str:
    return _lib.trellis_strerror(status).decode()


def raw() -> C.CDLL:
    """The loaded library, for callers that marshal their own arguments."""
    return _lib


def _check(fn: str, status: int) -> None:
    if status != OK:
        raise TrellisError(fn, status)


def _dev(t: torch.Tensor | None) -> _vp:
    if t is None:
        return _vp(0)
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("device tensors must be contiguous and on the GPU")
    return _vp(t.data_ptr())


def _stream(stream: torch.cuda.Stream | None) -> _vp:
    s = stream if stream is not None else torch.cuda.current_stream()
    return _vp(s.cuda_stream)


def _geom(g: Shape | Geometry) -> Geometry:
    return g if isinstance(g, Geometry) else Geometry.of(g)


def workspace_bytes(g: Shape | Geometry, M: int, op: int) -> int:
    n = _lib.trellis_workspace_bytes(C.byref(_geom(g)), M, op)
    if n == C.c_size_t(-1).value:
        raise TrellisError("trellis_workspace_bytes", ERR_GEOMETRY)
    return n


def lut_upload(host_lut, dev_lut: torch.Tensor | None = None, device=None,
               stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    import numpy as np

    h = np.ascontiguousarray(host_lut, dtype=np.float32)
    if dev_lut is None:
        dev_lut = torch.empty(h.size, dtype=torch.float32, device=device or "cuda")
    s = stream if stream is not None else torch.cuda.current_stream()
    _check("trellis_lut_upload", _lib.trellis_lut_upload(
        _vp(h.ctypes.data), h.size, _dev(dev_lut), _vp(s.cuda_stream)))
    s.synchronize()  # the copy is stream-ordered and h is this call's own array
    return dev_lut


def gemv(x, codes, scales, lut, g, y=None, stream=None) -> torch.Tensor:
    geom = _geom(g)
    if y is None:
        y = torch.empty(geom.out_features, dtype=torch.bfloat16, device=x.device)
    _check("trellis_gemv", _lib.trellis_gemv(_dev(x), _dev(codes), _dev(scales), _dev(lut),
                                             C.byref(geom), _dev(y), _stream(stream)))
    return y


def gemv_dual(x, a, b, g, y_a=None, y_b=None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Two axis-1 GEMVs over the same x in one launch; a and b are
    (codes, scales, lut) triples of the same geometry g."""
    geom = _geom(g)
    if y_a is None:
        y_a = torch.empty(geom.out_features, dtype=torch.bfloat16, device=x.device)
    if y_b is None:
        y_b = torch.empty(geom.out_features, dtype=torch.bfloat16, device=x.device)
    (ca, sa, la), (cb, sb, lb) = a, b
    _check("trellis_gemv_dual", _lib.trellis_gemv_dual(
        _dev(x), _dev(ca), _dev(sa), _dev(la), _dev(y_a), _dev(cb), _dev(sb), _dev(lb),
        _dev(y_b), C.byref(geom), _stream(stream)))
    return y_a, y_b


def gemv_scatter(x, codes, scales, lut, g, workspace=None, y=None, stream=None) -> torch.Tensor:
    geom = _geom(g)
    if y is None:
        y = torch.empty(geom.out_features, dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(workspace_bytes(geom, 1, OP_GEMV_SCATTER) // 4,
                                dtype=torch.float32, device=x.device)
    _check("trellis_gemv_scatter", _lib.trellis_gemv_scatter(
        _dev(x), _dev(codes), _dev(scales), _dev(lut), C.byref(geom), _dev(workspace),
        workspace.numel() * workspace.element_size(), _dev(y), _stream(stream)))
    return y


def gemv_scatter_static(x, codes, scales, lut, g, y=None, stream=None) -> torch.Tensor:
    """trellis_gemv_scatter with its partials in the library's static device
    array (no workspace); calls overlapping on one device race."""
    geom = _geom(g)
    if y is None:
        y = torch.empty(geom.out_features, dtype=torch.bfloat16, device=x.device)
    _check("trellis_gemv_scatter_static", _lib.trellis_gemv_scatter_static(
        _dev(x), _dev(codes), _dev(scales), _dev(lut), C.byref(geom), _dev(y), _stream(stream)))
    return y


def static_scratch_bytes() -> int:
    return int(_lib.trellis_static_scratch_bytes())


def prefill(x, codes, scales, lut, g, workspace=None, y=None, stream=None,
            balanced=True) -> torch.Tensor:
    """Without a workspace one of workspace_bytes is allocated. At axis 1 the
    workspace is optional: balanced=False passes none (the plan whose last
    16-row group of each workgroup may be partly empty)."""
    geom = _geom(g)
    M = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = torch.empty((M, geom.out_features), dtype=torch.bfloat16, device=x.device)
    if geom.axis == 1 and not balanced:
        workspace, nbytes = None, 0
    else:
        nbytes = workspace_bytes(geom, M, OP_PREFILL)
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes // 4, dtype=torch.float32, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("trellis_prefill", _lib.trellis_prefill(
        _dev(x), M, _dev(codes), _dev(scales), _dev(lut), C.byref(geom), _dev(workspace),
        ws_bytes, _dev(y), _stream(stream)))
    return y


def prefill_dual(x, a, b, g, y_a=None, y_b=None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Two axis-1 prefills over the same x [M][in]; a and b are (codes,
    scales, lut) triples of the same geometry g."""
    geom = _geom(g)
    M = x.shape[0] if x.dim() == 2 else 1
    if y_a is None:
        y_a = torch.empty((M, geom.out_features), dtype=torch.bfloat16, device=x.device)
    if y_b is None:
        y_b = torch.empty((M, geom.out_features), dtype=torch.bfloat16, device=x.device)
    (ca, sa, la), (cb, sb, lb) = a, b
    _check("trellis_prefill_dual", _lib.trellis_prefill_dual(
        _dev(x), M, _dev(ca), _dev(sa), _dev(la), _dev(y_a), _dev(cb), _dev(sb), _dev(lb),
        _dev(y_b), C.byref(geom), _stream(stream)))
    return y_a, y_b


def gate_up_swiglu(x, gate, up, g, h=None, stream=None) -> torch.Tensor:
    """h = bf16(silu(x Wg^T) * (x Wu^T)) for x [M][in] (or [in] for M = 1);
    gate and up are (codes, scales, lut) triples of the same axis-1 geometry
    g. Returns h, [M][out] (or [out] for a 1-D x)."""
    geom = _geom(g)
    M = x.shape[0] if x.dim() == 2 else 1
    if h is None:
        shape = (M, geom.out_features) if x.dim() == 2 else (geom.out_features,)
        h = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    (cg, sg, lg), (cu, su, lu) = gate, up
    _check("trellis_gate_up_swiglu", _lib.trellis_gate_up_swiglu(
        _dev(x), M, _dev(cg), _dev(sg), _dev(lg), _dev(cu), _dev(su), _dev(lu), C.byref(geom),
        _dev(h), _stream(stream)))
    return h


def expand(codes, scales, lut, g, w=None, stream=None) -> torch.Tensor:
    geom = _geom(g)
    rows = geom.out_features if geom.axis == 1 else geom.in_features
    cols = geom.in_features if geom.axis == 1 else geom.out_features
    if w is None:
        w = torch.empty((rows, cols), dtype=torch.bfloat16, device=codes.device)
    _check("trellis_expand", _lib.trellis_expand(_dev(codes), _dev(scales), _dev(lut),
                                                 C.byref(geom), _dev(w), _stream(stream)))
    return w


def repack(codes, g, to_block_interleave: int, out=None, stream=None) -> torch.Tensor:
    """Rewrite `codes` (in the layout g's block_interleave names) into layout
    `to_block_interleave` (0 row-major, 2 block pairs); returns `out`."""
    geom = _geom(g)
    if out is None:
        out = torch.empty_like(codes)
    _check("trellis_repack", _lib.trellis_repack(_dev(codes), _dev(out), C.byref(geom),
                                                 to_block_interleave, _stream(stream)))
    return out


def gather_probe(kind: int, rounds: int, out: torch.Tensor, stream=None) -> int:
    """Enqueue one launch of the LDS codebook-gather probe (trellis_probe.h);
    returns the number of decoded-weight values its timed loop reads."""
    status = _lib.trellis_gather_probe(kind, rounds, _dev(out), out.numel(), _stream(stream))
    if status != OK:
        raise RuntimeError(f"trellis_gather_probe: status {status}")
    return int(_lib.trellis_gather_probe_values(kind, rounds))


def gather_probe_out_floats() -> int:
    return int(_lib.trellis_gather_probe_out_floats())


# ---- grouped operations (trellis_grouped.h) ---------------------------------
#
# Every tensor is checked here (type, shape, contiguity, device): the C ABI sees
# only addresses. Outputs and workspaces that a call allocates belong to the
# stream it runs on.


class Route(NamedTuple):
    """Slots sorted by group (trellis_route), int32 on the GPU."""

    offsets: torch.Tensor   # [groups + 1] first place of each group
    order: torch.Tensor     # [tokens * top_k] slot at each place, -1 behind the last
    position: torch.Tensor  # [tokens, top_k] place of each slot, -1 if dropped


_INT32_MAX = 2 ** 31 - 1


def _want(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple, device: int) -> None:
    """Refuse a tensor that is not dense, of this type and shape, and on `device`."""
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != device):
        if t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name}: device tensors must be contiguous and on the GPU")
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{device}")


def _dims(name: str, t: torch.Tensor, n: int) -> torch.Size:
    if t.dim() != n:
        raise ValueError(f"{name}: expected {n} dimensions, got shape {tuple(t.shape)}")
    if max(t.shape) > _INT32_MAX:  # the C ABI's sizes would wrap around
        raise ValueError(f"{name}: a dimension of {tuple(t.shape)} is larger than {_INT32_MAX}")
    return t.shape


def _device(t: torch.Tensor) -> int:
    """The current device, which every tensor of a call has to be on."""
    return torch.cuda.current_device() if t.is_cuda else -2


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _apart(outputs: dict, inputs: dict) -> None:
    """Refuse an output that shares memory with an input or another output (new
    outputs, given as None, do not)."""
    outs = [(name, t.data_ptr(), t.nbytes) for name, t in outputs.items() if t is not None]
    ins = [(name, t.data_ptr(), t.nbytes) for name, t in inputs.items() if t is not None]
    for i, (a, a0, an) in enumerate(outs):
        for b, b0, bn in outs[i + 1:] + ins:
            if a0 < b0 + bn and b0 < a0 + an and an and bn:
                raise ValueError(f"{a} overlaps {b}")


_NO_STREAM = contextlib.nullcontext()


def _on(stream: torch.cuda.Stream | None, device: int):
    if stream is None:
        return _NO_STREAM
    if stream.device.index != device:
        raise ValueError(f"stream: of {stream.device}, but the current device is cuda:{device}")
    return torch.cuda.stream(stream)


def _handle(device: int) -> int:
    """The current stream's handle (torch.cuda.current_stream().cuda_stream, which
    builds a Stream object first: 2.8 against 0.1 us a call)."""
    return torch._C._cuda_getCurrentRawStream(device)


def _workspace(fn: str, nbytes: int, given: torch.Tensor | None, like: torch.Tensor) -> tuple:
    """(address, bytes, tensor) of the caller's workspace or of a new one."""
    if nbytes == C.c_size_t(-1).value:
        raise TrellisError(fn, ERR_GEOMETRY)
    if given is not None:
        if not given.is_contiguous() or given.get_device() != like.get_device():
            raise ValueError("workspace: expected a contiguous tensor on the device of the others")
        return given.data_ptr(), given.nbytes, given
    if not nbytes:
        return None, 0, None
    ws = like.new_empty(nbytes, dtype=torch.uint8)
    return ws.data_ptr(), nbytes, ws


def route(ids, groups: int, workspace=None, stream=None) -> Route:
    """Sort the slots of ids (int32 [tokens, top_k]) by group, equal ids in slot
    order; ids outside [0, groups) are dropped."""
    tokens, top_k = _dims("ids", ids, 2)
    dev = _device(ids)
    _want("ids", ids, torch.int32, (tokens, top_k), dev)
    fn = "trellis_route"
    if not 0 < groups <= _INT32_MAX:
        raise TrellisError(fn, ERR_GEOMETRY)
    nbytes = _lib.trellis_route_workspace_bytes(tokens, top_k, groups)
    with _on(stream, dev):
        ws, ws_bytes, keep = _workspace(fn, nbytes, workspace, ids)
        if workspace is not None:
            _apart({"workspace": workspace}, {"ids": ids})
        r = Route(ids.new_empty(groups + 1), ids.new_empty(tokens * top_k), torch.empty_like(ids))
        _check(fn, _lib.trellis_route(ids.data_ptr(), tokens, top_k, groups, r.offsets.data_ptr(),
                                      r.order.data_ptr(), r.position.data_ptr(), ws, ws_bytes,
                                      _handle(dev)))
    return r


def dispatch(x, route: Route, out=None, stream=None) -> torch.Tensor:
    """Rows of x [tokens, width] at the places of their slots ([tokens * top_k,
    width]); rows of `out` behind the last placed slot are left as they were.
    Its gradient is combine(dout, None, route)."""
    tokens, width = _dims("x", x, 2)
    top_k = _dims("position", route.position, 2)[1]
    dev = _device(x)
    _want("x", x, torch.bfloat16, (tokens, width), dev)
    _want("position", route.position, torch.int32, (tokens, top_k), dev)
    with _on(stream, dev):
        if out is None:
            out = x.new_empty((tokens * top_k, width))
        else:
            _want("out", out, torch.bfloat16, (tokens * top_k, width), dev)
            _apart({"out": out}, {"x": x, "position": route.position})
        _check("trellis_dispatch", _lib.trellis_dispatch(
            x.data_ptr(), route.position.data_ptr(), tokens, top_k, width, out.data_ptr(),
            _handle(dev)))
    return out


def combine(y, weights, route: Route, out=None, stream=None) -> torch.Tensor:
    """Every token's weighted sum of its slots' rows of y [tokens * top_k, width];
    weights: float32 [tokens, top_k], or None for the plain sum."""
    tokens, top_k = _dims("position", route.position, 2)
    width = _dims("y", y, 2)[1]
    dev = _device(y)
    _want("y", y, torch.bfloat16, (tokens * top_k, width), dev)
    _want("position", route.position, torch.int32, (tokens, top_k), dev)
    if weights is not None:
        _want("weights", weights, torch.float32, (tokens, top_k), dev)
    with _on(stream, dev):
        if out is None:
            out = y.new_empty((tokens, width))
        else:
            _want("out", out, torch.bfloat16, (tokens, width), dev)
            _apart({"out": out}, {"y": y, "weights": weights, "position": route.position})
        _check("trellis_combine", _lib.trellis_combine(
            y.data_ptr(), _ptr(weights), route.position.data_ptr(), tokens, top_k, width,
            out.data_ptr(), _handle(dev)))
    return out


def combine_backward(dout, y, weights, route: Route, dy=None, dweights=None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradients (dy, dweights) of combine(y, weights, route) from dout [tokens,
    width]; rows of `dy` behind the last placed slot are left as they were."""
    tokens, top_k = _dims("position", route.position, 2)
    width = _dims("y", y, 2)[1]
    dev = _device(y)
    _want("dout", dout, torch.bfloat16, (tokens, width), dev)
    _want("y", y, torch.bfloat16, (tokens * top_k, width), dev)
    _want("weights", weights, torch.float32, (tokens, top_k), dev)
    _want("position", route.position, torch.int32, (tokens, top_k), dev)
    with _on(stream, dev):
        given = {"dy": dy, "dweights": dweights}
        if dy is None:
            dy = torch.empty_like(y)
        if dweights is None:
            dweights = torch.empty_like(weights)
        _want("dy", dy, torch.bfloat16, (tokens * top_k, width), dev)
        _want("dweights", dweights, torch.float32, (tokens, top_k), dev)
        _apart(given, {"dout": dout, "y": y, "weights": weights, "position": route.position})
        _check("trellis_combine_backward", _lib.trellis_combine_backward(
            dout.data_ptr(), y.data_ptr(), weights.data_ptr(), route.position.data_ptr(), tokens,
            top_k, width, dy.data_ptr(), dweights.data_ptr(), _handle(dev)))
    return dy, dweights


def experts(x, offsets, codes, scales, lut, g, y=None, workspace=None, stream=None) -> torch.Tensor:
    """y [rows, out]: every row of x [rows, in] times the weights of its expert,
    rows [offsets[e], offsets[e + 1]) being expert e's (Route.offsets). codes:
    int32 [experts, ...], each expert's as for prefill with geometry g; scales:
    float32 [experts, stored rows]; lut: float32 [4096], shared. Rows of `y`
    outside every expert are left as they were. The gradient with respect to x
    is the same call with the geometry's axis flipped and in/out exchanged."""
    geom = _geom(g)
    rows = _dims("x", x, 2)[0]
    n = _dims("offsets", offsets, 1)[0] - 1
    stored, cols = ((geom.out_features, geom.in_features) if geom.axis == 1
                    else (geom.in_features, geom.out_features))
    dev = _device(x)
    _want("x", x, torch.bfloat16, (rows, geom.in_features), dev)
    _want("offsets", offsets, torch.int32, (n + 1,), dev)
    _want("scales", scales, torch.float32, (n, stored), dev)
    _want("lut", lut, torch.float32, (1 << 12,), dev)
    _want("codes", codes, torch.int32, codes.shape, dev)
    if codes.dim() < 1 or codes.shape[0] != n or codes.numel() != n * stored * cols * geom.k // 32:
        raise ValueError(f"codes: expected {n} experts of {stored} x {cols} weights of {geom.k} "
                         f"bits, got {tuple(codes.shape)}")
    fn = "trellis_experts"
    nbytes = _lib.trellis_experts_workspace_bytes(C.byref(geom), rows, n)
    with _on(stream, dev):
        given = {"y": y, "workspace": workspace}
        if y is None:
            y = x.new_empty((rows, geom.out_features))
        _want("y", y, torch.bfloat16, (rows, geom.out_features), dev)
        ws, ws_bytes, keep = _workspace(fn, nbytes, workspace, x)
        _apart(given, {"x": x, "offsets": offsets, "codes": codes, "scales": scales, "lut": lut})
        _check(fn, _lib.trellis_experts(
            x.data_ptr(), rows, offsets.data_ptr(), n, codes.data_ptr(), scales.data_ptr(),
            lut.data_ptr(), C.byref(geom), y.data_ptr(), ws, ws_bytes, _handle(dev)))
    return y


def _adapter_set(a, b, scales, device: int) -> AdapterSet:
    count, rank, i = _dims("a", a, 3)
    o = _dims("b", b, 3)[2]
    _want("a", a, torch.bfloat16, (count, rank, i), device)
    _want("b", b, torch.bfloat16, (count, rank, o), device)
    _want("scales", scales, torch.float32, (count,), device)
    return AdapterSet(a.data_ptr(), b.data_ptr(), scales.data_ptr(), count, rank, i, o)


def adapters_workspace_bytes(f: AdapterSet, rows: int, backward: bool) -> int:
    n = _lib.trellis_adapters_workspace_bytes(C.byref(f), rows, int(backward))
    if n == C.c_size_t(-1).value:
        raise TrellisError("trellis_adapters_workspace_bytes", ERR_GEOMETRY)
    return n


def adapters(x, ids, a, b, scales, base=None, y=None, u=None, keep_inner=False, workspace=None,
             stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(y, u): y = base + scales[i] * b[i]^T (a[i] x) for every row with i = ids[m]
    in [0, count), and base for the others. x: bf16 [rows, in]; a: bf16 [count,
    rank, in]; b: bf16 [count, rank, out]; base: bf16 [rows, out] (None: zeros),
    which y may be. u: float32 [rows, rank] of inner products, None unless given
    or keep_inner (the backward pass needs it)."""
    dev = _device(x)
    f = _adapter_set(a, b, scales, dev)
    rows = _dims("x", x, 2)[0]
    _want("x", x, torch.bfloat16, (rows, f.in_features), dev)
    _want("ids", ids, torch.int32, (rows,), dev)
    if base is not None:
        _want("base", base, torch.bfloat16, (rows, f.out_features), dev)
    nbytes = adapters_workspace_bytes(f, rows, False)
    with _on(stream, dev):
        given = None
        if y is not None or u is not None or workspace is not None:
            given = {"y": y, "u": u, "workspace": workspace}
        if y is None:
            y = x.new_empty((rows, f.out_features))
        else:
            _want("y", y, torch.bfloat16, (rows, f.out_features), dev)
        if u is not None:
            _want("u", u, torch.float32, (rows, f.rank), dev)
        elif keep_inner:
            u = x.new_empty((rows, f.rank), dtype=torch.float32)
        ws, ws_bytes, keep = _workspace("trellis_adapters", nbytes, workspace, x)
        if given is not None:
            same = base is not None and base.data_ptr() == y.data_ptr()
            _apart(given, {"x": x, "ids": ids, "a": a, "b": b, "scales": scales,
                           "base": None if same else base})
        _check("trellis_adapters", _lib.trellis_adapters(
            x.data_ptr(), ids.data_ptr(), rows, C.byref(f), _ptr(base), y.data_ptr(), _ptr(u), ws,
            ws_bytes, _handle(dev)))
    return y, u


def adapters_backward(dy, x, u, ids, a, b, scales, base=None, dx=None, da=None, db=None,
                      workspace=None, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients (dx, da, db) of adapters from dy [rows, out] with the forward
    pass's u: dx = base + a[i]^T g with g = scales[i] * b[i] dy, da and db whole
    (zeros for adapters without rows), all bf16. dx may be `base`. x: the forward
    pass's, as bf16 rows or as `keep` put them away."""
    dev = _device(dy)
    f = _adapter_set(a, b, scales, dev)
    rows = _dims("dy", dy, 2)[0]
    _want("dy", dy, torch.bfloat16, (rows, f.out_features), dev)
    kept = isinstance(x, Kept)
    if kept:
        _want_kept("x", x, rows, f.in_features, dev)
    else:
        _want("x", x, torch.bfloat16, (rows, f.in_features), dev)
    _want("u", u, torch.float32, (rows, f.rank), dev)
    _want("ids", ids, torch.int32, (rows,), dev)
    if base is not None:
        _want("base", base, torch.bfloat16, (rows, f.in_features), dev)
    nbytes = adapters_workspace_bytes(f, rows, True)
    with _on(stream, dev):
        given = {"dx": dx, "da": da, "db": db, "workspace": workspace}
        if dx is None:
            dx = dy.new_empty((rows, f.in_features))
        if da is None:
            da = torch.empty_like(a)
        if db is None:
            db = torch.empty_like(b)
        _want("dx", dx, torch.bfloat16, (rows, f.in_features), dev)
        _want("da", da, torch.bfloat16, a.shape, dev)
        _want("db", db, torch.bfloat16, b.shape, dev)
        ws, ws_bytes, hold = _workspace("trellis_adapters_backward", nbytes, workspace, dy)
        same = base is not None and base.data_ptr() == dx.data_ptr()
        rows_of_x = _kept_parts("x", x) if kept else {"x": x}
        _apart(given, {"dy": dy, **rows_of_x, "u": u, "ids": ids, "a": a, "b": b, "scales": scales,
                       "base": None if same else base})
        fn, where = "trellis_adapters_backward", None
        if kept:
            fn, where = "trellis_adapters_backward_kept", C.byref(_kept_rows(x))
        _check(fn, getattr(_lib, fn)(
            dy.data_ptr(), where if kept else x.data_ptr(), u.data_ptr(), ids.data_ptr(), rows,
            C.byref(f), _ptr(base), dx.data_ptr(), da.data_ptr(), db.data_ptr(), ws, ws_bytes,
            _handle(dev)))
    return dx, da, db


# ---- around an MLP or a layer of experts (trellis_mlp.h) ----------------------


class Kept(NamedTuple):
    """bf16 rows held in 8 bits (trellis_keep)."""

    codes: torch.Tensor      # int8 [rows, width]
    exponents: torch.Tensor  # uint8 [rows, ceil(width / 32)], one per 32 values


def _kept_rows(k: Kept) -> _KeptRows:
    return _KeptRows(k.codes.data_ptr(), k.exponents.data_ptr())


def _kept_parts(name: str, k: Kept) -> dict:
    return {f"{name}.codes": k.codes, f"{name}.exponents": k.exponents}


def _want_kept(name: str, k: Kept, rows: int, width: int, device: int) -> None:
    _want(f"{name}.codes", k.codes, torch.int8, (rows, width), device)
    _want(f"{name}.exponents", k.exponents, torch.uint8, (rows, -(-width // 32)), device)


def _new_kept(like: torch.Tensor, rows: int, width: int) -> Kept:
    return Kept(like.new_empty((rows, width), dtype=torch.int8),
                like.new_empty((rows, -(-width // 32)), dtype=torch.uint8))


def keep(x, kept: Kept | None = None, stream=None) -> Kept:
    """bf16 rows x [rows, width] put away in 8 bits: 32 adjacent values of a row share
    an exponent, and each is off by at most 1/128 of the group's largest magnitude."""
    rows, width = _dims("x", x, 2)
    dev = _device(x)
    _want("x", x, torch.bfloat16, (rows, width), dev)
    with _on(stream, dev):
        if kept is None:
            kept = _new_kept(x, rows, width)
        else:
            _want_kept("kept", kept, rows, width, dev)
            _apart(_kept_parts("kept", kept), {"x": x})
        _check("trellis_keep", _lib.trellis_keep(x.data_ptr(), rows, width, C.byref(_kept_rows(kept)),
                                                 _handle(dev)))
    return kept


def restore(kept: Kept, out=None, stream=None) -> torch.Tensor:
    """The bf16 rows that `kept` stands for."""
    rows, width = _dims("kept.codes", kept.codes, 2)
    dev = _device(kept.codes)
    _want_kept("kept", kept, rows, width, dev)
    with _on(stream, dev):
        if out is None:
            out = kept.codes.new_empty((rows, width), dtype=torch.bfloat16)
        else:
            _want("out", out, torch.bfloat16, (rows, width), dev)
            _apart({"out": out}, _kept_parts("kept", kept))
        _check("trellis_restore", _lib.trellis_restore(C.byref(_kept_rows(kept)), rows, width,
                                                       out.data_ptr(), _handle(dev)))
    return out


def swiglu(gu, h=None, keep=False, kept: Kept | None = None,
           stream=None) -> tuple[torch.Tensor, Kept | None]:
    """(h, kept): h = silu(g) * u for gu [rows, 2 * inter], a row being [g, u]. kept: gu
    in 8 bits for swiglu_backward (rows g and u apart: [2 * rows, inter]), None unless
    given or `keep`."""
    rows, width = _dims("gu", gu, 2)
    if width % 2:
        raise ValueError(f"gu: expected rows [g, u] of even length, got shape {tuple(gu.shape)}")
    inter = width // 2
    dev = _device(gu)
    _want("gu", gu, torch.bfloat16, (rows, width), dev)
    with _on(stream, dev):
        if h is not None:
            _want("h", h, torch.bfloat16, (rows, inter), dev)
        if kept is not None:
            _want_kept("kept", kept, 2 * rows, inter, dev)
        if h is not None or kept is not None:
            parts = _kept_parts("kept", kept) if kept is not None else {}
            _apart({"h": h, **parts}, {"gu": gu})
        if h is None:
            h = gu.new_empty((rows, inter))
        if kept is None and keep:
            kept = _new_kept(gu, 2 * rows, inter)
        _check("trellis_swiglu", _lib.trellis_swiglu(
            gu.data_ptr(), rows, inter, h.data_ptr(),
            None if kept is None else C.byref(_kept_rows(kept)), _handle(dev)))
    return h, kept


def swiglu_backward(dh, gu, dgu=None, h=None, again=False,
                    stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(dgu, h): the gradient of swiglu from dh [rows, inter], and h once more, None
    unless given or `again`. gu: bf16 [rows, 2 * inter], or as swiglu kept it."""
    rows, inter = _dims("dh", dh, 2)
    dev = _device(dh)
    _want("dh", dh, torch.bfloat16, (rows, inter), dev)
    kept = isinstance(gu, Kept)
    if kept:
        _want_kept("gu", gu, 2 * rows, inter, dev)
    else:
        _want("gu", gu, torch.bfloat16, (rows, 2 * inter), dev)
    with _on(stream, dev):
        if dgu is not None:
            _want("dgu", dgu, torch.bfloat16, (rows, 2 * inter), dev)
        if h is not None:
            _want("h", h, torch.bfloat16, (rows, inter), dev)
        if dgu is not None or h is not None:
            _apart({"dgu": dgu, "h": h},
                   {"dh": dh, **(_kept_parts("gu", gu) if kept else {"gu": gu})})
        if dgu is None:
            dgu = dh.new_empty((rows, 2 * inter))
        if h is None and again:
            h = torch.empty_like(dh)
        _check("trellis_swiglu_backward", _lib.trellis_swiglu_backward(
            dh.data_ptr(), None if kept else gu.data_ptr(),
            C.byref(_kept_rows(gu)) if kept else None, rows, inter, dgu.data_ptr(), _ptr(h),
            _handle(dev)))
    return dgu, h


def _expert_set(name: str, w: tuple, geom: Geometry, n: int, device: int) -> ExpertSet:
    codes, scales, lut = w
    stored, cols = ((geom.out_features, geom.in_features) if geom.axis == 1
                    else (geom.in_features, geom.out_features))
    _want(f"{name} scales", scales, torch.float32, (n, stored), device)
    _want(f"{name} lut", lut, torch.float32, (1 << 12,), device)
    _want(f"{name} codes", codes, torch.int32, codes.shape, device)
    if codes.dim() < 1 or codes.shape[0] != n or codes.numel() != n * stored * cols * geom.k // 32:
        raise ValueError(f"{name} codes: expected {n} experts of {stored} x {cols} weights of "
                         f"{geom.k} bits, got {tuple(codes.shape)}")
    return ExpertSet(codes.data_ptr(), scales.data_ptr(), lut.data_ptr(), geom)


def experts_mlp(x, ids, weights, up, down, g_up, g_down, out=None, workspace=None,
                stream=None) -> torch.Tensor:
    """A whole layer of experts for up to 32 tokens: out [tokens, hidden] = the sum over
    the experts e that a token chose of Wd_e (w silu(Wg_e x) * (Wu_e x)), what stands in
    brackets held in 16 bits of mantissa. x: bf16 [tokens, hidden]; ids: int32 [tokens,
    top_k] (others than [0, experts): no choice); weights: float32 [tokens, top_k], or None
    for ones. up and down: (codes, scales, lut) as for experts, with g_up of axis 1, hidden
    -> 2 * inter (the gate's rows, then the up's) and g_down of either axis, inter ->
    hidden. With one expert it is a dense MLP, which gate_up_swiglu and prefill (or a GEMV)
    mostly do in less time."""
    gu, gd = _geom(g_up), _geom(g_down)
    tokens, top_k = _dims("ids", ids, 2)
    dev = _device(x)
    _want("x", x, torch.bfloat16, (tokens, gu.in_features), dev)
    _want("ids", ids, torch.int32, (tokens, top_k), dev)
    if weights is not None:
        _want("weights", weights, torch.float32, (tokens, top_k), dev)
    n = _dims("up scales", up[1], 2)[0]
    su, sd = _expert_set("up", up, gu, n, dev), _expert_set("down", down, gd, n, dev)
    fn = "trellis_experts_mlp"
    nbytes = _lib.trellis_experts_mlp_workspace_bytes(tokens, top_k, n, C.byref(su), C.byref(sd))
    with _on(stream, dev):
        ws, ws_bytes, hold = _workspace(fn, nbytes, workspace, x)
        if out is not None or workspace is not None:
            if out is not None:
                _want("out", out, torch.bfloat16, (tokens, gu.in_features), dev)
            _apart({"out": out, "workspace": workspace},
                   {"x": x, "ids": ids, "weights": weights, "up codes": up[0], "up scales": up[1],
                    "up lut": up[2], "down codes": down[0], "down scales": down[1],
                    "down lut": down[2]})
        if out is None:
            out = torch.empty_like(x)
        _check(fn, _lib.trellis_experts_mlp(
            x.data_ptr(), ids.data_ptr(), _ptr(weights), tokens, top_k, n, C.byref(su), C.byref(sd),
            out.data_ptr(), ws, ws_bytes, _handle(dev)))
    return out
