"""ctypes binding over libtrellis.so (include/trellis.h, trellis_grouped.h).

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
            "trellis_experts_workspace_bytes")
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


_AP = C.POINTER(AdapterSet)
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
for _f in ("trellis_lut_upload", "trellis_gemv", "trellis_gemv_dual", "trellis_gemv_scatter",
           "trellis_prefill", "trellis_prefill_dual", "trellis_gate_up_swiglu", "trellis_expand",
           "trellis_repack", "trellis_gemv_scatter_static", "trellis_route", "trellis_dispatch",
           "trellis_combine", "trellis_combine_backward", "trellis_adapters",
           "trellis_adapters_backward", "trellis_experts"):
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
    (zeros for adapters without rows), all bf16. dx may be `base`."""
    dev = _device(x)
    f = _adapter_set(a, b, scales, dev)
    rows = _dims("x", x, 2)[0]
    _want("dy", dy, torch.bfloat16, (rows, f.out_features), dev)
    _want("x", x, torch.bfloat16, (rows, f.in_features), dev)
    _want("u", u, torch.float32, (rows, f.rank), dev)
    _want("ids", ids, torch.int32, (rows,), dev)
    if base is not None:
        _want("base", base, torch.bfloat16, (rows, f.in_features), dev)
    nbytes = adapters_workspace_bytes(f, rows, True)
    with _on(stream, dev):
        given = {"dx": dx, "da": da, "db": db, "workspace": workspace}
        if dx is None:
            dx = torch.empty_like(x)
        if da is None:
            da = torch.empty_like(a)
        if db is None:
            db = torch.empty_like(b)
        _want("dx", dx, torch.bfloat16, (rows, f.in_features), dev)
        _want("da", da, torch.bfloat16, a.shape, dev)
        _want("db", db, torch.bfloat16, b.shape, dev)
        ws, ws_bytes, keep = _workspace("trellis_adapters_backward", nbytes, workspace, x)
        same = base is not None and base.data_ptr() == dx.data_ptr()
        _apart(given, {"dy": dy, "x": x, "u": u, "ids": ids, "a": a, "b": b, "scales": scales,
                       "base": None if same else base})
        _check("trellis_adapters_backward", _lib.trellis_adapters_backward(
            dy.data_ptr(), x.data_ptr(), u.data_ptr(), ids.data_ptr(), rows, C.byref(f), _ptr(base),
            dx.data_ptr(), da.data_ptr(), db.data_ptr(), ws, ws_bytes, _handle(dev)))
    return dx, da, db
