"""Host-side argument checks of the grouped operations (no GPU): sizes, null and
misaligned pointers and workspaces are refused before anything is enqueued, and
the binding refuses tensors of a wrong type, shape or place."""
import ctypes as C
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below is refused or has no rows


@pytest.fixture(scope="module")
def T():
    if not os.path.exists(os.path.join(ROOT, "dequant_gemm_trellis_amd", "libtrellis.so")):
        import __graft_entry__

        __graft_entry__.build()
    from dequant_gemm_trellis_amd import trellis

    return trellis


def call(T, name, params, defaults, **kw):
    """Call an entry point with the defaults overridden by kw; integers named in
    `params` with a leading '#' are sizes, the rest addresses."""
    a = dict(defaults, **kw)
    args = [a[n[1:]] if n[0] == "#" else C.c_void_p(a[n]) for n in params]
    return getattr(T.raw(), name)(*args, C.c_void_p(0))


ROUTE = ("ids", "#tokens", "#top_k", "#groups", "offsets", "order", "position", "ws", "#ws_bytes")
ROUTE_ARGS = dict(ids=FAKE, tokens=5, top_k=2, groups=4, offsets=FAKE, order=FAKE, position=FAKE,
                  ws=0, ws_bytes=0)


def test_route_validation(T):
    def route(**kw):
        return call(T, "trellis_route", ROUTE, ROUTE_ARGS, **kw)

    for kw in (dict(tokens=-1), dict(top_k=0), dict(groups=0), dict(groups=1025),
               dict(tokens=1 << 20, top_k=3), dict(tokens=2 ** 31 - 1, top_k=2 ** 31 - 1)):
        assert route(**kw) == T.ERR_GEOMETRY, kw
    for arg in ("ids", "offsets", "order", "position"):
        assert route(**{arg: 0}) == T.ERR_NULL, arg
        assert route(**{arg: FAKE + 2}) == T.ERR_ALIGN, arg
    assert route(ws=FAKE + 8) == T.ERR_ALIGN
    need = T.raw().trellis_route_workspace_bytes(100000, 2, 4)
    assert need > 0
    assert route(tokens=100000) == T.ERR_WORKSPACE
    assert route(tokens=100000, ws=FAKE, ws_bytes=need - 1) == T.ERR_WORKSPACE


def test_route_workspace_bytes(T):
    f = T.raw().trellis_route_workspace_bytes
    none = C.c_size_t(-1).value
    assert f(4096, 2, 128) == 0                      # one workgroup sorts these
    assert f(4097, 2, 128) == 5 * 128 * 4            # five chunks of 2048 slots
    assert f(1 << 21, 1, 1024) == 256 * 1024 * 4     # never more than 256 chunks
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 1025), (1 << 20, 3, 1)):
        assert f(*bad) == none, bad


MOVES = {
    "trellis_dispatch": (("x", "position", "#tokens", "#top_k", "#width", "out"), ()),
    "trellis_combine": (("y", "weights", "position", "#tokens", "#top_k", "#width", "out"),
                        ("weights",)),
    "trellis_combine_backward": (("dout", "y", "weights", "position", "#tokens", "#top_k",
                                  "#width", "dy", "dweights"), ()),
}


@pytest.mark.parametrize("name", sorted(MOVES))
def test_moves_validation(T, name):
    order, optional = MOVES[name]
    args = {n.lstrip("#"): FAKE for n in order} | dict(tokens=5, top_k=2, width=64)

    def move(**kw):
        return call(T, name, order, args, **kw)

    for kw in (dict(tokens=-1), dict(top_k=0), dict(width=0), dict(width=(1 << 19) + 1),
               dict(tokens=1 << 20, top_k=3)):
        assert move(**kw) == T.ERR_GEOMETRY, kw
    for arg in order:
        if arg[0] == "#":
            continue
        if arg not in optional:
            assert move(**{arg: 0}) == T.ERR_NULL, arg
        assert move(**{arg: FAKE + 1}) == T.ERR_ALIGN, arg
    assert move(tokens=0) == T.OK  # nothing to do, nothing enqueued
    assert move(tokens=0, **{order[0]: 0}) == T.OK


def test_binding_refuses_host_and_mistyped_tensors(T):
    ids = torch.zeros((3, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        T.route(ids, 4)
    with pytest.raises(ValueError, match="int32"):
        T.route(ids.long(), 4)
    with pytest.raises(ValueError, match="2 dimensions"):
        T.route(ids.reshape(-1), 4)
    r = T.Route(torch.zeros(5, dtype=torch.int32), torch.zeros(6, dtype=torch.int32), ids)
    x = torch.zeros((3, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the GPU"):
        T.dispatch(x, r)
    with pytest.raises(ValueError, match="bfloat16"):
        T.dispatch(x.float(), r)
    with pytest.raises(ValueError):
        T.combine(x, None, r)  # 3 rows where 6 slots are
    with pytest.raises(ValueError):
        T.combine_backward(x, x, torch.zeros((3, 2)), r)


def test_overlap_check(T):
    a = torch.zeros(64, dtype=torch.bfloat16)
    T._apart({"out": a[:32]}, {"x": a[32:], "none": None})
    with pytest.raises(ValueError, match="out overlaps x"):
        T._apart({"out": a[:33]}, {"x": a[32:]})
    with pytest.raises(ValueError, match="dy overlaps dw"):
        T._apart({"dy": a, "dw": a[63:]}, {})
    T._apart({"out": a[:0]}, {"x": a})                # nothing written
    T._apart({"out": a[:8]}, {"x": a[16:], "y": a[16:]})  # inputs may share


ADAPTERS = {
    "trellis_adapters": ("x", "ids", "#rows", "set", "base", "y", "u", "ws", "#ws_bytes"),
    "trellis_adapters_backward": ("dy", "x", "u", "ids", "#rows", "set", "base", "dx", "da", "db",
                                  "ws", "#ws_bytes"),
}


@pytest.mark.parametrize("name", sorted(ADAPTERS))
def test_adapters_validation(T, name):
    order, backward = ADAPTERS[name], name.endswith("backward")
    f = T.AdapterSet(FAKE, FAKE, FAKE, 4, 16, 256, 300)
    need = T.adapters_workspace_bytes(f, 100, backward)
    args = {n.lstrip("#"): FAKE for n in order} | dict(rows=100, ws_bytes=need)

    def apply(f=f, **kw):
        a = dict(args, **kw)
        return getattr(T.raw(), name)(*[
            a[n[1:]] if n[0] == "#" else (C.byref(f) if f is not None else None) if n == "set"
            else C.c_void_p(a[n]) for n in order], C.c_void_p(0))

    def other(**kw):
        g = T.AdapterSet(FAKE, FAKE, FAKE, 4, 16, 256, 300)
        for k, v in kw.items():
            setattr(g, k, v)
        return g

    assert apply(None) == T.ERR_NULL
    for kw in (dict(count=0), dict(count=1025), dict(rank=0), dict(rank=129), dict(in_features=0),
               dict(in_features=(1 << 19) + 1), dict(out_features=0),
               dict(out_features=(1 << 19) + 1)):
        assert apply(other(**kw)) == T.ERR_GEOMETRY, kw
        assert T.raw().trellis_adapters_workspace_bytes(C.byref(other(**kw)), 100, backward) == \
            C.c_size_t(-1).value
    for rows in (-1, (1 << 20) + 1):
        assert apply(rows=rows) == T.ERR_GEOMETRY
    for kw in (dict(a=0), dict(b=0), dict(scales=0)):
        assert apply(other(**kw)) == T.ERR_NULL, kw
    for kw in (dict(a=FAKE + 1), dict(b=FAKE + 1), dict(scales=FAKE + 2)):
        assert apply(other(**kw)) == T.ERR_ALIGN, kw
    for arg in order:
        if arg[0] == "#" or arg in ("set", "ws"):
            continue
        if arg not in ("base",) and not (arg == "u" and not backward):
            assert apply(**{arg: 0}) == T.ERR_NULL, arg
        assert apply(**{arg: FAKE + 1}) == T.ERR_ALIGN, arg
    assert apply(ws=FAKE + 8) == T.ERR_ALIGN
    assert apply(ws=0) == T.ERR_WORKSPACE
    assert apply(ws_bytes=need - 1) == T.ERR_WORKSPACE
    if not backward:
        assert apply(rows=0, x=0, ids=0, y=0) == T.OK  # nothing to do, nothing enqueued


def test_adapters_workspace_stays_small(T):
    """The gradient's float32 sums are kept for adapters of over 1024 rows only:
    many adapters of a wide projection do not multiply the workspace."""
    f = T.AdapterSet(0, 0, 0, 1024, 64, 5120, 17408)
    assert T.adapters_workspace_bytes(f, 1000, True) < 1 << 30
    few = T.AdapterSet(0, 0, 0, 2, 64, 5120, 17408)
    shared = 2 * 4 * 64 * 17408 * 4  # at 4096 rows: at most 8 segments
    assert shared < T.adapters_workspace_bytes(few, 4096, True) < 3 * shared


def test_binding_refuses_mismatched_adapters(T):
    x, ids = torch.zeros((3, 8), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    a, b = torch.zeros((2, 4, 8), dtype=torch.bfloat16), torch.zeros((2, 5, 6), dtype=torch.bfloat16)
    s = torch.ones(2)
    with pytest.raises(ValueError, match="a: device tensors"):
        T.adapters(x, ids, a, b, s)
    with pytest.raises(ValueError, match="a: expected"):
        T.adapters(x, ids, a.float(), b, s)
    with pytest.raises(ValueError, match="3 dimensions"):
        T.adapters(x, ids, a[0], b, s)


EXPERTS = ("x", "#rows", "offsets", "#experts", "codes", "scales", "lut", "geom", "y", "ws",
           "#ws_bytes")


@pytest.mark.parametrize("axis", [0, 1])
def test_experts_validation(T, axis):
    g = T.Geometry(axis, 256, 12, 3, 512, 256, 0)
    need = T.raw().trellis_experts_workspace_bytes(C.byref(g), 100000, 4)
    assert need > 0  # the rows in another order
    assert T.raw().trellis_experts_workspace_bytes(C.byref(g), 4, 4) == 0
    args = dict(x=FAKE, rows=100000, offsets=FAKE, experts=4, codes=FAKE, scales=FAKE, lut=FAKE,
                y=FAKE, ws=FAKE, ws_bytes=need)

    def experts(g=g, **kw):
        a = dict(args, **kw)
        return T.raw().trellis_experts(*[
            a[n[1:]] if n[0] == "#" else (C.byref(g) if g is not None else None) if n == "geom"
            else C.c_void_p(a[n]) for n in EXPERTS], C.c_void_p(0))

    assert experts(None) == T.ERR_NULL
    for bad in (T.Geometry(2, 256, 12, 3, 512, 256, 0), T.Geometry(axis, 256, 12, 5, 512, 256, 0),
                T.Geometry(axis, 256, 12, 3, 0, 256, 0), T.Geometry(axis, 256, 12, 3, 300, 300, 0)):
        assert experts(bad) == T.ERR_GEOMETRY
        assert T.raw().trellis_experts_workspace_bytes(C.byref(bad), 10, 4) == C.c_size_t(-1).value
    for kw in (dict(rows=-1), dict(rows=(1 << 21) + 1), dict(experts=0), dict(experts=1025)):
        assert experts(**kw) == T.ERR_GEOMETRY, kw
    for arg in ("x", "offsets", "codes", "scales", "lut", "y"):
        assert experts(**{arg: 0}) == T.ERR_NULL, arg
        assert experts(**{arg: FAKE + 2}) == T.ERR_ALIGN, arg
    assert experts(ws=FAKE + 8) == T.ERR_ALIGN
    if need:
        assert experts(ws=0) == T.ERR_WORKSPACE
        assert experts(ws_bytes=need - 1) == T.ERR_WORKSPACE
    assert experts(rows=0, x=0, y=0) == T.OK  # nothing to do, nothing enqueued


def test_sizes_past_32_bits_do_not_wrap_around(T):
    """A dimension of 2^32 would arrive at the C ABI as zero."""
    for t in (torch.zeros((1, 1), dtype=torch.int32).expand(2 ** 32, 1),
              torch.zeros((1, 1), dtype=torch.int32).expand(1, 2 ** 32)):
        with pytest.raises(ValueError, match="larger than"):
            T.route(t, 4)
    x = torch.zeros((1, 1), dtype=torch.bfloat16).expand(2 ** 32, 1)
    r = T.Route(torch.zeros(5, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                torch.zeros((1, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="larger than"):
        T.dispatch(x, r)
    with pytest.raises(ValueError, match="larger than"):
        T.combine(x, None, r)
