"""Host-side argument checks of the operations around an MLP or a layer of experts
(no GPU): the C ABI refuses sizes, null and misaligned pointers and workspaces before
anything is enqueued, and the binding refuses tensors of a wrong type, shape or place."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

import kept_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below is refused or has no rows
NONE = C.c_size_t(-1).value


@pytest.fixture(scope="module")
def T():
    if not os.path.exists(os.path.join(ROOT, "dequant_gemm_trellis_amd", "libtrellis.so")):
        import __graft_entry__

        __graft_entry__.build()
    from dequant_gemm_trellis_amd import trellis

    return trellis


def expert_set(T, axis, i, o, k=3, codes=FAKE, scales=FAKE, lut=FAKE, T_=256):
    return T.ExpertSet(codes, scales, lut, T.Geometry(axis, T_, 12, k, i, o, 0))


def layer(T, up=None, down=None, **kw):
    up = expert_set(T, 1, 512, 600) if up is None else up
    down = expert_set(T, 0, 300, 512) if down is None else down
    a = dict(x=FAKE, ids=FAKE, weights=FAKE, tokens=5, top_k=2, experts=8, out=FAKE, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    by = [C.byref(s) if s is not False else None for s in (up, down)]
    need = T.raw().trellis_experts_mlp_workspace_bytes(a["tokens"], a["top_k"], a["experts"], *by)
    status = T.raw().trellis_experts_mlp(
        C.c_void_p(a["x"]), C.c_void_p(a["ids"]), C.c_void_p(a["weights"]), a["tokens"], a["top_k"],
        a["experts"], *by, C.c_void_p(a["out"]), C.c_void_p(a["ws"]), a["ws_bytes"], C.c_void_p(0))
    return status, need


def test_layer_validation(T):
    for kw in (dict(tokens=-1), dict(tokens=33), dict(top_k=0), dict(top_k=33), dict(experts=0),
               dict(experts=1025)):
        assert layer(T, **kw) == (T.ERR_GEOMETRY, NONE), kw
    wrong = [
        (expert_set(T, 0, 512, 768), None),                              # gate and up on axis 0
        (expert_set(T, 1, 512, 601), None),                              # an odd number of rows
        (expert_set(T, 1, 512, 598), None),                              # 299 where down has 300
        (None, expert_set(T, 0, 300, 256)),                              # another hidden width
        (None, expert_set(T, 1, 300, 512)),                              # inter in blocks of 256 only
        (expert_set(T, 1, 500, 600), None), (expert_set(T, 1, 512, 600, k=5), None),
        (None, expert_set(T, 0, 300, 512, T_=128)),
    ]
    for up, down in wrong:
        assert layer(T, up, down) == (T.ERR_GEOMETRY, NONE)
    assert layer(T, False) == (T.ERR_NULL, NONE) and layer(T, None, False) == (T.ERR_NULL, NONE)
    for arg in ("x", "ids", "out"):
        assert layer(T, **{arg: 0})[0] == T.ERR_NULL, arg
    for arg in ("x", "ids", "out", "weights"):
        assert layer(T, **{arg: FAKE + 2})[0] == T.ERR_ALIGN, arg
    for kw, status in ((dict(codes=0), T.ERR_NULL), (dict(scales=0), T.ERR_NULL), (dict(lut=0), T.ERR_NULL),
                       (dict(codes=FAKE + 4), T.ERR_ALIGN), (dict(lut=FAKE + 8), T.ERR_ALIGN),
                       (dict(scales=FAKE + 2), T.ERR_ALIGN)):
        assert layer(T, expert_set(T, 1, 512, 600, **kw))[0] == status, kw
        assert layer(T, None, expert_set(T, 0, 300, 512, **kw))[0] == status, kw
    need = layer(T, ws=0)[1]
    assert 0 < need < 1 << 30
    assert layer(T, ws=0)[0] == T.ERR_WORKSPACE
    assert layer(T, ws_bytes=need - 1)[0] == T.ERR_WORKSPACE
    assert layer(T, ws=FAKE + 8)[0] == T.ERR_ALIGN
    # nothing to do, nothing enqueued
    assert layer(T, tokens=0, x=0, ids=0, out=0, ws=0, ws_bytes=0) == (T.OK, 0)


MOVES = {
    "trellis_keep": ("x", "#rows", "#width", "kept"),
    "trellis_restore": ("kept", "#rows", "#width", "out"),
    "trellis_swiglu": ("gu", "#rows", "#width", "h", "kept"),
    "trellis_swiglu_backward": ("dh", "gu", "kept", "#rows", "#width", "dgu", "h"),
}
OPTIONAL = {("trellis_swiglu", "kept"), ("trellis_swiglu_backward", "h")}


@pytest.mark.parametrize("name", sorted(MOVES))
def test_rows_validation(T, name):
    order = MOVES[name]
    args = {n.lstrip("#"): FAKE for n in order} | dict(rows=5, width=64, kept=(FAKE, FAKE))
    if name == "trellis_swiglu_backward":
        args["gu"] = 0

    def move(**kw):
        a = dict(args, **kw)
        values = []
        for n in order:
            if n[0] == "#":
                values.append(a[n[1:]])
            elif n == "kept":
                values.append(None if a[n] is None else C.byref(T._KeptRows(*a[n])))
            else:
                values.append(C.c_void_p(a[n]))
        return getattr(T.raw(), name)(*values, C.c_void_p(0))

    most = 1 << 18 if "swiglu" in name else 1 << 19
    rows = 1 << 21 if "swiglu" in name else 1 << 22
    for kw in (dict(rows=-1), dict(width=0), dict(width=-5), dict(width=most + 1), dict(rows=rows + 1),
               dict(rows=rows, width=16384)):  # more than 2^34 values
        assert move(**kw) == T.ERR_GEOMETRY, kw
    for n in order:
        if n[0] == "#":
            continue
        if n == "kept":
            if (name, n) not in OPTIONAL:
                assert move(kept=None) == T.ERR_NULL
            for kept in ((0, FAKE), (FAKE, 0)):
                assert move(kept=kept) == T.ERR_NULL
            continue
        if (name, n) not in OPTIONAL and n != "gu" or name == "trellis_swiglu" and n == "gu":
            assert move(**{n: 0}) == T.ERR_NULL, n
        assert move(**{n: FAKE + 1}) in (T.ERR_ALIGN, T.ERR_GEOMETRY), n
    if name == "trellis_swiglu_backward":
        assert move(gu=FAKE) == T.ERR_GEOMETRY  # both forms of gu
        assert move(gu=FAKE + 1, kept=None) == T.ERR_ALIGN
        assert move(gu=0, kept=None) == T.ERR_NULL
    assert move(**({n.lstrip("#"): 0 for n in order if n != "kept"} | dict(width=64))) == T.OK  # no rows


def test_adapters_backward_kept_validation(T):
    order = ("dy", "x", "u", "ids", "#rows", "set", "base", "dx", "da", "db", "ws", "#ws_bytes")
    f = T.AdapterSet(FAKE, FAKE, FAKE, 4, 16, 256, 300)
    need = T.adapters_workspace_bytes(f, 100, True)
    args = {n.lstrip("#"): FAKE for n in order} | dict(rows=100, ws_bytes=need, x=(FAKE, FAKE), set=f)

    def apply(**kw):
        a = dict(args, **kw)
        values = []
        for n in order:
            if n[0] == "#":
                values.append(a[n[1:]])
            elif n == "set":
                values.append(C.byref(a[n]))
            elif n == "x":
                values.append(None if a[n] is None else C.byref(T._KeptRows(*a[n])))
            else:
                values.append(C.c_void_p(a[n]))
        return T.raw().trellis_adapters_backward_kept(*values, C.c_void_p(0))

    for x in (None, (0, FAKE), (FAKE, 0)):
        assert apply(x=x) == T.ERR_NULL, x
    for n in ("dy", "u", "ids", "dx", "da", "db"):
        assert apply(**{n: 0}) == T.ERR_NULL, n
        assert apply(**{n: FAKE + 1}) == T.ERR_ALIGN, n
    assert apply(base=FAKE + 1) == T.ERR_ALIGN
    assert apply(rows=-1) == T.ERR_GEOMETRY and apply(rows=(1 << 20) + 1) == T.ERR_GEOMETRY
    assert apply(ws=0) == T.ERR_WORKSPACE and apply(ws_bytes=need - 1) == T.ERR_WORKSPACE
    assert apply(ws=FAKE + 8) == T.ERR_ALIGN


def test_binding_refuses(T):
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    kept = T.Kept(torch.zeros((3, 64), dtype=torch.int8), torch.zeros((3, 2), dtype=torch.uint8))
    with pytest.raises(ValueError, match="on the GPU"):
        T.keep(x)
    with pytest.raises(ValueError, match="bfloat16"):
        T.keep(x.float())
    with pytest.raises(ValueError, match="2 dimensions"):
        T.keep(x[0])
    with pytest.raises(ValueError, match="on the GPU"):
        T.restore(kept)
    with pytest.raises(ValueError, match="exponents: expected"):
        T._want_kept("kept", kept._replace(exponents=torch.zeros((3, 3), dtype=torch.uint8)), 3, 64, -1)
    with pytest.raises(ValueError, match="codes: expected"):
        T.restore(kept._replace(codes=torch.zeros((3, 64), dtype=torch.uint8)))
    with pytest.raises(ValueError, match="even length"):
        T.swiglu(x[:, :63])
    with pytest.raises(ValueError, match="on the GPU"):
        T.swiglu(x)
    with pytest.raises(ValueError):
        T.swiglu_backward(x, x)  # [3, 64] where [3, 128] is
    with pytest.raises(ValueError):
        T.swiglu_backward(x, kept)  # 3 rows where 6 are
    ids = torch.zeros((3, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        T.experts_mlp(x.repeat(1, 4), ids, None, (x, x, x), (x, x, x), T.Geometry(1, 256, 12, 2, 256, 80, 0),
                      T.Geometry(0, 256, 12, 2, 40, 256, 0))
    with pytest.raises(ValueError, match="x: expected"):
        T.experts_mlp(x, ids, None, (x, x, x), (x, x, x), T.Geometry(1, 256, 12, 2, 256, 80, 0),
                      T.Geometry(0, 256, 12, 2, 40, 256, 0))


def test_overlaps_are_refused(T):
    a = torch.zeros(64, dtype=torch.int8)
    kept = T.Kept(a[:32].view(1, 32), a[40:41].view(torch.uint8).view(1, 1))
    T._apart(T._kept_parts("kept", kept), {"x": a[41:]})
    with pytest.raises(ValueError, match="kept.codes overlaps x"):
        T._apart(T._kept_parts("kept", kept), {"x": a[31:40]})


def test_reference_of_kept_rows():
    """The oracle itself: values at the edges of the format, by hand."""
    big = torch.tensor([[1.0, -1.9921875, 0.0078125, 0.0]]).to(torch.bfloat16)
    codes, exponents = ref.keep(big)
    # E = 127: steps of 2^-6; 127.5 steps are cut off at 127, half a step goes to the even 0
    assert exponents.tolist() == [[127]] and codes.tolist() == [[64, -127, 0, 0]]
    assert ref.restore(codes, exponents).tolist() == [[1.0, -1.984375, 0.0, 0.0]]
    tiny = ref.bf16(np.array([[1, 0x7F, 0x8005]], np.uint16))  # subnormals
    codes, exponents = ref.keep(tiny)
    assert exponents.tolist() == [[0]] and codes.tolist() == [[1, 127, -5]]
    assert torch.equal(ref.restore(codes, exponents), tiny)
    for bad in (float("inf"), float("nan")):
        codes, exponents = ref.keep(torch.tensor([[bad, 1.0]]).to(torch.bfloat16))
        assert exponents.tolist() == [[255]] and bool(ref.restore(codes, exponents).isnan().all())
