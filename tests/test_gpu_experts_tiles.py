"""The experts' coded products over many rows: tiles of 32, 64 or 128 rows of one
expert, whose rows are laid out in a workspace first.

Which tile a call takes goes by its rows, experts and outputs. Every test here
names the tile it is for and asserts it (the workspace's size tells which one
the library chose), so that a change of the rule cannot leave a kernel untested.
Exactness as in test_gpu_experts.py: integer sums, equal to the rounded bf16
value.
"""
import ctypes as C

import numpy as np
import pytest
import torch

from dequant_gemm_trellis_amd import synth
from helpers import TOL, gate, say
from test_gpu_experts import Problem

pytestmark = pytest.mark.gpu


def workspace_bytes(T, shape, rows, experts):
    g = T.Geometry.of(shape)
    return T.raw().trellis_experts_workspace_bytes(C.byref(g), rows, experts)


def tile_of(T, shape, rows, experts):
    """Rows of the call's tiles: 32, 64 or 128, or 0 where it takes no workspace."""
    nbytes = workspace_bytes(T, shape, rows, experts)
    if nbytes == 0:
        return 0
    values = (shape.in_features + 31) // 32 * 32
    fits = [per for per in (32, 64, 128)
            if (rows // per + min(experts, rows)) * per * values * 2 == nbytes]
    assert len(fits) == 1, fits
    return fits[0]


def wanted(T, p, tile):
    assert tile_of(T, p.shape, p.rows, len(p.counts)) == tile
    return p


# rows of five experts: one without rows, one of a single row, tiles that end early
COUNTS = {32: [463, 0, 1, 32, 505], 64: [1900, 0, 1, 65, 2037], 128: [3001, 0, 1, 257, 4747]}
# axis, in, out, k, tile, block interleave: two and three blocks of axis 1; on axis 0 whole 32-row
# steps, a part of one in rows of 16-byte pieces (264) and in others (300, 37)
TILES = [
    (1, 512, 2170, 2, 32, 0), (1, 768, 2170, 3, 32, 0), (1, 512, 2176, 4, 32, 2),
    (1, 768, 1085, 2, 64, 0), (1, 512, 1088, 3, 64, 2), (1, 512, 1085, 4, 64, 0),
    (1, 512, 1090, 2, 128, 2), (1, 768, 1085, 3, 128, 0), (1, 768, 1088, 4, 128, 0),
    (0, 300, 2304, 2, 32, 0), (0, 264, 2560, 3, 32, 2), (0, 96, 2304, 4, 32, 0),
    (0, 264, 1280, 2, 64, 0), (0, 37, 1280, 3, 64, 0), (0, 300, 1536, 4, 64, 2),
    (0, 96, 1536, 2, 128, 2), (0, 300, 1280, 3, 128, 0), (0, 264, 1280, 4, 128, 0),
]


@pytest.mark.parametrize("axis,i,o,k,tile,il", TILES)
def test_exact(gpu_lib, axis, i, o, k, tile, il):
    say(f"experts axis {axis} {i} -> {o} k={k}, tiles of {tile}, interleave {il}")
    p = wanted(gpu_lib, Problem(21, axis, i, o, k, COUNTS[tile], behind=5, il=il), tile)
    y = torch.full((p.rows, o), 3.0, dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.experts(*p.cuda(), p.shape, y=y) is y
    n = sum(p.counts)
    assert torch.equal(y[:n].cpu(), p.want().to(torch.bfloat16))
    assert bool((y[n:] == 3.0).all())  # rows behind the last expert, left as they were


@pytest.mark.parametrize("axis,i,o,k,tile", [(1, 2048, 1088, 3, 64), (1, 2048, 1088, 4, 128),
                                             (0, 1000, 1280, 2, 64), (0, 1000, 1280, 4, 128)])
def test_normal_values(gpu_lib, axis, i, o, k, tile):
    say(f"experts normal values axis {axis} {i} -> {o} k={k}, tiles of {tile}")
    p = wanted(gpu_lib, Problem(22, axis, i, o, k, COUNTS[tile], exact=False), tile)
    y = gpu_lib.experts(*p.cuda(), p.shape)
    assert gate(y.double().cpu().numpy(), p.want().numpy()) <= TOL
    for _ in range(3):  # a fixed order: equal bits
        assert torch.equal(gpu_lib.experts(*p.cuda(), p.shape), y)


@pytest.mark.parametrize("axis,i,o,tile", [(1, 512, 1085, 128), (0, 80, 1280, 64)])
def test_wild_offsets(gpu_lib, axis, i, o, tile):
    """Offsets outside [0, rows] are clamped, falling ones select nothing."""
    say(f"experts with wild offsets, axis {axis}, tiles of {tile}")
    rows = sum(COUNTS[tile])
    p = wanted(gpu_lib, Problem(23, axis, i, o, 3, [rows // 2, rows - rows // 2]), tile)
    x, _, codes, scales, lut = p.cuda()
    y = torch.full((rows, o), 3.0, dtype=torch.bfloat16, device="cuda")
    cut = torch.tensor([-7, rows // 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    gpu_lib.experts(x, cut, codes, scales, lut, p.shape, y=y)
    assert torch.equal(y.cpu(), p.want().to(torch.bfloat16))
    y.fill_(3.0)
    cut = torch.tensor([rows // 2, 0, -3], dtype=torch.int32, device="cuda")
    gpu_lib.experts(x, cut, codes, scales, lut, p.shape, y=y)
    assert bool((y == 3.0).all())


@pytest.mark.parametrize("axis,i,o", [(1, 256, 2176), (0, 64, 2304)])
def test_offsets_that_go_back_and_forth(gpu_lib, axis, i, o):
    """Eight times the tiles that ascending offsets can make: the ordered rows stay
    within a workspace of exactly the size that the library asks for, and every
    row is untouched or one expert's (here all experts are alike)."""
    rows, experts = 3000, 16
    say(f"experts with offsets back and forth, axis {axis}, {rows} rows")
    p = Problem(24, axis, i, o, 3, [rows])
    assert tile_of(gpu_lib, p.shape, rows, experts) > 0
    need = workspace_bytes(gpu_lib, p.shape, rows, experts)
    x, _, codes, scales, lut = p.cuda()
    y = torch.full((rows, o), 3.0, dtype=torch.bfloat16, device="cuda")
    room = torch.full((need + 2 * 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    cut = torch.tensor([0, rows] * 8 + [0], dtype=torch.int32, device="cuda")
    gpu_lib.experts(x, cut, codes.repeat(experts, 1, 1), scales.repeat(experts, 1), lut, p.shape,
                    y=y, workspace=room[4096:4096 + need])
    assert bool((room[:4096] == 0x5A).all()) and bool((room[4096 + need:] == 0x5A).all())
    want = p.want().to(torch.bfloat16)
    same = (y.cpu() == want).all(1)
    assert bool((same | (y.cpu() == 3.0).all(1)).all()) and bool(same.any())


@pytest.mark.parametrize("axis,i,o,tile", [(1, 512, 2170, 32), (1, 512, 1085, 128), (0, 80, 2304, 32),
                                           (0, 80, 1280, 128)])
def test_not_finite_rows_stay_alone(gpu_lib, axis, i, o, tile):
    """NaN in some rows and behind the last expert's; the workspace holds NaN before."""
    say(f"experts with NaN rows, axis {axis}, tiles of {tile}")
    p = wanted(gpu_lib, Problem(25, axis, i, o, 2, COUNTS[tile], behind=2), tile)
    n = sum(p.counts)
    bad = [1, p.counts[0] + 4, n - 1, p.rows - 1]
    want = p.want().to(torch.bfloat16)
    p.x[bad] = float("nan")
    need = workspace_bytes(gpu_lib, p.shape, p.rows, len(p.counts))
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    y = gpu_lib.experts(*p.cuda(), p.shape, workspace=ws)[:n].cpu()
    fine = torch.ones(n, dtype=torch.bool)
    fine[bad[:3]] = False
    assert torch.equal(y[fine], want[fine]) and bool(y[bad[:3]].isnan().all())


def test_gradient_is_the_other_axis(gpu_lib):
    """<experts(x), d> = <x, experts with the axis flipped (d)>, exactly for
    integers whose outputs stay below 2^8."""
    say("experts gradient on the other axis, tiles")
    g = np.random.default_rng(26)
    p = wanted(gpu_lib, Problem(26, 1, 2304, 2304, 3, COUNTS[32]), 32)
    flipped = synth.Shape(0, 256, 12, 3, 2304, 2304)
    assert tile_of(gpu_lib, flipped, p.rows, len(p.counts)) == 32
    p.scales[:] = 0.5
    p.x[torch.from_numpy(g.random(p.x.shape) < 0.99)] = 0
    d = torch.from_numpy(g.integers(-1, 2, (p.rows, 2304)).astype(np.float32))
    d[torch.from_numpy(g.random(d.shape) < 0.98)] = 0
    d = d.to(torch.bfloat16).cuda()
    x, offsets, codes, scales, lut = p.cuda()
    y = gpu_lib.experts(x, offsets, codes, scales, lut, p.shape)
    dx = gpu_lib.experts(d, offsets, codes, scales, lut, flipped)
    assert float(y.abs().max()) <= 128 and float(dx.abs().max()) <= 128
    assert float((y.double() * d.double()).sum()) == float((dx.double() * x.double()).sum())


def test_captured_and_replayed(gpu_lib):
    """Both axes in one graph, replayed with other rows and offsets between eager calls."""
    T, rows, e = gpu_lib, 1200, 5
    say(f"experts captured, {rows} rows, tiles")
    p = Problem(27, 1, 2304, 2304, 3, [rows] + [0] * (e - 1), exact=False)
    x, offsets, codes, scales, lut = p.cuda()
    flipped = synth.Shape(0, 256, 12, 3, 2304, 2304)
    assert tile_of(T, p.shape, rows, e) == 32 and tile_of(T, flipped, rows, e) == 32
    g = np.random.default_rng(27)
    sets = []
    for _ in range(3):
        cuts = np.concatenate([[0], np.sort(g.integers(0, rows + 1, e - 1)), [rows]]).astype(np.int32)
        sets.append((torch.from_numpy(g.standard_normal((rows, 2304)).astype(np.float32)).to(
            torch.bfloat16).cuda(), torch.from_numpy(cuts).cuda()))

    def chain(x, offsets):
        y = T.experts(x, offsets, codes, scales, lut, p.shape)
        return y, T.experts(y, offsets, codes, scales, lut, flipped)

    chain(x, offsets)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = chain(x, offsets)
    for n in (0, 1, 2, 2, 0):
        x.copy_(sets[n][0]), offsets.copy_(sets[n][1])
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(kept, chain(*sets[n])):
            assert torch.equal(got, want)


def test_two_calls_at_once(gpu_lib):
    """The same codes and rows on two streams at the same time, each call with a
    workspace of its own: every call's bits are those of a call alone."""
    say("experts on two streams at once, tiles")
    p = wanted(gpu_lib, Problem(28, 1, 512, 2170, 3, COUNTS[32]), 32)
    q = wanted(gpu_lib, Problem(28, 0, 300, 1280, 4, COUNTS[64]), 64)
    a, b = p.cuda(), q.cuda()
    want = [v.want().to(torch.bfloat16) for v in (p, q)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for args, shape in ((a, p.shape), (b, q.shape)):
            for n in range(2):
                got[n].append(gpu_lib.experts(*args, shape, stream=streams[n]))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for ys in got:
        for c, y in enumerate(ys):
            assert torch.equal(y.cpu(), want[c % 2])


def test_a_layer_of_experts(gpu_lib):
    """As they are used over a prompt: route, dispatch, the experts' product, combine
    and the gradients back to the tokens, on another stream than the current one."""
    T, tokens, top_k, e, n = gpu_lib, 400, 3, 5, 2304
    say(f"a layer of experts, {tokens} tokens, tiles")
    p = Problem(29, 1, n, n, 4, [0] * e, exact=False)
    flipped = synth.Shape(0, 256, 12, 4, n, n)
    assert tile_of(T, p.shape, tokens * top_k, e) == tile_of(T, flipped, tokens * top_k, e) == 32
    g = np.random.default_rng(29)
    ids = torch.from_numpy(np.stack([g.permutation(e)[:top_k] for _ in range(tokens)]).astype(np.int32))
    ids[torch.from_numpy(g.random(ids.shape) < 0.1)] = -1
    x, d = (torch.from_numpy(g.standard_normal((tokens, n)).astype(np.float32)).to(torch.bfloat16)
            for _ in range(2))
    w = torch.softmax(torch.from_numpy(g.standard_normal((tokens, top_k)).astype(np.float32)), 1)
    _, _, codes, scales, lut = p.cuda()
    dev_ids, dev_x, dev_w, dev_d = ids.cuda(), x.cuda(), w.cuda(), d.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = T.route(dev_ids, e)
        xs = T.dispatch(dev_x, r)
        ys = T.experts(xs, r.offsets, codes, scales, lut, p.shape)
        z = T.combine(ys, dev_w, r)
        dys, dw = T.combine_backward(dev_d, ys, dev_w, r)
        dxs = T.experts(dys, r.offsets, codes, scales, lut, flipped)
        dx = T.combine(dxs, None, r)
    torch.cuda.current_stream().wait_stream(side)
    # Every bf16 rounding is off by at most 2^-8 of its value; `slack` sums what
    # reaches an output: of the experts' rows, and of the output itself. Float32
    # sums are off by at most 2^-24 of the summed magnitudes per addition.
    xd, dd, wd, half = x.double(), d.double(), w.double(), 2.0 ** -8
    fp32 = 2 * n * 2.0 ** -24
    want, slack, want_dx, slack_dx = (torch.zeros((tokens, n)).double() for _ in range(4))
    want_dw, slack_dw = torch.zeros((2, tokens, top_k)).double()
    for a in range(e):
        c = p.weights(a)
        for j in range(top_k):
            m = (ids[:, j] == a).nonzero()[:, 0]
            if not len(m):
                continue
            wm = wd[m, j][:, None]
            row, size = xd[m] @ c, xd[m].abs() @ c.abs()
            back, bsize = wm * (dd[m] @ c.T), wm * (dd[m].abs() @ c.abs().T)
            want[m] += wm * row
            slack[m] += wm * (half * row.abs() + 2 * fp32 * size)
            want_dw[m, j] = (dd[m] * row).sum(1)
            slack_dw[m, j] = (dd[m].abs() * (half * row.abs() + 2 * fp32 * size)).sum(1)
            want_dx[m] += back
            slack_dx[m] += half * back.abs() + (half + 2 * fp32) * bsize
    for got, ref, more in ((z, want, slack), (dx, want_dx, slack_dx), (dw, want_dw, slack_dw)):
        assert bool(((got.double().cpu() - ref).abs() <= 1.01 * (more + half * (ref.abs() + more))).all())


@pytest.mark.parametrize("i,rows", [(37, 40), (5, 40), (300, 40), (264, 40), (37, 4003), (300, 4003),
                                    (264, 4003), (45, 8007)])
def test_infinite_weights_on_axis_0(gpu_lib, i, rows):
    """Stored rows whose weights overflow, where the last step of 32 stored rows is
    not full (i % 32): only what the product counts enters it, so an infinity stays
    one (or is NaN where its x is 0, by the formula)."""
    say(f"experts with infinite weights, axis 0, {i} inputs, {rows} rows")
    p = Problem(30, 0, i, 1280, 3, [rows // 3, rows - rows // 3])
    p.lut[p.lut == 0] = 1.0
    # the last stored row, and one that the last 32 stored rows hold beside the last step's
    bad = sorted({i - 1, max(0, 32 * ((i - 1) // 32) - 1)})
    p.scales[:, bad] = 3e38
    p.x[:, bad] = 1.0
    p.x[::5, bad[0]] = 0.0
    p.x[1::5] = p.x[1::5].abs()
    y = gpu_lib.experts(*p.cuda(), p.shape).cpu()
    parts, sizes, at = [], [], 0
    for e, n in enumerate(p.counts):
        w = p.weights(e)
        assert bool(w[bad].isinf().any())
        q = p.x[at:at + n].double()
        finite = q @ torch.where(w.isinf(), 0.0, w)
        sizes.append(q.abs() @ torch.where(w.isinf(), 0.0, w.abs()))
        for b in bad:  # infinite terms, added one by one
            finite += q[:, b, None] * torch.where(w[b].isinf(), w[b], 0.0)[None]
        parts.append(finite)
        at += n
    want, size = torch.cat(parts), torch.cat(sizes)
    rounded, y = want.to(torch.bfloat16).double(), y.double()
    assert bool(rounded.isinf().any()) and bool(rounded.isnan().any()) and bool(rounded.isfinite().any())
    assert torch.equal(y.isnan(), rounded.isnan())
    assert torch.equal(y[y.isinf()], rounded[rounded.isinf()])
    assert torch.equal(y.isinf(), rounded.isinf())
    # A weight of +-1 times the scale stays finite, and a float32 sum that it enters
    # is off by up to 2^-24 of the magnitudes per addition: two such weights of
    # opposite signs cancel and leave that error, not the small terms between them.
    fine = rounded.isfinite()
    off, fp32 = (y - want)[fine].abs(), (i + 1) * 2.0 ** -24 * size[fine]
    assert bool((off <= 2.0 ** -8 * (want[fine].abs() + fp32) + fp32).all())
