"""The experts' coded products over sorted rows (trellis_experts) against the CPU
oracle's weights in float64.

With an integer codebook, power-of-two scales and small-integer rows every sum
is exact in float32, so outputs must equal the exact value rounded to bf16. With
a normal codebook outputs stay within the library's floored 1e-2 relative error.
"""
import numpy as np
import pytest
import torch

import oracle
from dequant_gemm_trellis_amd import synth
from helpers import TOL, gate, say

pytestmark = pytest.mark.gpu


class Problem:
    """Host tensors: codes, scales, lut of `experts` projections, rows and offsets."""

    def __init__(self, seed, axis, i, o, k, counts, behind=0, exact=True, il=0):
        self.shape = synth.Shape(axis, 256, 12, k, i, o, il)
        plain = synth.Shape(axis, 256, 12, k, i, o)
        g = np.random.default_rng([seed, axis, i, o, k, len(counts)])
        e, rows = len(counts), sum(counts) + behind
        self.counts, self.rows = counts, rows
        codes = g.integers(0, 2 ** 32, (e, plain.rows, plain.words_per_row), dtype=np.uint32)
        self.lut = synth.integer_lut() if exact else g.standard_normal(4096).astype(np.float32)
        self.scales = (g.choice([0.5, 1.0, 2.0], (e, plain.rows)) if exact
                       else g.uniform(0.5, 1.5, (e, plain.rows))).astype(np.float32)
        x = g.integers(-2, 3, (rows, i)) if exact else g.standard_normal((rows, i))
        self.x = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
        self.offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
        self.plain_codes = codes
        if il:
            codes = np.stack([oracle.interleave_blocks(c, plain.rows, plain.cols // 256, 8 * k)
                              for c in codes])
        self.codes = torch.from_numpy(codes.view(np.int32))

    def weights(self, e):
        s = self.shape
        w = oracle.expand(self.plain_codes[e], self.scales[e], self.lut, s.axis, 256, 12, s.k,
                          s.in_features, s.out_features)
        w = torch.from_numpy(w.view(np.int16)).view(torch.bfloat16).double().reshape(s.rows, s.cols)
        return w.T.contiguous() if s.axis == 1 else w  # [in, out]

    def cuda(self):
        return (self.x.cuda(), self.offsets.cuda(), self.codes.cuda(),
                torch.from_numpy(self.scales).cuda(), torch.from_numpy(self.lut).cuda())

    def want(self):
        """[sum(counts), out] in float64."""
        parts, at = [], 0
        for e, n in enumerate(self.counts):
            if n:
                parts.append(self.x[at:at + n].double() @ self.weights(e))
            at += n
        return torch.cat(parts) if parts else torch.zeros((0, self.shape.out_features)).double()


# axis, in, out, k, rows of each expert
CASES = [
    (1, 256, 1, 2, [1]), (1, 256, 16, 3, [0, 1, 0]), (1, 512, 300, 4, [3, 0, 17, 1]),
    (1, 1024, 37, 2, [16, 16, 16]), (1, 2048, 129, 3, [5, 0, 0, 2, 9]),
    (1, 768, 260, 4, [1] * 70), (1, 2304, 96, 2, [2, 3]),
    (1, 512, 300, 2, [40, 0, 65, 3]), (1, 256, 70, 3, [64, 1]), (1, 512, 200, 4, [17, 33, 60]),
    (1, 512, 200, 2, [129, 127, 0]), (1, 768, 1000, 3, [300, 1]), (1, 256, 64, 4, [128, 400]),
    (0, 1, 256, 2, [1]), (0, 300, 256, 3, [0, 1, 0]), (0, 37, 512, 4, [3, 0, 17, 1]),
    (0, 256, 256, 2, [16, 16, 16]), (0, 1000, 256, 3, [1] * 70),
    (0, 300, 512, 2, [40, 0, 65, 3]), (0, 64, 256, 4, [32, 33, 31]),
    (0, 264, 512, 2, [129, 127, 0]), (0, 100, 768, 3, [300, 1]), (0, 33, 256, 4, [65, 130]),
]


@pytest.mark.parametrize("axis,i,o,k,counts", CASES)
def test_exact(gpu_lib, axis, i, o, k, counts):
    say(f"experts axis {axis} {i} -> {o} k={k} rows {counts[:5]}")
    p = Problem(1, axis, i, o, k, counts, behind=5)
    y = torch.full((p.rows, o), 3.0, dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.experts(*p.cuda(), p.shape, y=y) is y
    want = p.want().to(torch.bfloat16)
    n = sum(counts)
    assert torch.equal(y[:n].cpu(), want)
    assert bool((y[n:] == 3.0).all())  # rows behind the last expert, left as they were


@pytest.mark.parametrize("axis,i,o,k,counts", [(1, 1024, 300, 3, [7, 20, 0]), (0, 300, 1024, 4, [9, 1]),
                                               (1, 512, 100, 2, [100, 90]), (0, 70, 512, 2, [70, 50])])
def test_block_pairs(gpu_lib, axis, i, o, k, counts):
    say(f"experts block pairs axis {axis} {i} -> {o} k={k}")
    p = Problem(2, axis, i, o, k, counts, il=2)
    y = gpu_lib.experts(*p.cuda(), p.shape)
    assert torch.equal(y.cpu(), p.want().to(torch.bfloat16))


@pytest.mark.parametrize("axis,i,o,k,counts", [(1, 2048, 520, 3, [4] * 9), (1, 2048, 520, 2, [200, 3]),
                                               (0, 768, 512, 4, [4] * 9), (0, 768, 512, 3, [200, 3])])
def test_normal_values(gpu_lib, axis, i, o, k, counts):
    say(f"experts normal values axis {axis} {i} -> {o} k={k}")
    p = Problem(3, axis, i, o, k, counts, exact=False)
    y = gpu_lib.experts(*p.cuda(), p.shape)
    assert gate(y.double().cpu().numpy(), p.want().numpy()) <= TOL
    for _ in range(3):  # a fixed order: equal bits
        assert torch.equal(gpu_lib.experts(*p.cuda(), p.shape), y)


def test_no_rows(gpu_lib):
    say("experts without rows")
    p = Problem(4, 1, 256, 64, 2, [0, 0])
    assert tuple(gpu_lib.experts(*p.cuda(), p.shape).shape) == (0, 64)
    p = Problem(4, 0, 64, 256, 2, [0, 0], behind=3)
    y = torch.full((3, 256), 2.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.experts(*p.cuda(), p.shape, y=y)
    assert bool((y == 2.0).all())


@pytest.mark.parametrize("axis,i,o", [(1, 256, 80), (0, 80, 256)])
@pytest.mark.parametrize("rows", [30, 500])
def test_wild_offsets(gpu_lib, axis, i, o, rows):
    """Offsets outside [0, rows] are clamped, falling ones select nothing."""
    say(f"experts with wild offsets, axis {axis}, {rows} rows")
    p = Problem(5, axis, i, o, 3, [rows // 2, rows - rows // 2])
    x, _, codes, scales, lut = p.cuda()
    y = torch.full((rows, o), 3.0, dtype=torch.bfloat16, device="cuda")
    cut = torch.tensor([-7, rows // 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    gpu_lib.experts(x, cut, codes, scales, lut, p.shape, y=y)
    want = p.want().to(torch.bfloat16)
    assert torch.equal(y.cpu(), want)
    y.fill_(3.0)
    cut = torch.tensor([rows // 2, 0, -3], dtype=torch.int32, device="cuda")
    gpu_lib.experts(x, cut, codes, scales, lut, p.shape, y=y)
    assert bool((y == 3.0).all())


@pytest.mark.parametrize("axis,i,o", [(1, 256, 64), (0, 64, 256)])
@pytest.mark.parametrize("rows", [30, 3000])
def test_offsets_that_go_back_and_forth(gpu_lib, axis, i, o, rows):
    """More tiles than ascending offsets can make: within bounds, every row
    untouched or one expert's (here all experts are alike)."""
    say(f"experts with offsets back and forth, axis {axis}, {rows} rows")
    p = Problem(11, axis, i, o, 3, [rows])
    x, _, codes, scales, lut = p.cuda()
    y = torch.full((rows, o), 3.0, dtype=torch.bfloat16, device="cuda")
    cut = torch.tensor([0, rows] * 8 + [0], dtype=torch.int32, device="cuda")
    gpu_lib.experts(x, cut, codes.repeat(16, 1, 1), scales.repeat(16, 1), lut, p.shape, y=y)
    want = p.want().to(torch.bfloat16)
    same = (y.cpu() == want).all(1)
    assert bool((same | (y.cpu() == 3.0).all(1)).all()) and bool(same.any())


@pytest.mark.parametrize("axis,i,o", [(1, 512, 80), (0, 80, 512)])
def test_not_finite_rows_stay_alone(gpu_lib, axis, i, o):
    say(f"experts with NaN rows, axis {axis}")
    for counts in ([3, 20, 2], [150, 20, 2]):
        p = Problem(6, axis, i, o, 2, counts, behind=2)
        bad = [1, counts[0] + 4, p.rows - 1]
        want = p.want().to(torch.bfloat16)
        p.x[bad] = float("nan")
        y = gpu_lib.experts(*p.cuda(), p.shape)[:sum(counts)].cpu()
        fine = torch.ones(sum(counts), dtype=torch.bool)
        fine[bad[:2]] = False
        assert torch.equal(y[fine], want[fine]) and bool(y[bad[:2]].isnan().all())


@pytest.mark.parametrize("axis,i,o", [(0, 33, 2048), (1, 256, 2049)])
def test_offsets_past_32_bits(gpu_lib, axis, i, o):
    """More than 2^31 outputs, the last rows another expert's."""
    say(f"experts past 2^31 values, axis {axis}")
    rows, tail = 1050000, 200
    p = Problem(10, axis, i, o, 3, [50, tail])
    x, _, codes, scales, lut = p.cuda()
    assert rows * o > 2 ** 31
    x = torch.cat([x.new_zeros((rows - tail, i)), x[50:]])
    offsets = torch.tensor([0, rows - tail, rows], dtype=torch.int32, device="cuda")
    y = gpu_lib.experts(x, offsets, codes, scales, lut, p.shape)
    assert torch.equal(y[-tail:].cpu(), p.want()[50:].to(torch.bfloat16))
    assert not y[:-tail].any()


def test_gradient_is_the_other_axis(gpu_lib):
    """<experts(x), d> = <x, experts with the axis flipped (d)>, exactly for
    integers whose outputs stay below 2^8."""
    say("experts gradient on the other axis")
    g = np.random.default_rng(7)
    for counts in ([5, 0, 11], [90, 100]):
        p = Problem(7, 1, 256, 40, 3, counts)
        p.scales[:] = 0.5
        p.x[torch.from_numpy(g.random(p.x.shape) < 0.9)] = 0
        d = torch.from_numpy((g.integers(-1, 2, (p.rows, 40))).astype(np.float32)).to(torch.bfloat16)
        x, offsets, codes, scales, lut = p.cuda()
        y = gpu_lib.experts(x, offsets, codes, scales, lut, p.shape)
        dx = gpu_lib.experts(d.cuda(), offsets, codes, scales, lut, synth.Shape(0, 256, 12, 3, 40, 256))
        assert float(y.abs().max()) <= 128 and float(dx.abs().max()) <= 128
        assert float((y.double() * d.cuda().double()).sum()) == float((dx.double() * x.double()).sum())


@pytest.mark.parametrize("rows,e", [(40, 8), (900, 5)])
def test_captured_and_replayed(gpu_lib, rows, e):
    """Both axes in one graph, replayed with other rows and offsets."""
    say(f"experts captured, {rows} rows")
    T = gpu_lib
    p = Problem(8, 1, 512, 256, 3, [rows] + [0] * (e - 1), exact=False)
    x, offsets, codes, scales, lut = p.cuda()
    flipped = synth.Shape(0, 256, 12, 3, 256, 512)
    g = np.random.default_rng(8)
    sets = []
    for _ in range(3):
        cuts = np.concatenate([[0], np.sort(g.integers(0, rows + 1, e - 1)), [rows]]).astype(np.int32)
        sets.append((torch.from_numpy(g.standard_normal((rows, 512)).astype(np.float32)).to(
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


@pytest.mark.parametrize("tokens", [3, 150])
def test_a_layer_of_experts(gpu_lib, tokens):
    """As they are used: route, dispatch, the experts' product, combine, and the
    gradients back to the tokens, on another stream than the current one."""
    say(f"a layer of experts, {tokens} tokens")
    T, top_k, e, i, o = gpu_lib, 3, 8, 512, 256
    p = Problem(9, 1, i, o, 4, [0] * e, exact=False)
    g = np.random.default_rng(9)
    ids = torch.from_numpy(np.stack([g.permutation(e)[:top_k] for _ in range(tokens)]).astype(np.int32))
    ids[torch.from_numpy(g.random(ids.shape) < 0.1)] = -1
    x, d = (torch.from_numpy(g.standard_normal((tokens, n)).astype(np.float32)).to(torch.bfloat16)
            for n in (i, o))
    w = torch.softmax(torch.from_numpy(g.standard_normal((tokens, top_k)).astype(np.float32)), 1)
    _, _, codes, scales, lut = p.cuda()
    dev_ids, dev_x, dev_w, dev_d = ids.cuda(), x.cuda(), w.cuda(), d.cuda()
    flipped = synth.Shape(0, 256, 12, 4, o, i)
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
    # reaches an output: of the experts' rows, and of the output itself.
    weights = [p.weights(n) for n in range(e)]
    xd, dd, wd, half = x.double(), d.double(), w.double(), 2.0 ** -8
    fp32 = (i + o) * 2.0 ** -24  # float32 sums, per unit of summed magnitude
    want, slack = torch.zeros((2, tokens, o)).double()
    want_dx, slack_dx = torch.zeros((2, tokens, i)).double()
    want_dw, slack_dw = torch.zeros((2, tokens, top_k)).double()
    for m in range(tokens):
        for j in range(top_k):
            if ids[m, j] < 0:
                continue
            c = weights[ids[m, j]]
            row, back = xd[m] @ c, wd[m, j] * (c @ dd[m])
            size = xd[m].abs() @ c.abs()
            want[m] += wd[m, j] * row
            slack[m] += wd[m, j] * (half * row.abs() + 2 * fp32 * size)
            want_dw[m, j] = dd[m] @ row
            slack_dw[m, j] = dd[m].abs() @ (half * row.abs() + 2 * fp32 * size)
            want_dx[m] += back
            slack_dx[m] += half * back.abs() + (half + 2 * fp32) * wd[m, j] * (c.abs() @ dd[m].abs())
    for got, ref, more in ((z, want, slack), (dx, want_dx, slack_dx), (dw, want_dw, slack_dw)):
        assert bool(((got.double().cpu() - ref).abs() <= 1.01 * (more + half * (ref.abs() + more))).all())


@pytest.mark.parametrize("axis,i,o", [(1, 256, 16), (0, 32, 256)])
@pytest.mark.parametrize("most", [1, 40])
def test_the_most_experts(gpu_lib, axis, i, o, most):
    """1024 experts, three of four without rows; up to 40 rows of the others."""
    say(f"1024 experts axis {axis}, up to {most} rows each")
    g = np.random.default_rng([11, axis, most])
    counts = [int(n) if e % 4 == 1 or e == 1023 else 0 for e, n in enumerate(g.integers(1, most + 1, 1024))]
    p = Problem(11, axis, i, o, 2, counts)
    assert torch.equal(gpu_lib.experts(*p.cuda(), p.shape).cpu(), p.want().to(torch.bfloat16))


@pytest.mark.parametrize("groups", [0, 1025, 2 ** 32 + 4])
def test_route_refuses_numbers_of_groups(gpu_lib, groups):
    with pytest.raises(gpu_lib.TrellisError):
        gpu_lib.route(torch.zeros((3, 2), dtype=torch.int32, device="cuda"), groups)


def test_two_calls_at_once(gpu_lib):
    """The same codes and rows on two streams at the same time, each call with a
    workspace of its own: every call's bits are those of a call alone."""
    say("experts on two streams at once")
    p = Problem(12, 1, 512, 300, 3, [200, 0, 90, 170])
    q = Problem(12, 0, 300, 512, 4, [150, 40, 0, 300])
    a, b = p.cuda(), q.cuda()
    want = [v.want().to(torch.bfloat16) for v in (p, q)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        for args, shape in ((a, p.shape), (b, q.shape)):
            for n in range(2):
                got[n].append(gpu_lib.experts(*args, shape, stream=streams[n]))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for ys in got:
        for c, y in enumerate(ys):
            assert torch.equal(y.cpu(), want[c % 2])
