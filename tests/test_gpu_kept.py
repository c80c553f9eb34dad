"""Rows kept in 8 bits, SwiGLU over many rows and its gradient (trellis_keep,
trellis_restore, trellis_swiglu, trellis_swiglu_backward), and the adapters'
gradient that reads x in 8 bits.

Keeping is exact but for one rounding: codes and exponents must equal the
definition's, restored values the numbers they stand for.

SwiGLU is held to a bound on each value. With eps = 2^-24: the sigmoid's argument
-g log2(e) - 24 is rounded once and its constant once, an absolute error of at most
(1.45 |g| + 24) 2 eps, which exp2 makes a relative error of ln(2) times that; exp2,
the sum, the reciprocal and two products add 8 eps. For |g| <= 104 that is below
(2.1 |g| + 42) eps <= 2^-16. A bf16 result is off by at most half a step, 2^-8 of
its value. In the gradient 1 + g (1 - s) loses up to |g| times s's error besides.
A sigmoid below float32's smallest normal number (g < -87) is off by up to 2^-149
absolutely (its step there, or all of it below g = -104), times the factors of it:
|g u| in h, |dh u| (1 + |g|) in dg and |dh g| in du.
"""
import numpy as np
import pytest
import torch

import kept_reference as ref
from helpers import say

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8     # half a step of bf16
SIGMOID = 2.0 ** -16
STEP = 2.0 ** -149   # float32's subnormal step
TINY = 2.0 ** -133   # bf16's and float32's subnormals: an absolute error


def rows_of(seed, rows, width, std=1.0):
    """bf16 rows with channels of very different sizes, some zeros and a zero group."""
    g = np.random.default_rng([seed, rows, width])
    x = g.standard_normal((rows, width)) * np.exp2(g.integers(-6, 7, (1, width))) * std
    x[g.random((rows, width)) < 0.05] = 0.0
    x[rows // 2, :min(32, width)] = 0.0
    return torch.from_numpy(x).to(torch.bfloat16)


def off(t, values):
    """A dense copy on the GPU whose first element is `values` elements past 256 bytes."""
    flat = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
    at = flat[values:values + t.numel()].view(t.shape)
    at.copy_(t)
    return at


WIDTHS = [1, 7, 8, 9, 31, 32, 33, 63, 64, 255, 1000, 1003, 2047, 2048, 4111, 16391]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 67])
def test_keep_and_restore(gpu_lib, rows, width):
    say(f"keep {rows} x {width}")
    x = rows_of(1, rows, width)
    kept = gpu_lib.keep(x.cuda())
    codes, exponents = ref.keep(x)
    assert torch.equal(kept.exponents.cpu(), exponents)
    assert torch.equal(kept.codes.cpu(), codes)
    back = gpu_lib.restore(kept)
    assert torch.equal(back.cpu(), ref.restore(codes, exponents))
    # half a step of 2^(E - 133), 1/128 of the largest magnitude where E >= 1
    e = exponents.double().repeat_interleave(32, dim=1)[:, :width]
    assert bool(((back.cpu().double() - x.double()).abs() <= torch.exp2(e - 134)).all())


def test_every_bf16_value(gpu_lib):
    """Alone in its group, and beside the largest finite value and a middling one."""
    every = np.arange(1 << 16, dtype=np.uint16)
    say("keep every bf16 value")
    for beside in (None, 0x7F7F, 0x3F80, 0x0080, 0x7F80, 0x7FC0):
        b = np.zeros((1 << 16, 33), np.uint16)
        b[:, 0] = every
        if beside is not None:
            b[:, 31] = beside
        b[:, 32] = every  # and in the short group at the end
        x = ref.bf16(b)
        codes, exponents = ref.keep(x)
        kept = gpu_lib.keep(x.cuda())
        assert torch.equal(kept.exponents.cpu(), exponents)
        assert torch.equal(kept.codes.cpu()[exponents[:, 0] < 255], codes[exponents[:, 0] < 255])
        back, want = gpu_lib.restore(kept).cpu(), ref.restore(codes, exponents)
        assert torch.equal(back.isnan(), want.isnan())
        assert torch.equal(back.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("shift", [1, 2, 3, 5, 8])
def test_keep_off_16_bytes(gpu_lib, shift):
    say(f"keep, arrays {shift} elements off")
    for rows, width in ((5, 64), (3, 100), (70, 33)):
        x = rows_of(2, rows, width)
        codes, exponents = ref.keep(x)
        kept = gpu_lib.Kept(off(torch.zeros_like(codes), shift), off(torch.zeros_like(exponents), 2))
        assert gpu_lib.keep(off(x, shift), kept) is kept
        assert torch.equal(kept.codes.cpu(), codes) and torch.equal(kept.exponents.cpu(), exponents)
        out = off(torch.zeros_like(x), shift)
        gpu_lib.restore(kept, out=out)
        assert torch.equal(out.cpu(), ref.restore(codes, exponents))


def test_nothing_else_is_written(gpu_lib):
    """Bytes around the outputs stay as they were, whatever the row's end."""
    say("bytes around the outputs")
    for rows, width in ((3, 37), (2, 8), (9, 100)):
        x = rows_of(3, rows, width).cuda()
        n, groups = rows * width, -(-width // 32)
        c = torch.full((n + 64,), 85, dtype=torch.int8, device="cuda")
        e = torch.full((rows * groups + 64,), 85, dtype=torch.uint8, device="cuda")
        o = torch.full((n + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
        kept = gpu_lib.Kept(c[32:32 + n].view(rows, width), e[32:32 + rows * groups].view(rows, groups))
        gpu_lib.keep(x, kept)
        gpu_lib.restore(kept, out=o[32:32 + n].view(rows, width))
        for t, m, v in ((c, n, 85), (e, rows * groups, 85), (o, n, 3.0)):
            assert bool((t[:32] == v).all()) and bool((t[32 + m:] == v).all())


def test_no_rows(gpu_lib):
    x = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda")
    kept = gpu_lib.keep(x)
    assert kept.codes.shape == (0, 40) and gpu_lib.restore(kept).shape == (0, 40)
    h, kept = gpu_lib.swiglu(x, keep=True)
    assert h.shape == (0, 20) and kept.codes.shape == (0, 20)
    dgu, h = gpu_lib.swiglu_backward(h, kept, again=True)
    assert dgu.shape == (0, 40) and h.shape == (0, 20)


def near(got, want, slack):
    """Every value within half a bf16 step of its own plus `slack` of the float32 work;
    NaN where the definition has it, and infinities of its sign."""
    got, fine = got.double().cpu(), want.isfinite()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[want.isinf()], want[want.isinf()])
    err = (got - want).abs()[fine]
    bound = (HALF * (1 + 2.0 ** -10) * want.abs() + slack * (1 + HALF) + TINY)[fine]
    assert bool((err <= bound).all()), float((err / bound).max())


def forward_slack(gu):
    g, u = gu.chunk(2, dim=1)
    return SIGMOID * ref.swiglu(gu).abs() + STEP * (g * u).abs()


def backward_slack(dh, gu):
    g, u = gu.chunk(2, dim=1)
    s = torch.sigmoid(g)
    return torch.cat([SIGMOID * (dh * u).abs() * s * (1 + 2 * g.abs()) + STEP * (dh * u).abs() * (1 + g.abs()),
                      SIGMOID * (dh * g).abs() * s + STEP * (dh * g).abs()], dim=1)


INTERS = [1, 5, 8, 31, 32, 33, 100, 768, 1003, 4111, 16400]


@pytest.mark.parametrize("inter", INTERS)
@pytest.mark.parametrize("rows", [1, 66])
def test_swiglu(gpu_lib, rows, inter):
    say(f"swiglu {rows} x {inter}")
    gu = rows_of(4, rows, 2 * inter)
    h, kept = gpu_lib.swiglu(gu.cuda(), keep=True)
    near(h, ref.swiglu(gu.double()), forward_slack(gu.double()))
    codes, exponents = ref.keep(gu.reshape(2 * rows, inter))
    assert torch.equal(kept.codes.cpu(), codes) and torch.equal(kept.exponents.cpu(), exponents)
    alone, none = gpu_lib.swiglu(gu.cuda())
    assert none is None and torch.equal(alone, h)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("inter", INTERS)
@pytest.mark.parametrize("rows", [1, 66])
def test_swiglu_backward(gpu_lib, rows, inter, kept):
    say(f"swiglu backward {rows} x {inter}, kept {kept}")
    gu, dh = rows_of(5, rows, 2 * inter), rows_of(6, rows, inter)
    given = gu.cuda()
    if kept:
        codes, exponents = ref.keep(gu.reshape(2 * rows, inter))
        gu = ref.restore(codes, exponents).reshape(rows, 2 * inter)
        given = gpu_lib.Kept(codes.cuda(), exponents.cuda())
    dgu, h = gpu_lib.swiglu_backward(dh.cuda(), given, again=True)
    near(dgu, ref.swiglu_backward(dh.double(), gu.double()), backward_slack(dh.double(), gu.double()))
    assert torch.equal(h, gpu_lib.swiglu(gu.cuda())[0])
    alone, none = gpu_lib.swiglu_backward(dh.cuda(), given)
    assert none is None and torch.equal(alone, dgu)


@pytest.mark.parametrize("shift", [1, 3, 8])
def test_swiglu_off_16_bytes(gpu_lib, shift):
    say(f"swiglu, arrays {shift} elements off")
    for rows, inter in ((5, 64), (9, 37)):
        gu, dh = rows_of(7, rows, 2 * inter), rows_of(8, rows, inter)
        codes, exponents = ref.keep(gu.reshape(2 * rows, inter))
        kept = gpu_lib.Kept(off(torch.zeros_like(codes), shift), off(torch.zeros_like(exponents), shift))
        h = off(torch.zeros_like(dh), shift)
        assert gpu_lib.swiglu(off(gu, shift), h=h, kept=kept) == (h, kept)
        assert torch.equal(h, gpu_lib.swiglu(gu.cuda())[0])
        assert torch.equal(kept.codes.cpu(), codes) and torch.equal(kept.exponents.cpu(), exponents)
        dgu, again = off(torch.zeros_like(gu), shift), off(torch.zeros_like(dh), 2 * shift)
        gpu_lib.swiglu_backward(off(dh, shift), kept, dgu=dgu, h=again)
        want = gpu_lib.swiglu_backward(dh.cuda(), gpu_lib.Kept(codes.cuda(), exponents.cuda()), again=True)
        assert torch.equal(dgu, want[0]) and torch.equal(again, want[1])


def test_swiglu_at_the_edges(gpu_lib):
    """Gates from -300 to the largest value, infinities and NaN, with large and tiny u."""
    g = torch.tensor([-300.0, -105.0, -104.0, -103.0, -89.0, -88.0, -87.0, -60.0, -1.28, -1e-30, -0.0, 0.0,
                      1e-38, 1.0, 17.0, 88.0, 1e30, 3.3e38, float("inf"), float("nan"), -3.3e38])
    u = torch.tensor([1.0, -2.5, 1e-30, 1e-38, 0.0, 3e38, float("inf"), float("nan")])
    gu = torch.cat([g[:, None].expand(-1, len(u)), u[None, :].expand(len(g), -1)], dim=1)
    gu = gu.to(torch.bfloat16).contiguous()
    say("swiglu at the edges")
    h, _ = gpu_lib.swiglu(gu.cuda())
    g64, u64 = gu.double().chunk(2, dim=1)
    silu = g64 * torch.sigmoid(g64)
    want = (silu * u64)
    # float32's range: products past it are infinite, and a sigmoid below 2^-126 has
    # only 2^-149 as its step
    want = torch.where(want.abs() >= 3.3961e38, torch.sign(want) * torch.inf, want)
    few = (g64 < -87) & (g64 > -3e38)
    # below -105 the sigmoid is 0 in float32: -inf * 0 is not reached with finite g
    zero = g64 <= -104.0
    lost = (torch.where(few, 2.0 ** -149 * g64.abs(), torch.zeros_like(g64)) * u64.abs())
    lost = torch.where(zero, (silu * u64).abs(), lost)
    rows = ~(zero & u64.isinf())
    keep = rows & ~(few & u64.isinf())
    got = h.double().cpu()
    near(torch.where(keep, got, 0.0), torch.where(keep, want, 0.0),
         torch.where(keep & lost.isfinite(), SIGMOID * want.nan_to_num().abs().clamp(max=3.4e38) + lost, 0.0))


def test_gradient_against_differences(gpu_lib):
    """The formula's gradient is the forward formula's difference quotient (float64), and
    the kernel's is the formula's."""
    gu, dh = rows_of(9, 11, 2 * 45).double(), rows_of(10, 11, 45)
    want = ref.swiglu_backward(dh.double(), gu)
    step = 1e-5
    quotient = torch.empty_like(want)
    for n in range(gu.shape[1]):
        d = torch.zeros_like(gu)
        d[:, n] = step
        quotient[:, n] = ((ref.swiglu(gu + d) - ref.swiglu(gu - d)) / (2 * step) * dh.double()).sum(1)
    scale = dh.abs().double().repeat(1, 2) * (1 + gu.abs().max())
    assert bool(((quotient - want).abs() <= 1e-8 * scale + 1e-9).all())
    dgu, _ = gpu_lib.swiglu_backward(dh.cuda(), gu.to(torch.bfloat16).cuda())
    near(dgu, want, backward_slack(dh.double(), gu))


def test_captured_and_replayed(gpu_lib):
    """keep, swiglu with kept rows and its gradient in one graph, replayed with other
    values between the program's own work."""
    rows, inter = 37, 300
    gu, dh = torch.zeros((rows, 2 * inter), dtype=torch.bfloat16, device="cuda"), None
    dh = torch.zeros((rows, inter), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()

    def work():
        h, kept = gpu_lib.swiglu(gu, keep=True)
        again = gpu_lib.restore(gpu_lib.keep(h))
        return h, kept, again, gpu_lib.swiglu_backward(dh, kept)[0]

    with torch.cuda.stream(side):
        work()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for seed in (11, 12, 13, 14):
        say(f"replay {seed}")
        gu.copy_(rows_of(seed, rows, 2 * inter))
        dh.copy_(rows_of(seed + 20, rows, inter))
        graph.replay()
        torch.cuda.synchronize()
        want = work()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1].codes, want[1].codes)
        assert torch.equal(got[1].exponents, want[1].exponents)
        assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])


def test_another_stream(gpu_lib):
    gu = rows_of(15, 200, 1200).cuda()
    want = gpu_lib.swiglu(gu, keep=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, kept = gpu_lib.swiglu(gu, keep=True, stream=side)
    dgu, _ = gpu_lib.swiglu_backward(h, kept, stream=side)
    back = gpu_lib.restore(gpu_lib.keep(gu, stream=side), stream=side)
    side.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(kept.codes, want[1].codes)
    assert torch.equal(dgu, gpu_lib.swiglu_backward(want[0], want[1])[0])
    assert torch.equal(back, gpu_lib.restore(gpu_lib.keep(gu)))


def test_offsets_past_32_bits(gpu_lib):
    """Rows whose values lie beyond 2^31: the last rows are as alone."""
    rows, width = 66000, 33000  # 2.18e9 values
    say(f"keep {rows} x {width}")
    tail = rows_of(16, 3, width).cuda()
    x = torch.zeros((rows, width), dtype=torch.bfloat16, device="cuda")
    x[-3:] = tail
    kept = gpu_lib.keep(x)
    alone = gpu_lib.keep(tail)
    assert torch.equal(kept.codes[-3:], alone.codes) and torch.equal(kept.exponents[-3:], alone.exponents)
    assert not bool(kept.codes[:-3].any())
    out = x.fill_(3.0)
    gpu_lib.restore(kept, out=out)
    assert torch.equal(out[-3:], gpu_lib.restore(alone)) and not bool(out[:-3].any())
    del kept, alone
    gu = x.view(rows, width)
    gu[-3:] = tail
    h, kept = gpu_lib.swiglu(gu, keep=True)
    small = gpu_lib.swiglu(tail, keep=True)
    assert torch.equal(h[-3:], small[0]) and torch.equal(kept.codes[-6:], small[1].codes)
    assert torch.equal(kept.exponents[-6:], small[1].exponents)
    dgu, _ = gpu_lib.swiglu_backward(h, kept, dgu=None)
    assert torch.equal(dgu[-3:], gpu_lib.swiglu_backward(small[0], small[1])[0])


# ---- the adapters' gradient with x in 8 bits ----------------------------------------
#
# It computes the same sums from the values that the codes stand for, so its results
# equal those of the bf16 rows that `restore` gives, bit for bit: both read the same
# values into the same instructions.

SIZES = [(1, 256, 16, 1, 1), (2, 300, 520, 13, 3), (31, 1024, 300, 8, 40), (64, 2048, 264, 16, 5),
         (129, 7, 9, 5, 2), (200, 777, 1000, 33, 4), (500, 264, 640, 64, 70), (130, 512, 384, 128, 3),
         (97, 1, 1, 17, 1024), (257, 264, 392, 16, 6), (513, 64, 72, 8, 9), (1025, 136, 520, 16, 1),
         (2500, 256, 192, 32, 2), (3000, 64, 133, 8, 5), (700, 100, 1000, 40, 3), (203, 512, 4111, 8, 3)]


def adapter_inputs(seed, rows, i, o, rank, count):
    g = np.random.default_rng([seed, rows, i, o])
    draw = lambda *s: torch.from_numpy(g.standard_normal(s)).to(torch.bfloat16).cuda()  # noqa: E731
    return {"dy": draw(rows, o), "u": torch.from_numpy(g.standard_normal((rows, rank))).float().cuda(),
            "ids": torch.from_numpy(g.integers(-1, count, rows).astype(np.int32)).cuda(),
            "a": draw(count, rank, i), "b": draw(count, rank, o),
            "scales": torch.from_numpy(g.uniform(0.5, 2, count)).float().cuda(), "base": draw(rows, i)}


@pytest.mark.parametrize("rows,i,o,rank,count", SIZES)
def test_adapters_gradient(gpu_lib, rows, i, o, rank, count):
    say(f"adapters backward kept {rows} x {i} -> {o}, rank {rank}, {count} adapters")
    p = adapter_inputs(17, rows, i, o, rank, count)
    kept = gpu_lib.keep(rows_of(18, rows, i).cuda())
    args = [p[n] for n in ("u", "ids", "a", "b", "scales")]
    got = gpu_lib.adapters_backward(p["dy"], kept, *args, base=p["base"])
    want = gpu_lib.adapters_backward(p["dy"], gpu_lib.restore(kept), *args, base=p["base"])
    for name, a, b in zip(("dx", "da", "db"), got, want):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("rows", [40, 300])
def test_adapters_gradient_exact(gpu_lib, rows):
    """Small integers: every sum is exact, and so is keeping them."""
    i, o, rank, count = 200, 136, 16, 3
    say(f"adapters backward kept, integers, {rows} rows")
    g = np.random.default_rng(rows)
    draw = lambda *s: torch.from_numpy(g.integers(-1, 2, s)).to(torch.bfloat16)  # noqa: E731
    x, dy, a, b = draw(rows, i), draw(rows, o), draw(count, rank, i), draw(count, rank, o)
    ids = torch.from_numpy(g.integers(-1, count, rows).astype(np.int32))
    u = torch.from_numpy(g.integers(-4, 5, (rows, rank))).float()
    kept = gpu_lib.Kept(*(t.cuda() for t in ref.keep(x)))
    dx, da, db = gpu_lib.adapters_backward(dy.cuda(), kept, u.cuda(), ids.cuda(), a.cuda(), b.cuda(),
                                           torch.full((count,), 0.5, device="cuda"))
    for n in range(count):
        m = (ids == n).nonzero()[:, 0]
        v = 0.5 * (dy[m].double() @ b[n].double().T)
        assert torch.equal(da[n].cpu(), (v.T @ x[m].double()).to(torch.bfloat16))
        assert torch.equal(db[n].cpu(), (0.5 * (u[m].double().T @ dy[m].double())).to(torch.bfloat16))
        assert torch.equal(dx[m.cuda()].cpu(), (v @ a[n].double()).to(torch.bfloat16))
    assert not bool(dx[(ids < 0).cuda()].any())


@pytest.mark.parametrize("rows", [50, 400])
def test_adapters_gradient_off_8_bytes(gpu_lib, rows):
    say(f"adapters backward kept, off 8 bytes, {rows} rows")
    p = adapter_inputs(19, rows, 264, 136, 16, 3)
    kept = gpu_lib.keep(rows_of(20, rows, 264).cuda())
    args = [p[n] for n in ("u", "ids", "a", "b", "scales")]
    want = gpu_lib.adapters_backward(p["dy"], kept, *args)
    moved = gpu_lib.Kept(off(kept.codes, 3), off(kept.exponents, 1))
    for a, b in zip(gpu_lib.adapters_backward(p["dy"], moved, *args), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [50, 400])
def test_adapters_gradient_not_finite(gpu_lib, rows):
    """A group that stands for NaN reaches its own 32 columns of its own adapter's da."""
    say(f"adapters backward kept, NaN, {rows} rows")
    p = adapter_inputs(21, rows, 256, 136, 16, 3)
    p["ids"][:] = torch.arange(rows, device="cuda") % 3 - 1  # -1, 0, 1
    x = rows_of(22, rows, 256)
    x[1, 40] = torch.inf   # adapter 0
    x[3, 100] = torch.nan  # none
    got = gpu_lib.adapters_backward(p["dy"], gpu_lib.keep(x.cuda()),
                                    *[p[n] for n in ("u", "ids", "a", "b", "scales")])
    bad = got[1].isnan().cpu()
    assert bool(bad[0, :, 32:64].all()) and int(bad.sum()) == 16 * 32
    assert not bool(got[0].isnan().any()) and not bool(got[2].isnan().any())


def test_adapters_gradient_no_rows(gpu_lib):
    p = adapter_inputs(23, 0, 64, 72, 8, 3)
    kept = gpu_lib.keep(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    dx, da, db = gpu_lib.adapters_backward(p["dy"], kept, *[p[n] for n in ("u", "ids", "a", "b", "scales")])
    assert dx.shape == (0, 64) and not bool(da.any()) and not bool(db.any())


def test_a_training_step(gpu_lib):
    """An MLP's middle as a training run has it: adapters on both projections, [g, u] and x
    kept in 8 bits, h made again in the backward pass."""
    rows, i, n, o, rank, count = 300, 128, 200, 96, 8, 2
    say("a training step")
    g = np.random.default_rng(24)
    draw = lambda *s: torch.from_numpy(g.standard_normal(s)).to(torch.bfloat16).cuda()  # noqa: E731
    ids = torch.from_numpy(g.integers(0, count, rows).astype(np.int32)).cuda()
    scales = torch.ones(count, device="cuda")
    x, base, dy = draw(rows, i), draw(rows, 2 * n), draw(rows, o)
    a1, b1 = draw(count, rank, i) * i ** -0.5, draw(count, rank, 2 * n) * rank ** -0.5
    a2, b2 = draw(count, rank, n) * n ** -0.5, draw(count, rank, o) * rank ** -0.5
    gu, u1 = gpu_lib.adapters(x, ids, a1, b1, scales, base=base, keep_inner=True)
    h, kept = gpu_lib.swiglu(gu, keep=True)
    _, u2 = gpu_lib.adapters(h, ids, a2, b2, scales, keep_inner=True)
    kept_x = gpu_lib.keep(x)
    # backward: dh comes with da2 once h is there again
    dgu, again = gpu_lib.swiglu_backward(draw(rows, n), kept, again=True)
    dh, da2, db2 = gpu_lib.adapters_backward(dy, again, u2, ids, a2, b2, scales)
    dgu, _ = gpu_lib.swiglu_backward(dh, kept)
    dx, da1, db1 = gpu_lib.adapters_backward(dgu, kept_x, u1, ids, a1, b1, scales)
    # the same from the kept values in float64
    held = gpu_lib.restore(kept).reshape(rows, 2 * n).double().cpu()
    near(again, ref.swiglu(held), forward_slack(held))
    near(dgu, ref.swiglu_backward(dh.double().cpu(), held), backward_slack(dh.double().cpu(), held))
    xs, d = gpu_lib.restore(kept_x).double().cpu(), dgu.double().cpu()
    for k in range(count):
        m = (ids.cpu() == k).nonzero()[:, 0]
        v = d[m] @ b1[k].double().cpu().T
        want, size = v.T @ xs[m], v.abs().T @ xs[m].abs()
        # float32 sums of 300 rows and of 400 columns within them, and one rounding
        bound = HALF * want.abs() + (300 + 400) * 2.0 ** -24 * (d[m].abs() @ b1[k].double().cpu().abs().T).T @ xs[m].abs()
        assert bool(((da1[k].double().cpu() - want).abs() <= bound * (1 + HALF)).all())
        assert size.shape == want.shape
    assert bool(da2.isfinite().all()) and bool(db2.isfinite().all()) and bool(dx.isfinite().all())
    assert bool(db1.isfinite().all())


def test_a_layer_of_experts(gpu_lib):
    """A layer of experts, forward and backward, as a training run has it: [g, u] in 8 bits
    between the passes. The result and dx against float64: their norms' error is that of
    the bf16 roundings on the way (each below half a step of its value)."""
    from dequant_gemm_trellis_amd import synth

    tokens, top_k, n, hidden, inter = 50, 3, 7, 512, 256
    say("a layer of experts, forward and backward")
    g = np.random.default_rng(25)
    up, up_back = synth.Shape(1, 256, 12, 3, hidden, 2 * inter), synth.Shape(0, 256, 12, 3, 2 * inter, hidden)
    down, down_back = synth.Shape(0, 256, 12, 4, inter, hidden), synth.Shape(1, 256, 12, 4, hidden, inter)

    def coded(shape):
        codes = g.integers(0, 2 ** 32, (n, shape.rows, shape.words_per_row), dtype=np.uint32)
        scales = g.uniform(0.5, 1.5, (n, shape.rows)) * shape.in_features ** -0.5
        return (torch.from_numpy(codes.view(np.int32)).cuda(), torch.from_numpy(scales.astype(np.float32)).cuda(),
                torch.from_numpy(g.standard_normal(4096).astype(np.float32)).cuda())

    wu, wd = coded(up), coded(down)
    x = torch.from_numpy(g.standard_normal((tokens, hidden))).to(torch.bfloat16).cuda()
    dz = torch.from_numpy(g.standard_normal((tokens, hidden))).to(torch.bfloat16).cuda()
    ids = torch.from_numpy(np.stack([g.permutation(n)[:top_k] for _ in range(tokens)]).astype(np.int32)).cuda()
    w = torch.from_numpy(g.uniform(0.1, 1, (tokens, top_k)).astype(np.float32)).cuda()
    r = gpu_lib.route(ids, n)
    gu = gpu_lib.experts(gpu_lib.dispatch(x, r), r.offsets, *wu, up)
    h, kept = gpu_lib.swiglu(gu, keep=True)
    ys = gpu_lib.experts(h, r.offsets, *wd, down)
    z = gpu_lib.combine(ys, w, r)
    dys, dw = gpu_lib.combine_backward(dz, ys, w, r)
    dgu, again = gpu_lib.swiglu_backward(gpu_lib.experts(dys, r.offsets, *wd, down_back), kept, again=True)
    dx = gpu_lib.combine(gpu_lib.experts(dgu, r.offsets, *wu, up_back), None, r)
    # the same in float64 from the rows that each step had
    held = gpu_lib.restore(kept).reshape(gu.shape).double().cpu()
    near(h, ref.swiglu(gu.double().cpu()), forward_slack(gu.double().cpu()))
    near(again, ref.swiglu(held), forward_slack(held))
    want_z, want_dx = torch.zeros((tokens, hidden)).double(), torch.zeros((tokens, hidden)).double()
    place = r.position.cpu()
    for m in range(tokens):
        for k in range(top_k):
            e, s = int(ids[m, k]), int(place[m, k])
            we = gpu_lib.expand(wd[0][e], wd[1][e], wd[2], down).double().cpu()      # [inter, hidden]
            ue = gpu_lib.expand(wu[0][e], wu[1][e], wu[2], up).double().cpu()        # [2 inter, hidden]
            want_z[m] += float(w[m, k]) * (h[s].double().cpu() @ we)
            dh = float(w[m, k]) * (dz[m].double().cpu() @ we.T)
            want_dx[m] += ref.swiglu_backward(dh[None], held[s][None])[0] @ ue
    # dys, dh, dgu, the products' rows and dx are rounded: five half steps at most, and the
    # roundings of different values do not add up in the norm
    assert float((dx.double().cpu() - want_dx).norm() / want_dx.norm()) < 5 * HALF
    assert float((z.double().cpu() - want_z).norm() / want_z.norm()) < 2 * HALF
    assert bool(dw.isfinite().all())
