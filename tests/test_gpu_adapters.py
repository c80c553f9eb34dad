"""Low-rank adapters of many requests (trellis_adapters and its gradient)
against float64 references on the host.

Two kinds of inputs:
- small integers with scales that are powers of two: every product and sum of
  the definition is exact in float32 (magnitudes below 2^24) and every inner
  value fits the 16 bits of its two bf16 parts, so outputs must equal the exact
  value rounded to bf16, bit for bit;
- normal values: outputs within the library's floored 1e-2 relative error gate
  (bf16 half steps are 2^-8 = 4e-3; the float32 sums add less than 1e-4 at these
  lengths, the two-part inner values 2^-16).
"""
import numpy as np
import pytest
import torch

from dequant_gemm_trellis_amd import synth
from helpers import TOL, Dev, gate, say

pytestmark = pytest.mark.gpu


def some_ids(g, rows, count, kind):
    if kind == "runs":      # adjacent rows share an adapter
        ids = np.sort(g.integers(-1, count, rows))
    elif kind == "none":
        ids = np.full(rows, -1)
    elif kind == "one":     # every row the last adapter's
        ids = np.full(rows, count - 1)
    else:                   # mixed, some outside the adapters
        ids = g.choice(np.array(list(range(count)) + [-1, count, -2 ** 31, 2 ** 31 - 1]), rows)
    return torch.from_numpy(ids.astype(np.int32))


class Problem:
    """Host tensors of one call: bf16 x, a, b, dy, base_y, base_x; ids; scales."""

    def __init__(self, seed, rows, i, o, rank, count, kind="mixed", integers=True):
        g = np.random.default_rng([seed, rows, i, o, rank, count])
        self.rows, self.i, self.o, self.rank, self.count = rows, i, o, rank, count
        self.ids = some_ids(g, rows, count, kind)

        def draw(*shape, std=1.0):
            v = g.integers(-1, 2, shape) if integers else g.standard_normal(shape) * std
            return torch.from_numpy(np.asarray(v, dtype=np.float32)).to(torch.bfloat16)

        self.x, self.dy = draw(rows, i), draw(rows, o)
        self.base_y, self.base_x = draw(rows, o), draw(rows, i)
        self.a, self.b = draw(count, rank, i, std=i ** -0.5), draw(count, rank, o, std=rank ** -0.5)
        self.scales = torch.from_numpy(g.choice([0.5, 1.0, 2.0], count).astype(np.float32))

    def forward(self, base=True):
        """(y, u) in float64."""
        x, a, b = self.x.double(), self.a.double(), self.b.double()
        y = self.base_y.double() if base else torch.zeros((self.rows, self.o), dtype=torch.float64)
        u = torch.zeros((self.rows, self.rank), dtype=torch.float64)
        for n in range(self.count):
            m = (self.ids == n).nonzero()[:, 0]
            if len(m):
                u[m] = x[m] @ a[n].T
                y[m] += float(self.scales[n]) * (u[m] @ b[n])
        return y, u

    def backward(self, u, base=True):
        """(dx, da, db) in float64."""
        x, dy, a, b = (t.double() for t in (self.x, self.dy, self.a, self.b))
        dx = self.base_x.double() if base else torch.zeros((self.rows, self.i), dtype=torch.float64)
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        for n in range(self.count):
            m = (self.ids == n).nonzero()[:, 0]
            if len(m):
                s = float(self.scales[n])
                v = s * (dy[m] @ b[n].T)
                dx[m] += v @ a[n]
                da[n], db[n] = v.T @ x[m], s * (u[m].double().T @ dy[m])
        return dx, da, db

    def cuda(self):
        return {n: getattr(self, n).cuda()
                for n in ("x", "dy", "base_y", "base_x", "a", "b", "scales", "ids")}


def same(got, want):
    return torch.equal(got.cpu(), want.to(torch.bfloat16))


def near(got, want):
    """Within the gate; an all-zero reference has no scale and must be met exactly."""
    if not want.any():
        return not got.any()
    return gate(got.double().cpu().numpy(), want.numpy()) <= TOL


# rows, in, out, rank, count: one row to several tiles and segments; lengths
# that are multiples of 8 and odd ones; ranks around the 16-rank operands
SIZES = [(1, 256, 16, 1, 1), (1, 512, 4111, 16, 8), (2, 300, 520, 13, 3), (31, 1024, 300, 8, 40),
         (64, 2048, 264, 16, 5), (65, 256, 256, 16, 1), (66, 512, 4111, 24, 3), (129, 7, 9, 5, 2),
         (200, 777, 1000, 33, 4), (500, 264, 640, 64, 70), (130, 512, 384, 128, 3),
         (97, 1, 1, 17, 1024), (256, 264, 392, 16, 6), (257, 264, 392, 16, 6),
         (512, 64, 72, 8, 9), (513, 64, 72, 8, 9), (8, 512, 1032, 16, 3), (9, 512, 1032, 16, 3),
         (200, 520, 1030, 16, 3), (201, 520, 1030, 16, 3), (256, 72, 515, 12, 2), (25, 264, 600, 128, 3),
         (1025, 136, 520, 16, 1), (2500, 256, 192, 32, 2),
         (3000, 64, 133, 8, 5)]


@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("rows,i,o,rank,count", SIZES)
def test_forward_exact(gpu_lib, rows, i, o, rank, count, kind):
    say(f"adapters {rows} x {i} -> {o}, rank {rank}, {count} adapters, {kind}")
    p = Problem(1, rows, i, o, rank, count, kind)
    d = p.cuda()
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=d["base_y"],
                            keep_inner=True)
    want_y, want_u = p.forward()
    assert torch.equal(u.double().cpu(), want_u)
    assert same(y, want_y)


@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("rows,i,o,rank,count", SIZES)
def test_backward_exact(gpu_lib, rows, i, o, rank, count, kind):
    say(f"adapters backward {rows} x {i} -> {o}, rank {rank}, {count} adapters, {kind}")
    p = Problem(2, rows, i, o, rank, count, kind)
    d = p.cuda()
    _, u = p.forward()
    dx, da, db = gpu_lib.adapters_backward(d["dy"], d["x"], u.float().cuda(), d["ids"], d["a"],
                                           d["b"], d["scales"], base=d["base_x"])
    want_dx, want_da, want_db = p.backward(u)
    assert same(dx, want_dx)
    assert same(da, want_da)
    assert same(db, want_db)


@pytest.mark.parametrize("kind", ["none", "one"])
@pytest.mark.parametrize("rows", [5, 150])
def test_no_adapter_or_one(gpu_lib, rows, kind):
    say(f"adapters, {rows} rows, {kind}")
    p = Problem(3, rows, 256, 320, 16, 4, kind)
    d = p.cuda()
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=d["base_y"],
                            keep_inner=True)
    want_y, want_u = p.forward()
    assert same(y, want_y) and torch.equal(u.double().cpu(), want_u)
    grads = gpu_lib.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                      base=d["base_x"])
    for got, want in zip(grads, p.backward(want_u)):
        assert same(got, want)


@pytest.mark.parametrize("rows", [9, 300])
def test_in_place_and_without_base(gpu_lib, rows):
    say(f"adapters in place, {rows} rows")
    p = Problem(4, rows, 512, 264, 16, 3)
    d = p.cuda()
    args = (d["x"], d["ids"], d["a"], d["b"], d["scales"])
    want, want_u = p.forward()
    assert same(gpu_lib.adapters(*args)[0], p.forward(base=False)[0])
    y = d["base_y"].clone()
    got, none = gpu_lib.adapters(*args, base=y, y=y)
    assert got is y and none is None and same(y, want)
    u = want_u.float().cuda()
    bargs = (d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"])
    assert same(gpu_lib.adapters_backward(*bargs)[0], p.backward(want_u, base=False)[0])
    dx = d["base_x"].clone()
    got = gpu_lib.adapters_backward(*bargs, base=dx, dx=dx)
    assert got[0] is dx and same(dx, p.backward(want_u)[0])


def test_no_rows(gpu_lib):
    say("adapters without rows")
    p = Problem(5, 0, 256, 264, 16, 3)
    d = p.cuda()
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], keep_inner=True)
    assert tuple(y.shape) == (0, 264) and tuple(u.shape) == (0, 16)
    da = torch.full_like(d["a"], 7.0)
    db = torch.full_like(d["b"], 7.0)
    dx, _, _ = gpu_lib.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                         da=da, db=db)
    assert tuple(dx.shape) == (0, 256) and not da.any() and not db.any()


@pytest.mark.parametrize("rows", [20, 200])
def test_rows_off_16_bytes(gpu_lib, rows):
    """Row lengths that are multiples of 8 in arrays that are not 16-byte aligned."""
    say(f"adapters off 16 bytes, {rows} rows")
    p = Problem(6, rows, 256, 264, 16, 3)
    d = p.cuda()

    def moved(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    want, want_u = p.forward()
    y = moved(torch.zeros_like(d["base_y"]))
    gpu_lib.adapters(moved(d["x"]), d["ids"], moved(d["a"]), moved(d["b"]), d["scales"],
                     base=moved(d["base_y"]), y=y)
    assert same(y, want)
    grads = gpu_lib.adapters_backward(moved(d["dy"]), moved(d["x"]), want_u.float().cuda(), d["ids"],
                                      moved(d["a"]), moved(d["b"]), d["scales"],
                                      base=moved(d["base_x"]), dx=moved(torch.zeros_like(d["x"])))
    for got, want in zip(grads, p.backward(want_u)):
        assert same(got, want)


@pytest.mark.parametrize("rows", [40, 700])
def test_not_finite_stays_where_it_is(gpu_lib, rows):
    """A row's NaN reaches its own outputs and its adapter's gradients only; rows
    without an adapter and adapters without rows reach nothing."""
    say(f"adapters with NaN and infinity, {rows} rows")
    p = Problem(7, rows, 264, 328, 24, 5)
    p.ids[p.ids == 4] = 3          # adapter 4 has no rows
    p.ids[0], p.ids[1] = 2, -1
    p.x[0, 5], p.dy[0, 3] = float("nan"), float("inf")
    p.x[1], p.dy[1] = float("nan"), float("nan")
    p.a[4], p.b[4] = float("inf"), float("nan")
    d = p.cuda()
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=d["base_y"],
                            keep_inner=True)
    want, want_u = p.forward()
    clean = torch.ones(rows, dtype=torch.bool)
    clean[0] = False
    assert same(y[clean.cuda()], want[clean]) and y[0].isnan().all()
    assert torch.equal(u.double().cpu()[clean], want_u[clean]) and u[0].isnan().all()
    dx, da, db = gpu_lib.adapters_backward(d["dy"], d["x"], want_u.float().cuda(), d["ids"], d["a"],
                                           d["b"], d["scales"], base=d["base_x"])
    want_dx, want_da, want_db = p.backward(want_u)
    assert same(dx[clean.cuda()], want_dx[clean])
    others = [0, 1, 3, 4]
    assert same(da[others], want_da[others]) and same(db[others], want_db[others])
    assert da[2].isnan().any() and db[2].isnan().any()


@pytest.mark.parametrize("rows,i,o,rank,count", [(1, 5120, 17408, 16, 8), (32, 17408, 5120, 16, 32),
                                                 (64, 5120, 4111, 64, 9), (333, 5120, 2048, 16, 3),
                                                 (1500, 2048, 5000, 40, 6)])
def test_normal_values(gpu_lib, rows, i, o, rank, count):
    say(f"adapters, normal values, {rows} x {i} -> {o}, rank {rank}")
    p = Problem(8, rows, i, o, rank, count, integers=False)
    d = p.cuda()
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=d["base_y"],
                            keep_inner=True)
    want, want_u = p.forward()
    assert near(y, want)
    # float32 sums of `in` products: 2^-24 of their magnitudes, per addition
    size = p.x.double().abs().sum(1).max() * p.a.double().abs().max()
    assert float((u.double().cpu() - want_u).abs().max()) <= i * 2.0 ** -24 * float(size)
    grads = gpu_lib.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                      base=d["base_x"])
    for got, ref in zip(grads, p.backward(u.cpu())):
        assert near(got, ref)


def test_gradient_against_differences(gpu_lib):
    """y is linear in x, in a and in b: the change of <dy, y> over a step of one
    of them is the step's product with its gradient, exactly for integers whose
    outputs stay below 2^8 (exact in bf16)."""
    say("adapters gradient against differences")
    T = gpu_lib
    p = Problem(9, 70, 24, 20, 3, 3, "mixed")
    g = np.random.default_rng(9)
    for t in (p.x, p.a, p.b, p.dy):  # three quarters zeros: small sums
        t[torch.from_numpy(g.random(t.shape) < 0.75)] = 0
    d = p.cuda()

    def value(**other):
        v = d | other
        y, _ = T.adapters(v["x"], v["ids"], v["a"], v["b"], v["scales"])
        assert float(y.abs().max()) <= 128
        return float((d["dy"].double() * y.double()).sum())

    _, u = T.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], keep_inner=True)
    dx, da, db = T.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"])
    for name, grad in (("x", dx), ("a", da), ("b", db)):
        assert float(grad.abs().max()) <= 128
        step = torch.from_numpy(g.integers(-1, 2, grad.shape).astype(np.float32)).cuda()
        moved = (d[name].float() + step).to(torch.bfloat16)
        assert value(**{name: moved}) - value() == float((step.double() * grad.double()).sum())


@pytest.mark.parametrize("rows", [33, 900])
def test_repeats(gpu_lib, rows):
    say(f"adapters repeated, {rows} rows")
    d = Problem(10, rows, 1024, 1000, 16, 7, integers=False).cuda()
    args = (d["x"], d["ids"], d["a"], d["b"], d["scales"])
    y, u = gpu_lib.adapters(*args, base=d["base_y"], keep_inner=True)
    grads = gpu_lib.adapters_backward(d["dy"], d["x"], u, *args[1:], base=d["base_x"])
    for _ in range(3):
        y2, u2 = gpu_lib.adapters(*args, base=d["base_y"], keep_inner=True)
        assert torch.equal(y, y2) and torch.equal(u, u2)
        for p, q in zip(grads, gpu_lib.adapters_backward(d["dy"], d["x"], u, *args[1:],
                                                         base=d["base_x"])):
            assert torch.equal(p, q)


@pytest.mark.parametrize("rows", [24, 1100])
def test_captured_and_replayed(gpu_lib, rows):
    """Forward and backward in one graph, replayed with other rows and ids
    between eager calls; every replay against eager."""
    say(f"adapters captured, {rows} rows")
    T = gpu_lib
    sets = [Problem(seed, rows, 512, 264, 16, 6, kind, integers=False).cuda()
            for seed, kind in ((11, "mixed"), (12, "runs"), (13, "one"))]
    d = {n: t.clone() for n, t in sets[0].items()}

    def chain(v):
        y, u = T.adapters(v["x"], v["ids"], v["a"], v["b"], v["scales"], base=v["base_y"],
                          keep_inner=True)
        return (y, u) + T.adapters_backward(v["dy"], v["x"], u, v["ids"], v["a"], v["b"],
                                            v["scales"], base=v["base_x"])

    chain(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = chain(d)
    for n in (1, 2, 0, 2, 2):
        for name, t in d.items():
            t.copy_(sets[n][name])
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(kept, chain(sets[n])):
            assert torch.equal(got, want)


def test_another_stream(gpu_lib):
    say("adapters on another stream")
    p = Problem(14, 300, 512, 264, 16, 6)
    d = p.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=d["base_y"],
                            keep_inner=True, stream=side)
    grads = gpu_lib.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                      base=d["base_x"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want, want_u = p.forward()
    assert same(y, want)
    for got, ref in zip(grads, p.backward(want_u)):
        assert same(got, ref)


def test_offsets_past_32_bits(gpu_lib):
    """More than 2^31 outputs: the last rows equal those of a short call (exact
    integers, so both sums give the same bits)."""
    say("adapters past 2^31 values")
    T, rows, tail = gpu_lib, 131072, 300
    p = Problem(16, tail, 64, 17408, 8, 2, "one")
    d = p.cuda()
    assert rows * 17408 > 2 ** 31

    def long(t):
        return torch.cat([t.new_zeros((rows - tail, t.shape[1])), t])

    ids = torch.cat([torch.zeros(rows - tail, dtype=torch.int32, device="cuda"), d["ids"]])
    y, u = T.adapters(long(d["x"]), ids, d["a"], d["b"], d["scales"], base=long(d["base_y"]),
                      keep_inner=True)
    want, want_u = p.forward()
    assert same(y[-tail:], want) and not y[:-tail].any()
    del y
    dx, da, db = T.adapters_backward(long(d["dy"]), long(d["x"]), u, ids, d["a"], d["b"],
                                     d["scales"], base=long(d["base_x"]))
    for got, ref in zip((dx[-tail:], da, db), p.backward(want_u)):
        assert same(got, ref)


@pytest.mark.parametrize("M", [1, 20])
def test_beside_the_projection(gpu_lib, M):
    """As it is used: the coded projection of all rows, each row's adapter added
    in place, and the gradient through both (the transposed product is the same
    codes on the other axis)."""
    import oracle

    T = gpu_lib
    say(f"projection and adapters, {M} rows")
    shape = synth.Shape(1, 256, 12, 3, 1024, 768)
    flipped = synth.Shape(0, 256, 12, 3, 768, 1024)
    w = synth.make_problem(shape, M, synth.CONFIG_IDS["test"], proj=31)
    dev = Dev(w, T)
    p = Problem(15, M, 1024, 768, 16, 3, integers=False)
    p.x = torch.from_numpy(w.x.view(np.int16)).view(torch.bfloat16).reshape(M, 1024)
    d = p.cuda()
    base = T.prefill(d["x"], dev.codes, dev.scales, dev.lut, shape)
    y, u = T.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=base, keep_inner=True)
    weights = torch.from_numpy(oracle.expand(w.codes, w.scales, w.lut, 1, 256, 12, 3, 1024, 768)
                               .view(np.int16)).view(torch.bfloat16).double().reshape(768, 1024)

    def both(got, x, w, added):
        """The shared product is rounded to bf16 (2^-8 of it), then the sum is (2^-8
        of the sum of the rounded product and the adapter): where the two cancel,
        the first rounding is large beside the result, so errors are held to the
        two values, with the product's float32 sum (2^-24 of the magnitudes, per
        addition) and the adapter's (2^-10 of its own size, with its two-part
        inner values) on top."""
        product = x.double() @ w
        sums = x.shape[1] * 2.0 ** -24 * (x.double().abs() @ w.abs())
        first = 2.0 ** -8 * (product.abs() + sums) + sums
        inner = 2.0 ** -10 * added.abs().max()
        total = product + added
        assert bool(((got.double().cpu() - total).abs() <=
                     first + inner + 2.0 ** -8 * (total.abs() + first + inner)).all())

    both(y, p.x, weights.T, p.forward(base=False)[0])
    dx0 = T.prefill(d["dy"], dev.codes, dev.scales, dev.lut, flipped)
    dx, da, db = T.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                     base=dx0, dx=dx0)
    ref_dx, ref_da, ref_db = p.backward(u.cpu(), base=False)
    both(dx, p.dy, weights, ref_dx)
    assert near(da, ref_da) and near(db, ref_db)


def test_long_runs_of_some_of_many_adapters(gpu_lib):
    """Adapters of several 1024-row segments among many of few rows or none, past
    the 64 adapters that a wave looks at together."""
    say("adapters, 2100 rows of one of 130")
    p = Problem(18, 5000, 40, 72, 8, 130)
    ids = np.random.default_rng(18).integers(-1, 130, 5000).astype(np.int32)
    ids[::5][:900] = 3
    ids[1:4600:2] = 70
    ids[2::4][:1150] = 129
    p.ids = torch.from_numpy(ids)
    d = p.cuda()
    _, u = p.forward()
    grads = gpu_lib.adapters_backward(d["dy"], d["x"], u.float().cuda(), d["ids"], d["a"], d["b"],
                                      d["scales"], base=d["base_x"])
    for got, want in zip(grads, p.backward(u)):
        assert same(got, want)
