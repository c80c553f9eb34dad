"""Low-rank adapters over many rows, whose rows are sorted into tiles of one
adapter's: arrays off 16 bytes, rows of odd lengths, no row with an adapter, and
adapters beside a shared projection of more rows than one prefill takes.

Few rows follow their own adapters without a sort; every test here asserts that
its call does not (the workspace's size tells). Inputs and exactness as in
test_gpu_adapters.py.
"""
import numpy as np
import pytest
import torch

from dequant_gemm_trellis_amd import synth
from helpers import say
from test_gpu_adapters import Problem, same

pytestmark = pytest.mark.gpu


def sorted_tiles(T, p, backward):
    """Whether the call takes the sorted tiles: its workspace is not that of few rows,
    the inner products' column splits of 512 and, for the gradient, their sums."""
    f = T.AdapterSet(0, 0, 0, p.count, p.rank, p.i, p.o)
    one = p.rows * p.rank
    splits = -(-(p.o if backward else p.i) // 512)
    few = 4 * ((splits * one + 3) // 4 * 4 + one) if backward else 4 * splits * one
    return T.adapters_workspace_bytes(f, p.rows, backward) not in (0, few)


def tiled(T, p):
    assert sorted_tiles(T, p, False) and sorted_tiles(T, p, True)
    return p


def moved(t):
    """The same values, 2 bytes off a 16-byte boundary."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


# rows, in, out, rank, count: each number of 16-rank operands (1, 2, 4, 8) with
# row lengths off 8 on both sides, on one side, and one value past a step
ODD = [(700, 263, 391, 8, 3), (700, 391, 264, 16, 4), (600, 264, 391, 24, 3), (601, 263, 395, 32, 2),
       (520, 777, 1031, 24, 5), (600, 257, 519, 40, 3), (515, 391, 264, 64, 2), (520, 263, 397, 128, 3),
       (530, 1031, 264, 100, 2), (2100, 33, 1031, 24, 2), (600, 5, 3, 24, 2)]


@pytest.mark.parametrize("rows,i,o,rank,count", ODD)
def test_odd_lengths(gpu_lib, rows, i, o, rank, count):
    say(f"adapters in tiles, {rows} x {i} -> {o}, rank {rank}, {count} adapters")
    p = tiled(gpu_lib, Problem(41, rows, i, o, rank, count))
    d = p.cuda()
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=d["base_y"],
                            keep_inner=True)
    want_y, want_u = p.forward()
    assert torch.equal(u.double().cpu(), want_u) and same(y, want_y)
    grads = gpu_lib.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                      base=d["base_x"])
    for got, want in zip(grads, p.backward(want_u)):
        assert same(got, want)


@pytest.mark.parametrize("rank", [16, 24, 64, 128])
def test_rows_off_16_bytes(gpu_lib, rank):
    """Row lengths that are multiples of 8 in arrays that are not 16-byte aligned."""
    say(f"adapters in tiles off 16 bytes, rank {rank}")
    p = tiled(gpu_lib, Problem(42, 700, 256, 264, rank, 3))
    d = p.cuda()
    want, want_u = p.forward()
    y = moved(torch.zeros_like(d["base_y"]))
    gpu_lib.adapters(moved(d["x"]), d["ids"], moved(d["a"]), moved(d["b"]), d["scales"],
                     base=moved(d["base_y"]), y=y)
    assert same(y, want)
    dx, da, db = (moved(torch.zeros_like(d[n])) for n in ("x", "a", "b"))
    gpu_lib.adapters_backward(moved(d["dy"]), moved(d["x"]), want_u.float().cuda(), d["ids"],
                              moved(d["a"]), moved(d["b"]), d["scales"], base=moved(d["base_x"]),
                              dx=dx, da=da, db=db)
    for got, want in zip((dx, da, db), p.backward(want_u)):
        assert same(got, want)


@pytest.mark.parametrize("side", ["in", "out"])
def test_one_side_off_16_bytes(gpu_lib, side):
    """Only the arrays with rows of one length are off 16 bytes."""
    say(f"adapters in tiles, side {side} off 16 bytes")
    p = tiled(gpu_lib, Problem(43, 700, 256, 264, 24, 3))
    d = p.cuda()
    for n in ("x", "a", "base_x") if side == "in" else ("dy", "b", "base_y"):
        d[n] = moved(d[n])
    want, want_u = p.forward()
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=d["base_y"],
                            keep_inner=True)
    assert same(y, want) and torch.equal(u.double().cpu(), want_u)
    grads = gpu_lib.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                      base=d["base_x"])
    for got, want in zip(grads, p.backward(want_u)):
        assert same(got, want)


@pytest.mark.parametrize("kind", ["none", "one"])
@pytest.mark.parametrize("i,o,rank", [(256, 320, 16), (263, 391, 24), (256, 320, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_no_adapter_or_one(gpu_lib, i, o, rank, kind, in_place):
    say(f"adapters in tiles, {i} -> {o}, rank {rank}, {kind}, in place {in_place}")
    p = tiled(gpu_lib, Problem(44, 700, i, o, rank, 4, kind))
    d = p.cuda()
    y, dx = (d["base_y"].clone(), d["base_x"].clone()) if in_place else (None, None)
    base_y, base_x = (y, dx) if in_place else (d["base_y"], d["base_x"])
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=base_y, y=y,
                            keep_inner=True)
    want_y, want_u = p.forward()
    assert same(y, want_y) and torch.equal(u.double().cpu(), want_u)
    grads = gpu_lib.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                      base=base_x, dx=dx)
    for got, want in zip(grads, p.backward(want_u)):
        assert same(got, want)


@pytest.mark.parametrize("M", [33, 700])
def test_beside_a_projection_of_many_rows(gpu_lib, M):
    """More rows than one prefill takes: the shared projection is the experts'
    product with a single expert, whose rows are all rows; its gradient the same on
    the other axis. Integers: each of the two roundings is the exact value's."""
    import oracle

    T = gpu_lib
    say(f"a projection of {M} rows and adapters")
    shape, flipped = synth.Shape(1, 256, 12, 3, 512, 256), synth.Shape(0, 256, 12, 3, 256, 512)
    w = synth.make_problem(shape, 1, synth.CONFIG_IDS["test"], proj=32)
    lut, scales = synth.integer_lut(), np.where(np.arange(256) % 2, 0.5, 1.0).astype(np.float32)
    codes = torch.from_numpy(w.codes.view(np.int32)).cuda().reshape(1, 256, -1)
    dev_scales = torch.from_numpy(scales).cuda().reshape(1, 256)
    dev_lut = T.lut_upload(lut)
    p = Problem(45, M, 512, 256, 16, 3)
    assert sorted_tiles(T, p, False) == (M == 700)
    d = p.cuda()
    whole = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    base = T.experts(d["x"], whole, codes, dev_scales, dev_lut, shape)
    y, u = T.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=base, y=base, keep_inner=True)
    weights = torch.from_numpy(oracle.expand(w.codes, scales, lut, 1, 256, 12, 3, 512, 256)
                               .view(np.int16)).view(torch.bfloat16).double().reshape(256, 512)
    p.base_y = (p.x.double() @ weights.T).to(torch.bfloat16)
    want, want_u = p.forward()
    assert torch.equal(u.double().cpu(), want_u) and same(y, want)
    dx = T.experts(d["dy"], whole, codes, dev_scales, dev_lut, flipped)
    dx, da, db = T.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                     base=dx, dx=dx)
    p.base_x = (p.dy.double() @ weights).to(torch.bfloat16)
    for got, ref in zip((dx, da, db), p.backward(want_u)):
        assert same(got, ref)


@pytest.mark.parametrize("i,o,rank", [(512, 264, 16), (511, 391, 24), (512, 264, 64)])
def test_inner_values_keep_their_mantissa(gpu_lib, i, o, rank):
    """Inner values of up to 20 bits and outputs below 2^24: exact in float32, so
    equal to the rounded exact value. (With u and g cut to 16 bits, hundreds of
    these outputs round to another bf16 value.)"""
    say(f"adapters in tiles, long inner values, {i} -> {o}, rank {rank}")
    p = tiled(gpu_lib, Problem(46, 600, i, o, rank, 8))
    g = np.random.default_rng(46)

    def wide(t):
        v = g.integers(-127, 128, tuple(t.shape)).astype(np.float32)
        return torch.from_numpy(v).to(torch.bfloat16)

    small = {n: getattr(p, n) for n in ("x", "a", "dy", "b")}
    most = 2.0 ** 24

    p.x, p.a = wide(p.x), wide(p.a)  # long u, short b: the forward pass and db
    d = p.cuda()
    want, want_u = p.forward()
    assert float(want_u.abs().max()) >= 2 ** 17
    assert float((want_u.abs().sum(1)).max()) * 2 < most
    y, u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=d["base_y"],
                            keep_inner=True)
    assert torch.equal(u.double().cpu(), want_u) and same(y, want)
    p.x, p.a = small["x"], small["a"]
    d = p.cuda()
    db = gpu_lib.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"])[2]
    assert max(float(want_u[p.ids == n].abs().sum(0).max()) for n in range(8)) * 2 < most
    assert same(db, p.backward(want_u)[2])

    p.dy, p.b = wide(p.dy), wide(p.b)  # long g, short a and x: dx and da
    d = p.cuda()
    u = torch.zeros((600, rank), device="cuda")
    dx, da, _ = gpu_lib.adapters_backward(d["dy"], d["x"], u, d["ids"], d["a"], d["b"], d["scales"],
                                          base=d["base_x"])
    for n in range(8):
        v = (float(p.scales[n]) * (p.dy[p.ids == n].double() @ p.b[n].double().T)).abs()
        assert float(v.max()) >= 2 ** 17 and float(v.sum(0).max()) < most and float(v.sum(1).max()) < most
    want_dx, want_da, _ = p.backward(u.double().cpu())
    assert same(dx, want_dx) and same(da, want_da)


@pytest.mark.parametrize("rows", [40, 700])
@pytest.mark.parametrize("rank", [16, 24, 64])
def test_infinities_keep_their_sign(gpu_lib, rows, rank):
    """An infinite value of a factor or of a wide row: the outputs that it enters are
    the formula's infinities, and no other changes. Over many rows an output is NaN
    where the second or the third of the parts that its inner value is cut into (the
    upper 8 bits of what is left, each) is 0: known here of u, not of g."""
    say(f"adapters with infinities, {rows} rows, rank {rank}")
    p = Problem(47, rows, 264, 328, rank, 3, "runs", integers=False)
    many = rows == 700
    assert sorted_tiles(gpu_lib, p, False) == sorted_tiles(gpu_lib, p, True) == many
    d = p.cuda()
    u = gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], keep_inner=True)[1].cpu()
    m = int((p.ids == 1).nonzero()[0])  # a row of adapter 1

    def cut(v):
        return (v.contiguous().view(torch.int32) & -65536).view(torch.float32)

    def run(which):
        d = p.cuda()
        if which == "y":
            return gpu_lib.adapters(d["x"], d["ids"], d["a"], d["b"], d["scales"], base=d["base_y"])[0].cpu()
        grads = gpu_lib.adapters_backward(d["dy"], d["x"], u.cuda(), d["ids"], d["a"], d["b"],
                                          d["scales"], base=d["base_x"])
        return grads[("dx", "da", "db").index(which)].cpu()

    def check(before, got, hit, inner, sign):
        """got[hit] are infinities of `sign` times the signs of `inner` (float32: NaN
        where a part of it is 0; float64: some are infinities), the rest as before."""
        assert torch.equal(got[~hit], before[~hit])
        value, want = got[hit].float(), sign * inner.sign().float()
        assert not value.isfinite().any()
        fine = ~value.isnan()
        assert torch.equal(value[fine].sign(), want[fine]) and bool(fine.any())
        if not many:
            assert bool(fine.all())
        elif inner.dtype is torch.float32:
            rest = inner - cut(inner)
            assert torch.equal(fine, (rest != 0) & (rest - cut(rest) != 0))

    def set_one(name, at, which, hit, inner):
        t = getattr(p, name)
        before, kept = run(which), t[at].clone()
        for sign in (1, -1):
            t[at] = sign * float("inf")
            check(before, run(which), hit, inner, sign)
        t[at] = kept

    r = rank // 2
    one = p.ids == 1
    hit = torch.zeros((rows, 328), dtype=torch.bool)
    hit[one, 7] = True
    set_one("b", (1, r, 7), "y", hit, u[one, r])
    g = p.dy.double() @ p.b[1].double().T
    hit = torch.zeros((rows, 264), dtype=torch.bool)
    hit[one, 9] = True
    set_one("a", (1, r, 9), "dx", hit, g[one, r])
    hit = torch.zeros((3, rank, 264), dtype=torch.bool)
    hit[1, :, 11] = True
    set_one("x", (m, 11), "da", hit, g[m])
    hit = torch.zeros((3, rank, 328), dtype=torch.bool)
    hit[1, :, 3] = True
    set_one("dy", (m, 3), "db", hit, u[m])
