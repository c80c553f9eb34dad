"""An MLP's middle in a training step, every output against float64: adapters with scales
of their own on both projections, rows without an adapter, x and [g, u] kept in 8 bits, h
made again in the backward pass.

Bounds, value by value, with eps = 2^-24: a float32 sum of n terms, in any order, is off by
at most n eps times the sum of the terms' magnitudes; 16 eps more stand for a scale's product,
parts of a float32 value that are multiplied one by one, and the sums of a few partial sums.
A result is rounded to bf16 once, by at most 2^-8 of it.
"""
import numpy as np
import pytest
import torch

import kept_reference as ref
from helpers import say
from test_gpu_kept import backward_slack, forward_slack, near

pytestmark = pytest.mark.gpu

EPS, HALF = 2.0 ** -24, 2.0 ** -8


def within(name, got, want, size, terms, rounded=True):
    """Sums of `terms` terms whose magnitudes add up to `size`."""
    slack = (terms + 16) * EPS * size
    if rounded:
        slack = slack * (1 + HALF) + HALF * want.abs()
    err = (got.double().cpu() - want).abs()
    assert bool((err <= slack).all()), (name, float((err / (slack + 1e-300)).max()))


def inner(x, p, factor):
    """s_i * factor_i x per row, and the sums of magnitudes; zeros for rows without an adapter."""
    each = torch.einsum("mi,nri->mnr", x, factor)
    size = torch.einsum("mi,nri->mnr", x.abs(), factor.abs())
    return tuple((p["of"][:, :, None] * t).sum(1) for t in (each, size))


def check_forward(p, x, base, a, b, y, u):
    """y = base + s b^T u with u = a x."""
    want, size = inner(x, p, a)
    within("u", u, want, size, x.shape[1], rounded=False)
    su = p["s"] * u.double().cpu() * p["of"].sum(1, keepdim=True)
    spread = torch.einsum("mn,mr->mnr", p["of"], su)
    want = base + torch.einsum("mnr,nro->mo", spread, b)
    size = base.abs() + torch.einsum("mnr,nro->mo", spread.abs(), b.abs())
    within("y", y, want, size, a.shape[1] + 1)


def check_backward(p, dy, x, u, base, a, b, got):
    """dx = base + a^T v, da = sum v x^T, db = s sum u dy^T with v = s b dy."""
    v, size_v = (p["s"] * t for t in inner(dy, p, b))
    rows, rank, out = len(dy), a.shape[1], dy.shape[1]
    v_of, size_of = (torch.einsum("mn,mr->mnr", p["of"], t) for t in (v, size_v))
    dx, da, db = got
    within("dx", dx, base + torch.einsum("mnr,nri->mi", v_of, a),
           base.abs() + torch.einsum("mnr,nri->mi", size_of, a.abs()), out + rank + 1)
    within("da", da, torch.einsum("mnr,mi->nri", v_of, x), torch.einsum("mnr,mi->nri", size_of, x.abs()),
           out + rows)
    u_of = torch.einsum("mn,mr->mnr", p["of"], p["s"] * u.double().cpu())
    within("db", db, torch.einsum("mnr,mo->nro", u_of, dy), torch.einsum("mnr,mo->nro", u_of.abs(), dy.abs()),
           rows)


# rows, width of x, inter, width of y, rank, adapters
@pytest.mark.parametrize("rows,i,n,o,rank,count", [(300, 128, 200, 96, 8, 2), (41, 100, 77, 64, 5, 3),
                                                   (600, 64, 96, 136, 24, 3)])
def test_every_output_of_a_step(gpu_lib, rows, i, n, o, rank, count):
    say(f"a training step, {rows} rows {i} -> {n} -> {o}, rank {rank}, {count} adapters")
    g = np.random.default_rng([61, rows])
    draw = lambda *s: torch.from_numpy(g.standard_normal(s)).to(torch.bfloat16)  # noqa: E731
    ids = torch.from_numpy(g.integers(-1, count, rows).astype(np.int32))
    scales = torch.from_numpy(g.uniform(0.5, 2, count)).float()
    of = (ids[:, None] == torch.arange(count)).double()
    p = {"of": of, "s": (of @ scales.double())[:, None]}
    x, base, base2, dy, dx_base = draw(rows, i), draw(rows, 2 * n), draw(rows, o), draw(rows, o), draw(rows, i)
    a1, b1 = draw(count, rank, i) * i ** -0.5, draw(count, rank, 2 * n) * rank ** -0.5
    a2, b2 = draw(count, rank, n) * n ** -0.5, draw(count, rank, o) * rank ** -0.5
    c = {k: t.cuda() for k, t in dict(x=x, base=base, base2=base2, dy=dy, dx_base=dx_base, a1=a1, b1=b1, a2=a2,
                                      b2=b2, ids=ids, scales=scales).items()}
    first, second = (c["ids"], c["a1"], c["b1"], c["scales"]), (c["ids"], c["a2"], c["b2"], c["scales"])
    gu, u1 = gpu_lib.adapters(c["x"], *first, base=c["base"], keep_inner=True)
    h, kept = gpu_lib.swiglu(gu, keep=True)
    y, u2 = gpu_lib.adapters(h, *second, base=c["base2"], keep_inner=True)
    kept_x = gpu_lib.keep(c["x"])
    dh_base = draw(rows, n)  # the projection's share of dh
    # h is made again for the second pair's gradient, whose dh then goes through SwiGLU
    _, again = gpu_lib.swiglu_backward(dh_base.cuda(), kept, again=True)
    dh, da2, db2 = gpu_lib.adapters_backward(c["dy"], again, u2, *second, base=dh_base.cuda())
    dgu, _ = gpu_lib.swiglu_backward(dh, kept)
    dx, da1, db1 = gpu_lib.adapters_backward(dgu, kept_x, u1, *first, base=c["dx_base"])

    wide = lambda t: t.double().cpu()  # noqa: E731
    check_forward(p, wide(x), wide(base), wide(a1), wide(b1), gu, u1)
    near(h, ref.swiglu(wide(gu)), forward_slack(wide(gu)))
    check_forward(p, wide(h), wide(base2), wide(a2), wide(b2), y, u2)
    held = wide(gpu_lib.restore(kept)).reshape(rows, 2 * n)
    near(again, ref.swiglu(held), forward_slack(held))
    check_backward(p, wide(dy), wide(again), u2, wide(dh_base), wide(a2), wide(b2), (dh, da2, db2))
    near(dgu, ref.swiglu_backward(wide(dh), held), backward_slack(wide(dh), held))
    check_backward(p, wide(dgu), wide(gpu_lib.restore(kept_x)), u1, wide(dx_base), wide(a1), wide(b1),
                   (dx, da1, db1))
