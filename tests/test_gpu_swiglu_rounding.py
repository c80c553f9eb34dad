"""SwiGLU over many rows and its gradient round float32 values that are nearly exact.

With eps = 2^-24: exp(-g) is the square of exp2 of an exact argument, off by 2 eps (one
last bit) each time, times a factor 1 - x that stands for exp(-x), x < 2^-11.2 above g =
-87, off by x^2 / 2 < 1.5 eps; with the factor, the product and the sum rounded (3 eps) the
denominator is off by 8.5 eps. The reciprocal is off by 2 eps: the sigmoid s is off by at
most 10.5 eps of it, h = g s u and du = dh (g s) by 12.5 eps. In the gradient 1 - s is off by
10.5 eps s + eps (1 - s), which enters dg = dh s (1 + g (1 - s)) u with |g|, and the rest of
dg by 10.5 + 4 eps of it. All is below

    16 eps |h|,   16 eps |du|,   16 eps |dh s u| (|g| + |1 + g (1 - s)|),

and a result lies between the bf16 roundings of the ends of that interval, 2^-133 (the
smallest bf16) further on each side.
"""
import numpy as np
import pytest
import torch

import kept_reference as ref
from helpers import say

pytestmark = pytest.mark.gpu

EPS, LEAST = 2.0 ** -24, 2.0 ** -133


def between(got, want, slack):
    got, slack = got.float().cpu(), slack + LEAST
    lo, hi = ((want + d).float().to(torch.bfloat16).float() for d in (-slack, slack))
    off = (got < lo) | (got > hi)
    assert not bool(off.any()), f"{int(off.sum())} of {off.numel()} outside"


def inputs(seed, rows, inter):
    """g over the range where s is a normal float32, most of it where s is not nearly 1."""
    r = np.random.default_rng([seed, rows, inter])
    g = np.where(r.random((rows, inter)) < 0.5, r.uniform(-80, 30, (rows, inter)),
                 r.standard_normal((rows, inter)) * 2)
    gu = np.concatenate([g, r.standard_normal((rows, inter)) * 3], axis=1)
    return torch.from_numpy(gu).to(torch.bfloat16), torch.from_numpy(r.standard_normal((rows, inter))).to(torch.bfloat16)


@pytest.mark.parametrize("rows,inter", [(512, 2048), (701, 1003)])
def test_swiglu(gpu_lib, rows, inter):
    say(f"swiglu, rounding, {rows} x {inter}")
    gu, _ = inputs(41, rows, inter)
    want = ref.swiglu(gu.double())
    between(gpu_lib.swiglu(gu.cuda())[0], want, 16 * EPS * want.abs())


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("rows,inter", [(512, 2048), (701, 1003)])
def test_gradient(gpu_lib, rows, inter, kept):
    say(f"swiglu backward, rounding, {rows} x {inter}, kept {kept}")
    gu, dh = inputs(42, rows, inter)
    given = gu.cuda()
    if kept:
        given = gpu_lib.keep(gu.reshape(2 * rows, inter).cuda())
        gu = gpu_lib.restore(given).cpu().reshape(rows, 2 * inter)
    dgu, h = gpu_lib.swiglu_backward(dh.cuda(), given, again=True)
    gu, dh = gu.double(), dh.double()
    want = ref.swiglu_backward(dh, gu)
    g, u = gu.chunk(2, dim=1)
    s, left = torch.sigmoid(g), torch.sigmoid(-g)
    slack = torch.cat([(dh * s * u).abs() * (g.abs() + (1 + g * left).abs()), want[:, inter:].abs()], dim=1)
    between(dgu, want, 16 * EPS * slack)
    between(h, ref.swiglu(gu), 16 * EPS * ref.swiglu(gu).abs())
