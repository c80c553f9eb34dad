"""What holds h between the two products of trellis_experts_mlp: two bf16 parts, 16 bits
of its mantissa, whatever the number of tokens.

A token has one input that is not zero, so that g and u are exact (products of two bf16
values, and zeros). Then, value by value, with eps = 2^-24: h's float32 work (exp,
division, three products) is off by 16 eps of it; its upper part is cut off after 8 bits,
so what is left is below 2^-7 of h, and its rounding moves h by at most 2^-8 of that,
2^-15 of h; out has all that times |Wd|, sums of 2 inter products, the sums of up to 40
parts, and half a bf16 step, 2^-8 of it.
"""
import pytest
import torch

from helpers import say
from test_gpu_layer import EPS, HALF, Layer

pytestmark = pytest.mark.gpu

PARTS = 2.0 ** -15


def few_inputs(seed, *size):
    p = Layer(seed, *size)
    at = torch.arange(len(p.ids)) * 37 % p.hidden
    p.x[:, :] = 0
    p.x[torch.arange(len(p.ids)), at] = torch.linspace(-9, 8, len(p.ids)).to(torch.bfloat16)
    return p


def want(p):
    """(out, bound) in float64."""
    out = torch.zeros((len(p.ids), p.hidden), dtype=torch.float64)
    bound, sums = torch.zeros_like(out), torch.zeros_like(out)
    for e in range(p.experts):
        mine = p.ids == e
        m = mine.any(1).nonzero()[:, 0]
        if not len(m):
            continue
        w = torch.where(mine, p.w, torch.zeros(())).double().sum(1)[m][:, None]
        wu, wd = p.weights(p.up, e), p.weights(p.down, e)
        g, u = (p.x[m].double() @ wu.T).chunk(2, dim=1)
        h = w * g * torch.sigmoid(g) * u
        out[m] += h @ wd.T
        sums[m] += h.abs() @ wd.abs().T
    return out, (PARTS + (16 + 2 * p.inter + 40) * EPS) * sums * (1 + HALF) + HALF * out.abs()


# top_k, experts, hidden, inter, k, k of down, axis of down
SIZES = [(2, 5, 512, 150, 2, 2, 0), (2, 5, 512, 31, 3, 3, 0), (2, 5, 512, 41, 4, 4, 0),
         (1, 6, 512, 256, 2, 2, 1), (1, 6, 768, 256, 3, 3, 1), (1, 1, 256, 256, 4, 4, 1),
         # more units of 8 columns than 256 compute units have waves
         (1, 70, 256, 256, 2, 4, 1), (1, 70, 256, 241, 3, 2, 0)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("tokens", [1, 8, 9, 16, 17, 32])
def test_as_precise_in_any_batch(gpu_lib, tokens, size):
    say(f"layer, parts of h, {tokens} tokens {size}")
    p = few_inputs(31, tokens, *size)
    got = gpu_lib.experts_mlp(*p.cuda()).double().cpu()
    out, bound = want(p)
    assert bool(((got - out).abs() <= bound).all()), float(((got - out).abs() / bound).max())


@pytest.mark.parametrize("axis,inter", [(0, 300), (0, 39), (1, 256)])
def test_a_token_alone_and_in_a_batch(gpu_lib, axis, inter):
    """Both are within the same bound, so no further apart than two of it."""
    say(f"layer, alone and in a batch, axis {axis}")
    p = few_inputs(32, 32, 2, 6, 512, inter, 3, 3, axis)
    x, ids, w, *rest = p.cuda()
    _, bound = want(p)
    all32 = gpu_lib.experts_mlp(x, ids, w, *rest).double().cpu()
    for n in (1, 5, 12, 23):
        few = gpu_lib.experts_mlp(x[:n], ids[:n], w[:n], *rest).double().cpu()
        assert bool(((few - all32[:n]).abs() <= 2 * bound[:n]).all())


TINY = 2.0 ** -132  # what two parts of at least 2^-133, the smallest bf16, may be off


@pytest.mark.parametrize("exponent", [-60, -104, -110, -113, -116, -119, -122, -125, -128, -131])
@pytest.mark.parametrize("tokens", [5, 12, 20])
def test_small_h(gpu_lib, tokens, exponent):
    """Weights of the tokens that leave h near the end of bf16's range: finite weights of
    the experts give what h gives, and infinite ones the infinity that it gives."""
    say(f"layer, h of about 2^{exponent}, {tokens} tokens")
    p = few_inputs(33, tokens, 1, 4, 256, 33, 3, 3, 0)
    p.w *= 2.0 ** exponent
    p.down["scales"] *= 2.0 ** 66
    p.down["lut"][p.down["lut"] == 0] = 1.0
    out, bound = want(p)
    slack = torch.stack([TINY * p.weights(p.down, int(e)).abs().sum(1) for e in p.ids[:, 0]])
    got = gpu_lib.experts_mlp(*p.cuda())
    assert bool(((got.double().cpu() - out).abs() <= bound + slack * (1 + HALF)).all())
    # a token's sign of every column's infinity is that of the last column's h times the weight
    last = 32
    p.down["scales"][:, last] = torch.inf
    got = gpu_lib.experts_mlp(*p.cuda()).double().cpu()
    seen = 0
    for m, e in enumerate(p.ids[:, 0]):
        g, u = (p.weights(p.up, int(e)) @ p.x[m].double()).chunk(2)
        h = (p.w[m, 0].double() * g * torch.sigmoid(g) * u)[last]
        if h.abs() < 2.0 ** -147:  # may be zero in float32
            continue
        seen += 1
        assert torch.equal(got[m], h * p.weights(p.down, int(e))[:, last])
    assert seen > tokens // 2
