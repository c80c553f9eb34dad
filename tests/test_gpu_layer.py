"""A whole layer of experts for few tokens (trellis_experts_mlp) against the CPU
oracle's weights in float64.

Bounds, value by value, with eps = 2^-24 (float32) and half a bf16 step 2^-8 of a
value: a product's float32 sum of n terms is off by at most n eps times the sum of
the terms' magnitudes (in any order); g's error reaches h by at most 1.1 w |u|
(silu's slope is below 1.1), u's by w |silu(g)|; h's own float32 work (exp,
division, three products) adds 16 eps of it, and its rounding half a step (up to 8
tokens: the half step 2^-8 of what is left behind its upper 8 bits, 2^-7 of it); out
has all that times |Wd|, its own sums, and half a step.
"""
import numpy as np
import pytest
import torch

import oracle
from dequant_gemm_trellis_amd import synth
from helpers import say

pytestmark = pytest.mark.gpu

EPS, HALF = 2.0 ** -24, 2.0 ** -8


class Layer:
    """Host tensors of one layer and its tokens."""

    def __init__(self, seed, tokens, top_k, experts, hidden, inter, k, k_down, axis, il=0, distinct=True,
                 wild=False):
        g = np.random.default_rng([seed, tokens, top_k, experts, hidden, inter, k, axis])
        self.args = tokens, top_k, experts, hidden, inter, k, k_down, axis
        self.hidden, self.inter, self.experts = hidden, inter, experts
        self.up_shape = synth.Shape(1, 256, 12, k, hidden, 2 * inter, il)
        self.down_shape = synth.Shape(axis, 256, 12, k_down, inter, hidden, il)
        self.up = self.matrices(g, synth.Shape(1, 256, 12, k, hidden, 2 * inter), experts, il)
        self.down = self.matrices(g, synth.Shape(axis, 256, 12, k_down, inter, hidden), experts, il)
        self.x = torch.from_numpy(g.standard_normal((tokens, hidden))).to(torch.bfloat16)
        if distinct and top_k <= experts:
            ids = np.stack([g.permutation(experts)[:top_k] for _ in range(tokens)]) if tokens else \
                np.zeros((0, top_k))
        else:
            ids = g.integers(0, experts, (tokens, top_k))
        if wild:
            ids = np.where(g.random(ids.shape) < 0.4, g.choice([-1, experts, 2 ** 31 - 1, -2 ** 31], ids.shape), ids)
        self.ids = torch.from_numpy(ids.astype(np.int32))
        self.w = torch.from_numpy(g.uniform(0.1, 1, (tokens, top_k)).astype(np.float32))

    @staticmethod
    def matrices(g, shape, experts, il):
        codes = g.integers(0, 2 ** 32, (experts, shape.rows, shape.words_per_row), dtype=np.uint32)
        scales = (g.uniform(0.5, 1.5, (experts, shape.rows)) * shape.in_features ** -0.5).astype(np.float32)
        lut = g.standard_normal(4096).astype(np.float32)
        stored = codes
        if il:
            stored = np.stack([oracle.interleave_blocks(c, shape.rows, shape.cols // 256, 8 * shape.k)
                               for c in codes])
        return {"shape": shape, "codes": codes, "stored": stored, "scales": scales, "lut": lut}

    def weights(self, m, e):
        """[out, in] of expert e in float64."""
        s = m["shape"]
        w = oracle.expand(m["codes"][e], m["scales"][e], m["lut"], s.axis, 256, 12, s.k, s.in_features,
                          s.out_features)
        w = torch.from_numpy(w.view(np.int16)).view(torch.bfloat16).double().reshape(s.rows, s.cols)
        return w if s.axis == 1 else w.T.contiguous()

    def want(self, weighted=True):
        """(out, bound) in float64."""
        tokens = len(self.ids)
        out = torch.zeros((tokens, self.hidden), dtype=torch.float64)
        bound, size_of_sums = torch.zeros_like(out), torch.zeros_like(out)
        for e in range(self.experts):
            mine = self.ids == e
            m = mine.any(1).nonzero()[:, 0]
            if not len(m):
                continue
            share = torch.where(mine, self.w if weighted else torch.ones_like(self.w), torch.zeros(())).double()
            w = share.sum(1)[m][:, None]
            wu, wd, x = self.weights(self.up, e), self.weights(self.down, e), self.x[m].double()
            gu, size = x @ wu.T, x.abs() @ wu.abs().T * (self.hidden * EPS)
            g, u = gu.chunk(2, dim=1)
            dg, du = size.chunk(2, dim=1)
            silu = g * torch.sigmoid(g)
            h = w * silu * u
            off = w.abs() * (1.1 * (u.abs() + du) * dg + silu.abs() * du) + h.abs() * ((HALF if tokens > 8 else 2.0 ** -15) + 16 * EPS)
            out[m] += h @ wd.T
            bound[m] += (off + 2 * (self.inter + 8) * EPS * h.abs()) @ wd.abs().T
            size_of_sums[m] += h.abs() @ wd.abs().T
        # the experts' sums meet in float32, and the whole is rounded once
        return out, (bound + 40 * EPS * size_of_sums) * (1 + HALF) + HALF * out.abs()

    def cuda(self, weighted=True):
        def dev(m):
            return (torch.from_numpy(m["stored"].view(np.int32)).cuda(), torch.from_numpy(m["scales"]).cuda(),
                    torch.from_numpy(m["lut"]).cuda())

        return (self.x.cuda(), self.ids.cuda(), self.w.cuda() if weighted else None, dev(self.up),
                dev(self.down), self.up_shape, self.down_shape)


def check(got, want, bound):
    err = (got.double().cpu() - want).abs()
    assert bool((err <= bound + 1e-30).all()), float((err / (bound + 1e-30)).max())


# tokens, top_k, experts, hidden, inter, k, k of down, axis of down
SIZES = [
    (1, 1, 1, 256, 8, 2, 2, 0), (1, 2, 4, 256, 40, 3, 4, 0), (2, 2, 8, 512, 256, 2, 3, 1),
    (1, 8, 64, 512, 256, 3, 3, 1), (5, 2, 8, 1024, 300, 4, 4, 0), (16, 4, 16, 256, 33, 2, 2, 0),
    (17, 4, 16, 256, 33, 3, 2, 0), (32, 8, 70, 256, 64, 4, 3, 0), (32, 8, 24, 512, 256, 2, 2, 1),
    (9, 3, 5, 768, 512, 4, 2, 1), (31, 32, 40, 256, 9, 3, 3, 0), (3, 5, 1024, 256, 31, 2, 4, 0),
    (32, 1, 1, 512, 1, 2, 3, 0), (7, 2, 6, 2304, 256, 3, 4, 1), (24, 2, 3, 768, 100, 2, 2, 0),
    (13, 4, 15, 1280, 272, 4, 4, 0), (4, 1, 1, 1280, 1000, 3, 3, 0), (20, 1, 1, 1024, 768, 2, 4, 1),
    (32, 8, 9, 8448, 40, 2, 3, 0), (32, 8, 64, 768, 256, 3, 3, 1), (18, 3, 200, 1280, 52, 4, 2, 0),
    (32, 2, 8, 2048, 8, 2, 2, 0), (29, 1, 300, 256, 300, 3, 4, 0), (17, 8, 64, 512, 129, 2, 4, 0),
    (32, 32, 55, 256, 150, 2, 3, 0),
    # more units of 8 columns than 256 compute units have waves, of few tokens each ...
    (32, 8, 64, 256, 264, 2, 4, 0), (17, 8, 130, 256, 129, 3, 3, 0), (30, 6, 70, 512, 256, 3, 2, 1),
    (21, 5, 40, 768, 412, 4, 2, 0), (32, 1, 300, 256, 521, 2, 3, 0), (32, 32, 70, 256, 237, 4, 4, 0),
    # ... of many, and as many units as waves
    (17, 3, 3, 256, 5470, 2, 2, 0), (32, 4, 16, 512, 1024, 3, 3, 1),
    # few units a workgroup of many blocks, many units of few
    (32, 2, 3, 5120, 700, 4, 3, 0), (16, 2, 3, 5120, 700, 2, 4, 0), (32, 1, 1, 256, 17408, 2, 2, 0),
]


@pytest.mark.parametrize("size", SIZES)
def test_layer(gpu_lib, size):
    say(f"layer {size}")
    p = Layer(1, *size)
    check(gpu_lib.experts_mlp(*p.cuda()), *p.want())


@pytest.mark.parametrize("popular", [16, 17, 25, 32])
@pytest.mark.parametrize("k,axis,inter", [(2, 1, 512), (3, 0, 348), (4, 0, 345), (3, 0, 3), (2, 1, 768),
                                            (3, 0, 700), (4, 0, 697)])
def test_one_expert_has_most(gpu_lib, popular, k, axis, inter):
    """Many tokens of few per expert, but for one that 16, 17 or all of them chose: it
    has one tile of tokens or two (with fewer columns than 690 all are two operands)."""
    say(f"layer, {popular} of 32 tokens for one expert, k={k}")
    p = Layer(16, 32, 2, 24, 512, inter, k, k, axis)
    p.ids[:, 0] = torch.where(torch.randperm(32, generator=torch.Generator().manual_seed(popular)) < popular, 5, -1)
    p.ids[:, 1] = torch.arange(32) % 24
    check(gpu_lib.experts_mlp(*p.cuda()), *p.want())


@pytest.mark.parametrize("size", [(2, 2, 8, 512, 512, 2, 3, 1), (18, 4, 6, 1024, 100, 3, 2, 0),
                                  (18, 4, 40, 512, 512, 2, 4, 1)])
def test_block_pairs(gpu_lib, size):
    say(f"layer, pairs, {size}")
    p = Layer(2, *size, il=2)
    check(gpu_lib.experts_mlp(*p.cuda()), *p.want())


@pytest.mark.parametrize("size", [(3, 4, 6, 256, 40, 3, 3, 0), (30, 6, 5, 512, 256, 2, 4, 1),
                                  (30, 6, 48, 256, 180, 3, 2, 0), (30, 6, 48, 256, 360, 3, 2, 0)])
@pytest.mark.parametrize("weighted", [True, False])
def test_same_expert_twice_and_none(gpu_lib, size, weighted):
    """Ids that occur more than once in a token, and ids that choose none."""
    say(f"layer, repeated and dropped ids, {size}")
    p = Layer(3, *size, distinct=False, wild=True)
    p.ids[1] = -1
    p.ids[2] = p.ids[2].clamp(0, 0)
    out = gpu_lib.experts_mlp(*p.cuda(weighted))
    check(out, *p.want(weighted))
    assert not bool(out[1].any())


def test_nobody_chooses(gpu_lib):
    p = Layer(4, 6, 2, 8, 512, 100, 3, 3, 0)
    p.ids.fill_(-1)
    out = torch.full((6, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.experts_mlp(*p.cuda(), out=out) is out
    assert not bool(out.any())


def test_no_tokens(gpu_lib):
    p = Layer(5, 0, 2, 8, 256, 40, 2, 2, 0)
    assert gpu_lib.experts_mlp(*p.cuda()).shape == (0, 256)


@pytest.mark.parametrize("size", [(6, 2, 8, 512, 100, 3, 3, 0), (20, 2, 8, 512, 256, 2, 4, 1), (20, 3, 6, 512, 100, 2, 4, 0),
                                  (20, 3, 48, 256, 200, 3, 3, 0), (20, 3, 48, 256, 365, 3, 3, 0)])
def test_not_finite_stays_where_it_is(gpu_lib, size):
    """NaN in one token's row, and an expert of infinite weights, reach only the tokens
    that have them."""
    say(f"layer, not finite, {size}")
    p = Layer(6, *size)
    want, bound = p.want()
    p.x[2, 7] = torch.nan
    p.x[4, 3] = torch.inf
    bad = int(p.ids[0, 0])  # an expert of token 0
    p.down["scales"][bad] = np.inf
    other = int(p.ids[1, 0])
    p.up["scales"][other, ::2] = np.nan
    out = gpu_lib.experts_mlp(*p.cuda())
    hit = ((p.ids == bad) | (p.ids == other)).any(1)
    hit[2] = hit[4] = True
    assert not bool(out[hit.cuda()].isfinite().all(1).any())
    clean = (~hit).nonzero()[:, 0]
    assert len(clean)
    check(out[clean.cuda()], want[clean], bound[clean])


@pytest.mark.parametrize("tokens", [5, 12, 20])
@pytest.mark.parametrize("inter", [33, 300, 40, 4110])
def test_infinite_last_row(gpu_lib, inter, tokens):
    """The last stored row of a partial step may be infinite: its column of h makes
    infinities of it, and nothing makes NaN."""
    p = Layer(7, tokens, 2, 4, 256, inter, 3, 3, 0)
    say(f"layer, infinite last row, inter {inter}")
    p.down["scales"][:, inter - 1] = np.inf
    p.down["lut"][p.down["lut"] == 0] = 1.0
    # h of the last column: sums of infinities of both signs are NaN, so one expert each
    p.ids[:, 1] = -1
    out = gpu_lib.experts_mlp(*p.cuda())
    assert bool(out.isinf().all())


def test_workspace_holds_anything(gpu_lib):
    """Nothing that lay in the workspace enters, NaN or other."""
    for size in ((5, 2, 8, 512, 300, 3, 3, 0), (20, 3, 8, 512, 256, 2, 2, 1), (20, 3, 48, 256, 365, 3, 3, 0)):
        say(f"layer, workspace {size}")
        p = Layer(8, *size)
        args = p.cuda()
        want = gpu_lib.experts_mlp(*args)
        ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
        for fill in (0, 255, 127):
            ws.fill_(fill)
            assert torch.equal(gpu_lib.experts_mlp(*args, workspace=ws), want)


@pytest.mark.parametrize("size", [(1, 8, 64, 512, 300, 3, 3, 0), (32, 4, 16, 512, 256, 2, 2, 1),
                                  (32, 4, 40, 256, 216, 4, 3, 0), (32, 4, 40, 256, 420, 4, 3, 0)])
def test_captured_and_replayed(gpu_lib, size):
    """Replays with other tokens and other experts, between the program's own calls."""
    p = Layer(9, *size)
    args = p.cuda()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        gpu_lib.experts_mlp(*args)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpu_lib.experts_mlp(*args)
    for seed in (10, 11, 12):
        say(f"layer, replay {seed}")
        q = Layer(seed, *size, wild=seed == 12)
        for t, v in zip(args[:3], (q.x, q.ids, q.w)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, gpu_lib.experts_mlp(*args))
        q.up, q.down = p.up, p.down
        check(out, *q.want())


def test_two_calls_at_once(gpu_lib):
    """Calls on two streams, each with a workspace of its own."""
    a, b = Layer(13, 8, 4, 16, 512, 300, 3, 3, 0), Layer(14, 30, 4, 16, 512, 256, 2, 2, 1)
    args = a.cuda(), b.cuda()
    want = [gpu_lib.experts_mlp(*x) for x in args]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    say("layer, two streams")
    for _ in range(5):
        got = [gpu_lib.experts_mlp(*x, stream=s) for x, s in zip(args, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_a_decode_step(gpu_lib):
    """The layer against the calls that it stands for: sort, dispatch, the experts'
    products, SwiGLU and combine, whose intermediate roundings differ."""
    p = Layer(15, 32, 4, 16, 512, 256, 3, 4, 0)
    say("a decode step")
    x, ids, w, up, down, g_up, g_down = args = p.cuda()
    out = gpu_lib.experts_mlp(*args)
    r = gpu_lib.route(ids, 16)
    gu = gpu_lib.experts(gpu_lib.dispatch(x, r), r.offsets, *up, g_up)
    y = gpu_lib.experts(gpu_lib.swiglu(gu)[0], r.offsets, *down, g_down)
    chain = gpu_lib.combine(y, w, r)
    want, bound = p.want()
    check(out, want, bound)
    # the chain rounds g, u and y too: 3 more half steps of the parts' magnitudes
    assert float((chain.double().cpu() - want).norm() / want.norm()) < 5 * HALF
    assert float((out.double() - chain.double()).norm() / chain.double().norm()) < 5 * HALF
