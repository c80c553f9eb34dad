"""Slots sorted by group and rows moved to their places and back, against plain
float64 (or integer) references on the host.

Tolerances. A bf16 store is off by at most half a step, 2^-8 of the value. A
float32 sum of n products is off by at most (n + 1) 2^-24 times the sum of
their magnitudes (each product and each addition rounds once); n is the longest
chain of additions an operation makes.
"""
import numpy as np
import pytest
import torch

from helpers import say

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8
FP32 = 2.0 ** -24


def sorted_slots(ids, groups):
    """offsets, order, position by their definition, in plain Python."""
    flat = ids.reshape(-1).tolist()
    placed = sorted((g, i) for i, g in enumerate(flat) if 0 <= g < groups)
    order = np.full(len(flat), -1, dtype=np.int32)
    position = np.full(len(flat), -1, dtype=np.int32)
    for p, (_, i) in enumerate(placed):
        order[p], position[i] = i, p
    counts = np.bincount([g for g, _ in placed], minlength=groups)
    return np.concatenate([[0], np.cumsum(counts)]), order, position.reshape(ids.shape)


def check_route(r, ids, groups):
    offsets, order, position = sorted_slots(ids, groups)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.position.cpu().numpy(), position)


def some_ids(seed, tokens, top_k, groups, kind="spread"):
    g = np.random.default_rng([seed, tokens, top_k, groups])
    if kind == "one":       # every slot in one group, the same id twice in a token
        ids = np.full((tokens, top_k), groups - 1)
    elif kind == "none":    # nothing selected
        ids = np.full((tokens, top_k), -1)
    elif kind == "wild":    # ids far outside the groups among the others
        ids = g.choice([-2 ** 31, -1, 0, groups - 1, groups, 2 ** 31 - 1], (tokens, top_k))
    else:                   # uneven, some groups without slots, some slots dropped
        ids = (g.random((tokens, top_k)) ** 2 * (groups + 1)).astype(np.int64) - 1
    return ids.astype(np.int32)


def routed(T, ids, groups):
    return T.route(torch.from_numpy(ids).cuda(), groups)


@pytest.mark.parametrize("kind", ["spread", "one", "none", "wild"])
@pytest.mark.parametrize("tokens,top_k,groups", [(1, 1, 1), (1, 8, 128), (3, 5, 2), (63, 1, 1024),
                                                 (64, 2, 7), (65, 3, 64), (1000, 8, 256)])
def test_route(gpu_lib, tokens, top_k, groups, kind):
    say(f"route {tokens} x {top_k} into {groups}, {kind}")
    ids = some_ids(1, tokens, top_k, groups, kind)
    check_route(routed(gpu_lib, ids, groups), ids, groups)


@pytest.mark.parametrize("tokens,top_k,groups", [
    (1024, 8, 128),      # the most slots one workgroup sorts
    (8193, 1, 1),        # one more: five chunks, the last of one slot
    (4100, 2, 1024),     # a short last chunk, many groups
    (70001, 8, 60),      # more slots than 256 chunks of 2048: longer chunks
])
@pytest.mark.parametrize("kind", ["spread", "one", "none"])
def test_route_many_slots(gpu_lib, tokens, top_k, groups, kind):
    say(f"route {tokens} x {top_k} into {groups}, {kind}")
    ids = some_ids(2, tokens, top_k, groups, kind)
    check_route(routed(gpu_lib, ids, groups), ids, groups)


def test_route_no_tokens(gpu_lib):
    say("route of no tokens")
    r = gpu_lib.route(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert r.offsets.tolist() == [0] * 10
    assert r.order.numel() == 0 and tuple(r.position.shape) == (0, 4)


@pytest.mark.parametrize("tokens", [37, 9000])
def test_route_repeats(gpu_lib, tokens):
    """Equal ids in equal order: nothing depends on the order of atomics."""
    say(f"route repeated, {tokens} tokens")
    ids = torch.from_numpy(some_ids(3, tokens, 4, 33)).cuda()
    first = gpu_lib.route(ids, 33)
    for _ in range(5):
        for a, b in zip(first, gpu_lib.route(ids, 33)):
            assert torch.equal(a, b)


def bf16(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)


SIZES = [(1, 1, 1, 8), (1, 8, 16, 2048), (5, 3, 4, 7), (33, 2, 8, 264), (130, 6, 60, 1000),
         (17, 8, 128, 4111), (300, 1, 3, 5120)]


def state(T, seed, tokens, top_k, groups, width):
    g = np.random.default_rng([seed, tokens, top_k, width])
    ids = some_ids(seed, tokens, top_k, groups)
    r = routed(T, ids, groups)
    _, order, position = sorted_slots(ids, groups)
    return g, r, order, position


@pytest.mark.parametrize("tokens,top_k,groups,width", SIZES)
def test_dispatch(gpu_lib, tokens, top_k, groups, width):
    say(f"dispatch {tokens} x {top_k}, width {width}")
    g, r, order, _ = state(gpu_lib, 4, tokens, top_k, groups, width)
    x = bf16(g.standard_normal((tokens, width)))
    x[0, 0] = float("nan")  # moved like any other value
    out = torch.full((tokens * top_k, width), 3.0, dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.dispatch(x.cuda(), r, out=out) is out
    want = torch.full((tokens * top_k, width), 3.0, dtype=torch.bfloat16)
    live = order >= 0
    want[live] = x[order[live] // top_k]
    assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,top_k,groups,width", SIZES)
def test_combine(gpu_lib, tokens, top_k, groups, width, weighted):
    say(f"combine {tokens} x {top_k}, width {width}, weighted {weighted}")
    g, r, order, position = state(gpu_lib, 5, tokens, top_k, groups, width)
    y = bf16(g.standard_normal((tokens * top_k, width)))
    y[(order < 0).nonzero()[0]] = float("nan")  # behind the last slot: not read
    w = torch.from_numpy(g.standard_normal((tokens, top_k)).astype(np.float32))
    w[torch.from_numpy(position) < 0] = float("inf")  # dropped slots: not used
    got = gpu_lib.combine(y.cuda(), w.cuda() if weighted else None, r).double().cpu().numpy()
    yd, wd = y.double().numpy(), (w.double().numpy() if weighted else np.ones((tokens, top_k)))
    want, size = np.zeros((tokens, width)), np.zeros((tokens, width))
    for m in range(tokens):
        for j in range(top_k):
            if position[m, j] >= 0:
                want[m] += wd[m, j] * yd[position[m, j]]
                size[m] += abs(wd[m, j] * yd[position[m, j]])
    fp32 = (top_k + 1) * FP32 * size
    assert np.all(np.abs(got - want) <= BF16 * (np.abs(want) + fp32) + fp32)


@pytest.mark.parametrize("tokens,top_k,groups,width", SIZES)
def test_combine_backward(gpu_lib, tokens, top_k, groups, width):
    say(f"combine backward {tokens} x {top_k}, width {width}")
    g, r, order, position = state(gpu_lib, 6, tokens, top_k, groups, width)
    y, dout = bf16(g.standard_normal((tokens * top_k, width))), bf16(g.standard_normal((tokens, width)))
    y[(order < 0).nonzero()[0]] = float("nan")
    w = torch.from_numpy(g.standard_normal((tokens, top_k)).astype(np.float32))
    w[torch.from_numpy(position) < 0] = float("nan")
    dy = torch.full((tokens * top_k, width), 3.0, dtype=torch.bfloat16, device="cuda")
    dy2, dw = gpu_lib.combine_backward(dout.cuda(), y.cuda(), w.cuda(), r, dy=dy)
    assert dy2 is dy
    got, gotw = dy.double().cpu().numpy(), dw.double().cpu().numpy()
    dd, yd, wd = dout.double().numpy(), y.double().numpy(), w.double().numpy()
    chain = -(-width // 64) + 16  # a lane's products, then six steps across the wave
    for m in range(tokens):
        for j in range(top_k):
            p = position[m, j]
            if p < 0:
                assert gotw[m, j] == 0
                continue
            want = wd[m, j] * dd[m]
            assert np.all(np.abs(got[p] - want) <= BF16 * np.abs(want) * (1 + FP32) + FP32 * np.abs(want))
            assert abs(gotw[m, j] - dd[m] @ yd[p]) <= chain * FP32 * (np.abs(dd[m]) @ np.abs(yd[p]))
    assert np.all(got[order < 0] == 3.0)


def test_gradient_against_differences(gpu_lib):
    """combine is linear in y and in the weights: a step of the weights changes
    <dout, out> by the step times dweights, and a step of y by the step times dy
    (float64 references of the outputs' roundings as above)."""
    say("combine gradient against differences")
    T, (tokens, top_k, groups, width) = gpu_lib, (40, 4, 10, 512)
    g, r, order, position = state(T, 7, tokens, top_k, groups, width)
    y, dout = bf16(g.standard_normal((tokens * top_k, width))), bf16(g.standard_normal((tokens, width)))
    w = torch.from_numpy(g.standard_normal((tokens, top_k)).astype(np.float32))
    dy, dw = T.combine_backward(dout.cuda(), y.cuda(), w.cuda(), r, dy=torch.zeros_like(y).cuda())
    step_w = torch.from_numpy(g.standard_normal((tokens, top_k)).astype(np.float32))
    d = dout.double()

    def value(yy, ww):  # <dout, combine>, with the rounding error the outputs may have
        out = T.combine(yy.cuda(), ww.cuda(), r).double().cpu()
        return float((d * out).sum()), float((d * out).abs().sum()) * BF16

    v0, e0 = value(y, w)
    v1, e1 = value(y, w + step_w)
    exact_step = ((w + step_w).double() - w.double())
    assert abs((v1 - v0) - float((dw.double().cpu() * exact_step).sum())) <= 1.01 * (e0 + e1)
    y2 = bf16(g.standard_normal((tokens * top_k, width)))
    v2, e2 = value(y2, w)
    step_y = y2.double() - y.double()
    inner = dy.double().cpu() * step_y
    assert abs((v2 - v0) - float(inner.sum())) <= 1.01 * (e0 + e2 + BF16 * float(inner.abs().sum()))


def test_gradient_is_exactly_the_differences(gpu_lib):
    """combine is linear in y and in the weights: for sparse small integers, whose
    outputs and products are exact in bf16, the change of <dout, out> over a step of
    the weights or of y is the step's product with its gradient, to the last bit."""
    say("combine gradient against exact differences")
    T, (tokens, top_k, groups, width) = gpu_lib, (40, 4, 10, 512)
    g, r, order, position = state(T, 9, tokens, top_k, groups, width)

    def draw(*shape, zeros=0.75):
        v = g.integers(-2, 3, shape) * (g.random(shape) >= zeros)
        return torch.from_numpy(v.astype(np.float32))

    y, dout = draw(tokens * top_k, width).to(torch.bfloat16), draw(tokens, width).to(torch.bfloat16)
    w = draw(tokens, top_k, zeros=0.2)
    dy, dw = T.combine_backward(dout.cuda(), y.cuda(), w.cuda(), r, dy=torch.zeros_like(y).cuda())
    dy, dw = dy.double().cpu(), dw.double().cpu()

    def value(yy, ww):
        out = T.combine(yy.to(torch.bfloat16).cuda(), ww.cuda(), r).double().cpu()
        assert float(out.abs().max()) <= 128
        return float((dout.double() * out).sum())

    before = value(y, w)
    for scale in (1, -1):
        step = scale * draw(tokens, top_k, zeros=0.2)
        change = float((dw * step.double()).sum())
        assert value(y, w + step) - before == change and change != 0
        step = scale * draw(tokens * top_k, width)
        change = float((dy * step.double()).sum())
        assert value(y.float() + step, w) - before == change and change != 0


def test_dispatch_gradient_is_the_plain_combine(gpu_lib):
    """<dispatch(x), g> = <x, combine(g)> for exactly summed small integers."""
    say("dispatch and its gradient")
    T, (tokens, top_k, groups, width) = gpu_lib, (50, 4, 9, 96)
    g, r, order, _ = state(T, 8, tokens, top_k, groups, width)
    x, d = (bf16(g.integers(-3, 4, (n, width))) for n in (tokens, tokens * top_k))
    out = T.dispatch(x.cuda(), r, out=torch.zeros_like(d).cuda()).double().cpu()
    dx = T.combine(d.cuda(), None, r).double().cpu()
    live = torch.from_numpy(order >= 0)
    assert float((out[live] * d.double()[live]).sum()) == float((x.double() * dx).sum())


def test_captured_and_replayed(gpu_lib):
    """route, dispatch, combine and the gradient in one graph, replayed with
    other ids and rows between eager calls; every replay against eager."""
    say("grouped moves captured")
    T, (tokens, top_k, groups, width) = gpu_lib, (2100, 4, 40, 256)
    sets = []
    for seed in (9, 10, 11):
        g = np.random.default_rng(seed)
        sets.append((torch.from_numpy(some_ids(seed, tokens, top_k, groups)).cuda(),
                     bf16(g.standard_normal((tokens, width))).cuda(),
                     torch.from_numpy(g.random((tokens, top_k)).astype(np.float32)).cuda()))
    ids, x, w = (t.clone() for t in sets[0])
    out = torch.zeros((tokens * top_k, width), dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(out)

    def chain(ids, x, w, out, dy):
        r = T.route(ids, groups)
        T.dispatch(x, r, out=out)
        z = T.combine(out, w, r)
        _, dw = T.combine_backward(z, out, w, r, dy=dy)
        return r.offsets, r.order, r.position, z, dw

    chain(ids, x, w, out, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = chain(ids, x, w, out, dy)
    for n in (1, 2, 0, 1, 1):
        for t, v in zip((ids, x, w), sets[n]):
            t.copy_(v)
        out.zero_(), dy.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager_out, eager_dy = torch.zeros_like(out), torch.zeros_like(dy)
        for a, b in zip(kept + (out, dy), chain(*sets[n], eager_out, eager_dy) + (eager_out, eager_dy)):
            assert torch.equal(a, b)


def test_another_stream(gpu_lib):
    say("route and moves on another stream")
    T, (tokens, top_k, groups, width) = gpu_lib, (3000, 4, 40, 512)
    ids = some_ids(12, tokens, top_k, groups)
    x = bf16(np.random.default_rng(12).standard_normal((tokens, width))).cuda()
    dev_ids = torch.from_numpy(ids).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = T.route(dev_ids, groups, stream=side)
    out = torch.zeros((tokens * top_k, width), dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    T.dispatch(x, r, out=out, stream=side)
    z = T.combine(out, None, r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check_route(r, ids, groups)
    assert torch.equal(z, T.combine(out, None, r))


def test_wild_positions_select_no_row(gpu_lib):
    """Positions outside the slots are skipped like dropped ones."""
    say("positions outside the slots")
    T = gpu_lib
    pos = torch.tensor([[0, 2 ** 31 - 1], [-5, 4], [3, -2 ** 31]], dtype=torch.int32, device="cuda")
    r = T.Route(None, None, pos)
    x = torch.ones((3, 16), dtype=torch.bfloat16, device="cuda")
    out = T.dispatch(x, r, out=torch.zeros((6, 16), dtype=torch.bfloat16, device="cuda"))
    assert out.sum(1).tolist() == [16, 0, 0, 16, 16, 0]
    z = T.combine(torch.ones((6, 16), dtype=torch.bfloat16, device="cuda"), None, r)
    assert z[:, 0].tolist() == [1, 1, 1]


def test_offsets_past_32_bits(gpu_lib):
    """More than 2^31 values in the sorted rows: the last rows are the tokens'."""
    say("dispatch and combine past 2^31 values")
    T, tokens, top_k, width = gpu_lib, 66000, 8, 4096
    ids = torch.zeros((tokens, top_k), dtype=torch.int32, device="cuda")
    x = torch.arange(tokens, device="cuda").remainder(251).to(torch.bfloat16)[:, None].repeat(1, width)
    r = T.route(ids, 2)
    assert tokens * top_k * width > 2 ** 31
    out = T.dispatch(x, r)
    assert torch.equal(out[-top_k - 3:], x[[-2] * 3 + [-1] * top_k])
    assert torch.equal(T.combine(out, None, r)[-5:], (x[-5:].float() * top_k).to(torch.bfloat16))
    dy, dw = T.combine_backward(x, out, torch.full((tokens, top_k), 2.0, device="cuda"), r)
    assert torch.equal(dy[-9:], (2 * x[[-2] + [-1] * 8].float()).to(torch.bfloat16))
    assert torch.equal(dw[-1], (x[-1].double() @ x[-1].double()).float().repeat(top_k))
