"""Workloads of the operators around a layer of experts: the whole layer for a
few tokens, SwiGLU over many rows with its gradient, rows kept in 8 bits for the
backward pass, and the adapters' gradient that reads them.

Each case is one call (or the calls a user makes in a row) with inputs drawn from
a seed. `run` computes it in plain float32 torch operations, or, where `own` is
set, through the package's entry points. `exact` computes the same in float64,
written from the definitions below.

Definitions:
  layer            out[m] = sum over the experts e that token m chose of
                   W_e^down (w silu(W_e^gate x[m]) * (W_e^up x[m])), w the sum of m's
                   weights for e; gate and up stacked, weights decoded from their
                   trellis codes and rounded to bf16
  swiglu           h = silu(g) u with [g, u] the halves of a row, silu(g) = g s,
                   s = 1 / (1 + exp(-g))
  swiglu_gradient  dg = dh u s (1 + g (1 - s)), du = dh g s
  keep             groups of 32 values of a row in 8 bits: with E the largest exponent
                   field of the group's bf16 values, a value x is held as the integer
                   q = x 2^(133 - E), rounded half to even and cut off at +-127, and
                   stands for q 2^(E - 133) (a row's last group may be shorter). Rows
                   of [g, u] are kept as two rows, g and u
  adapters_gradient_kept   (a = ids[m]; rows with a outside [0, count) have none)
                   g[m] = s[a] B[a] dy[m],  dx[m] = base[m] + A[a]^T g[m],
                   dA[a] = sum_m g[m] x[m]^T,  dB[a] = s[a] sum_m u[m] dy[m]^T,
                   x held in 8 bits
"""
from __future__ import annotations

import torch

own = False

# (hidden, inter, most experts); on axis 1 of the down projection inter is a multiple of 256
_LAYERS = ((2048, 768, 64), (1024, 768, 64), (1024, 300, 64), (512, 1000, 64), (2048, 512, 64),
           (256, 40, 64), (5120, 1280, 15), (4096, 1024, 24))
_ADAPTED = ((5120, 17408), (17408, 5120), (2048, 2048), (512, 4111), (1024, 300), (768, 5000))


def listed():
    return [
        # one request decodes a token through a layer of 64 experts
        {"name": "layer_token", "op": "layer", "tokens": 1, "top_k": 8, "experts": 64,
         "hidden": 2048, "inter": 768, "k": 3, "k_down": 3, "axis_down": 0},
        # a full decode batch; nearly every expert is chosen by someone
        {"name": "layer_batch", "op": "layer", "tokens": 32, "top_k": 8, "experts": 64,
         "hidden": 2048, "inter": 768, "k": 2, "k_down": 3, "axis_down": 1},
        # a few requests of a small model whose inner width is no multiple of anything
        {"name": "layer_small", "op": "layer", "tokens": 7, "top_k": 2, "experts": 8,
         "hidden": 1024, "inter": 300, "k": 4, "k_down": 4, "axis_down": 0},
        # a drafted sequence is checked in a wide layer of few experts
        {"name": "layer_wide", "op": "layer", "tokens": 13, "top_k": 4, "experts": 15,
         "hidden": 5120, "inter": 1280, "k": 4, "k_down": 4, "axis_down": 0},
        # between the two products of a prompt of 2048 tokens with 8 experts each
        {"name": "swiglu_prompt", "op": "swiglu", "rows": 16384, "inter": 768},
        # the same for a decode batch of more tokens than the whole layer takes, odd rows
        {"name": "swiglu_decode", "op": "swiglu", "rows": 203, "inter": 1003},
        # a training step of a dense MLP: forward with [g, u] kept in 8 bits, then backward from them
        {"name": "swiglu_training", "op": "swiglu_pass", "rows": 4096, "inter": 17408},
        # backward from bf16 rows of odd length, h made again for an adapter of the down projection
        {"name": "swiglu_gradient", "op": "swiglu_gradient", "rows": 811, "inter": 4111,
         "kept": False, "again": True},
        # a training batch's input of a projection is put away in 8 bits and brought back
        {"name": "keep_rows", "op": "keep", "rows": 4096, "width": 5120},
        # a few rows whose last group is short
        {"name": "keep_small", "op": "keep", "rows": 77, "width": 1000},
        # backward of one training batch: two adapters on the up projection
        {"name": "adapters_gradient_kept", "op": "adapters_gradient_kept", "rows": 4096, "in": 5120,
         "out": 17408, "rank": 32, "count": 2, "runs": True},
        # backward over a short, odd batch of a small projection
        {"name": "adapters_gradient_kept_small", "op": "adapters_gradient_kept", "rows": 203,
         "in": 512, "out": 4111, "rank": 8, "count": 3, "runs": True},
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread over the logarithm."""
    return min(hi, int(lo * ((hi + 1) / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["layer", "layer", "layer", "swiglu", "swiglu_pass", "swiglu_gradient", "keep",
                     "adapters_gradient_kept", "adapters_gradient_kept"])
    if op == "layer":
        hidden, inter, most = rng.choice(_LAYERS)
        experts = _log(rng, 4, most)
        return {"op": op, "tokens": _log(rng, 1, 32), "top_k": rng.randint(1, min(8, experts)),
                "experts": experts, "hidden": hidden, "inter": inter, "k": rng.choice([2, 3, 4]),
                "k_down": rng.choice([2, 3, 4]),
                "axis_down": rng.choice([0, 1]) if inter % 256 == 0 else 0}
    if op == "adapters_gradient_kept":
        i, o = rng.choice(_ADAPTED)
        return {"op": op, "rows": _log(rng, 1, 4096), "in": i, "out": o,
                "rank": rng.choice([4, 8, 13, 16, 24, 32]), "count": _log(rng, 1, 16),
                "runs": rng.random() < 0.5}
    rows, width = _log(rng, 1, 16384), _log(rng, 40, 4200)
    width = width if rng.random() < 0.4 else -(-width // 32) * 32
    if op == "keep":
        return {"op": op, "rows": rows, "width": width}
    c = {"op": op, "rows": rows, "inter": width}
    if op == "swiglu_gradient":
        c["kept"], c["again"] = rng.random() < 0.5, rng.random() < 0.5
    return c


# ---- inputs -------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 29)
    return g


def _normal(g, *shape, std=1.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda")
    return t.normal_(0.0, std, generator=g)


def _activations(g, rows, width):
    """bf16 rows of which some channels are much larger than the others."""
    channel = torch.exp(_normal(g, 1, width, std=0.8))
    return (_normal(g, rows, width) * channel).to(torch.bfloat16)


def _codes(g, experts, rows, cols, k):
    """(codes, scales) of the experts' stored matrices [rows][cols]."""
    words = torch.randint(-2 ** 31, 2 ** 31, (experts, rows, cols * k // 32), dtype=torch.int64,
                          device="cuda", generator=g)
    # the decoded weights of a trained matrix have a standard deviation of about cols^-1/2
    return words.to(torch.int32), (torch.rand((experts, rows), device="cuda", generator=g) + 0.5) * cols ** -0.5


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op == "layer":
        t, k, e = case["tokens"], case["top_k"], case["experts"]
        hidden, inter = case["hidden"], case["inter"]
        s["x"] = _normal(g, t, hidden).to(torch.bfloat16)
        # top_k distinct experts per token, some of them more popular, a few choices dropped
        score = _normal(g, t, e) + _normal(g, 1, e, std=0.7)
        ids = score.topk(k, dim=1).indices.to(torch.int32)
        drop = torch.rand((t, k), device="cuda", generator=g) < 0.02
        s["ids"] = torch.where(drop, torch.full_like(ids, -1), ids).contiguous()
        s["w"] = torch.softmax(_normal(g, t, k), dim=1)
        s["up"] = _codes(g, e, 2 * inter, hidden, case["k"]) + (_normal(g, 4096),)
        stored = (hidden, inter) if case["axis_down"] == 1 else (inter, hidden)
        s["down"] = _codes(g, e, *stored, case["k_down"]) + (_normal(g, 4096),)
        return s
    if op == "keep":
        s["x"] = _activations(g, case["rows"], case["width"])
        return s
    if op == "adapters_gradient_kept":
        m, i, o, r, n = (case[x] for x in ("rows", "in", "out", "rank", "count"))
        if case["runs"]:  # packed sequences: each request's rows are adjacent
            cuts = torch.randint(0, m + 1, (n,), device="cuda", generator=g).sort().values
            run_of = torch.searchsorted(cuts, torch.arange(m, device="cuda"), right=True)
            ids = torch.randint(-1 if n > 2 else 0, n, (n + 1,), device="cuda", generator=g)[run_of]
        else:
            ids = torch.randint(0, n, (m,), device="cuda", generator=g)
        s["ids"] = ids.to(torch.int32).contiguous()
        x = _activations(g, m, i)
        s["codes"], s["exponents"] = _held(x)  # put away by the forward pass
        s["a"] = _normal(g, n, r, i, std=i ** -0.5).to(torch.bfloat16)
        s["b"] = _normal(g, n, r, o, std=r ** -0.5).to(torch.bfloat16)
        s["scales"] = torch.rand(n, device="cuda", generator=g) * 1.5 + 0.5
        s["dy"] = _normal(g, m, o).to(torch.bfloat16)
        s["base"] = _normal(g, m, i).to(torch.bfloat16)  # the projection's share of dx
        s["u"] = _spread((x.float() @ s["a"].float().reshape(n * r, i).t()).reshape(m, n, r), ids, n).sum(1)
        return s
    rows, n = case["rows"], case["inter"]
    gu = _activations(g, rows, 2 * n)
    if op != "swiglu":
        s["dh"] = _normal(g, rows, n).to(torch.bfloat16)
    if op == "swiglu_gradient" and case["kept"]:
        s["codes"], s["exponents"] = _held(gu.reshape(2 * rows, n))
    else:
        s["gu"] = gu
    return s


# ---- the plain forms ------------------------------------------------------------


def _power(e):
    """2^e in float64, exact (exp2 may be off by a last bit, which moves ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _held(x):
    """(codes int8 [rows, width], exponents uint8 [rows, groups]) of bf16 rows in 8 bits."""
    rows, width = x.shape
    groups = -(-width // 32)
    wide = torch.zeros((rows, groups * 32), dtype=x.dtype, device=x.device)
    wide[:, :width] = x
    wide = wide.reshape(rows, groups, 32)
    field = (wide.view(torch.int16).to(torch.int32) >> 7) & 255
    largest = field.amax(2)
    q = torch.round(wide.double() * _power(133 - largest)[:, :, None]).clamp(-127, 127)
    q = torch.where((largest < 255)[:, :, None], q, torch.zeros_like(q))
    return q.reshape(rows, -1)[:, :width].to(torch.int8).contiguous(), largest.to(torch.uint8)


def _values(codes, exponents):
    """The float32 values that rows in 8 bits stand for."""
    step = _power(exponents.int() - 133)
    step = torch.where(exponents < 255, step, torch.full_like(step, float("nan")))
    step = step.repeat_interleave(32, dim=1)[:, :codes.shape[1]]
    return (codes.double() * step).float()


def _spread(v, ids, count):
    """[rows, count, rank] with v[m] at adapter ids[m] and zeros elsewhere."""
    mine = ids.long()[:, None] == torch.arange(count, device=ids.device)[None, :]
    return torch.where(mine[:, :, None], v, torch.zeros_like(v))


def _weights(codes, scales, lut, k):
    """[experts, rows, cols] float32 values of the bf16 weights."""
    e, rows, words = codes.shape
    w = (codes.long() & 0xFFFFFFFF).reshape(e, rows, words // (8 * k), 8 * k)
    bit = (255 - torch.arange(256, device=codes.device)) * k
    at = bit // 32
    both = w[..., at] | (w[..., (at + 1) % (8 * k)] << 32)
    window = (both >> (bit % 32)) & 4095
    return (lut[window] * scales[:, :, None, None]).to(torch.bfloat16).float().reshape(e, rows, -1)


def _run_layer(s):
    case, ids = s["case"], s["ids"].long()
    tokens, top_k = ids.shape
    (uc, us, ul), (dc, ds, dl) = s["up"], s["down"]
    if tokens * top_k < case["experts"]:  # decode each choice's expert, else every expert
        at = ids.reshape(-1)
        uc, us, dc, ds = (t[at.clamp(min=0)] for t in (uc, us, dc, ds))
        token = torch.arange(tokens * top_k, device=ids.device) // top_k
        mine = (token[None, :] == torch.arange(tokens, device=ids.device)[:, None]) & (at >= 0)[None, :]
        share = torch.where(mine, s["w"].reshape(1, -1), torch.zeros((), device=ids.device))
    else:
        every = torch.arange(case["experts"], device=ids.device)
        share = ((ids[:, :, None] == every) * s["w"][:, :, None]).sum(1)
    up = _weights(uc, us, ul, case["k"]).transpose(1, 2).contiguous()
    gu = torch.bmm(s["x"].float()[None].expand(up.shape[0], -1, -1), up)
    del up
    g, u = gu[:, :, :case["inter"]], gu[:, :, case["inter"]:]
    h = g / (1 + torch.exp(-g)) * u * share.t()[:, :, None]
    down = _weights(dc, ds, dl, case["k_down"])
    if case["axis_down"] == 1:
        down = down.transpose(1, 2).contiguous()
    return torch.bmm(h, down).sum(0).to(torch.bfloat16)


def _forward(gu):
    g, u = gu[:, :gu.shape[1] // 2], gu[:, gu.shape[1] // 2:]
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)


def _gradient(dh, gu):
    dh = dh.float()
    g, u = gu[:, :gu.shape[1] // 2], gu[:, gu.shape[1] // 2:]
    s = 1 / (1 + torch.exp(-g))
    return torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], dim=1).to(torch.bfloat16)


def _run_swiglu(s):
    return _forward(s["gu"].float())


def _run_swiglu_pass(s):
    rows, n = s["dh"].shape
    kept = _values(*_held(s["gu"].reshape(2 * rows, n))).reshape(rows, 2 * n)
    return {"h": _forward(s["gu"].float()), "dgu": _gradient(s["dh"], kept)}


def _run_swiglu_gradient(s):
    rows, n = s["dh"].shape
    gu = s["gu"].float() if "gu" in s else _values(s["codes"], s["exponents"]).reshape(rows, 2 * n)
    out = {"dgu": _gradient(s["dh"], gu)}
    return out | {"h": _forward(gu)} if s["case"]["again"] else out


def _run_keep(s):
    return _values(*_held(s["x"])).to(torch.bfloat16)


def _run_adapters_gradient_kept(s):
    a, b, ids = s["a"].float(), s["b"].float(), s["ids"]
    count, rank, _ = a.shape
    dy, x = s["dy"].float(), _values(s["codes"], s["exponents"])
    every = (dy @ b.reshape(count * rank, -1).t()).reshape(-1, count, rank)
    g = _spread(every * s["scales"][None, :, None], ids, count).reshape(-1, count * rank)
    u = _spread(s["u"][:, None, :] * s["scales"][None, :, None], ids, count)
    u = u.reshape(-1, count * rank)
    dx = s["base"].float() + g @ a.reshape(count * rank, -1)
    return {"dx": dx.to(torch.bfloat16),
            "da": (g.t() @ x).reshape(a.shape).to(torch.bfloat16),
            "db": (u.t() @ dy).reshape(b.shape).to(torch.bfloat16)}


def _own(s):
    from dequant_gemm_trellis_amd import synth, trellis

    case, op = s["case"], s["case"]["op"]
    if op == "layer":
        hidden, inter = case["hidden"], case["inter"]
        up = synth.Shape(1, 256, 12, case["k"], hidden, 2 * inter)
        down = synth.Shape(case["axis_down"], 256, 12, case["k_down"], inter, hidden)
        return trellis.experts_mlp(s["x"], s["ids"], s["w"], s["up"], s["down"], up, down)
    if op == "keep":
        return trellis.restore(trellis.keep(s["x"]))
    if op == "adapters_gradient_kept":
        x = trellis.Kept(s["codes"], s["exponents"])
        dx, da, db = trellis.adapters_backward(s["dy"], x, s["u"], s["ids"], s["a"], s["b"],
                                               s["scales"], base=s["base"])
        return {"dx": dx, "da": da, "db": db}
    if op == "swiglu":
        return trellis.swiglu(s["gu"])[0]
    if op == "swiglu_pass":
        h, kept = trellis.swiglu(s["gu"], keep=True)
        return {"h": h, "dgu": trellis.swiglu_backward(s["dh"], kept)[0]}
    gu = s["gu"] if "gu" in s else trellis.Kept(s["codes"], s["exponents"])
    dgu, h = trellis.swiglu_backward(s["dh"], gu, again=case["again"])
    return {"dgu": dgu, "h": h} if case["again"] else {"dgu": dgu}


def run(state):
    if own:
        return _own(state)
    return globals()["_run_" + state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------


def work(case):
    op = case["op"]
    if op == "layer":
        slots = case["tokens"] * case["top_k"]
        one = case["hidden"] * case["inter"]
        stored = case["hidden"] if case["axis_down"] == 1 else case["inter"]
        expert = one * (2 * case["k"] + case["k_down"]) // 8 + 4 * (2 * case["inter"] + stored)
        return {"bytes": min(case["experts"], slots) * expert + 4 * case["tokens"] * case["hidden"]
                + 8 * slots + 32768, "flops": 6 * slots * one}
    if op == "adapters_gradient_kept":
        m, i, o, r, n = (case[x] for x in ("rows", "in", "out", "rank", "count"))
        return {"bytes": 2 * (m * o + 2 * m * i + (min(n, m) + n) * r * (i + o)) + m * i + m * -(-i // 32)
                + 4 * m * (r + 1), "flops": 4 * m * r * (i + o)}
    if op == "keep":
        values, groups = case["rows"] * case["width"], case["rows"] * -(-case["width"] // 32)
        return {"bytes": 4 * values + 2 * (values + groups), "flops": 4 * values}
    values = case["rows"] * case["inter"]
    held = 2 * (values + case["rows"] * -(-case["inter"] // 32))
    if op == "swiglu":
        return {"bytes": 6 * values, "flops": 6 * values}
    if op == "swiglu_pass":
        return {"bytes": 6 * values + 2 * held + 6 * values, "flops": 24 * values}
    return {"bytes": 6 * values + (held if case["kept"] else 4 * values) + (2 * values if case["again"] else 0),
            "flops": 16 * values}


# ---- the definitions in float64 ---------------------------------------------------


def _exact_weights(codes, scales, lut, k):
    """One expert's weights, each window read bit by bit."""
    at = torch.arange(256, device=codes.device)
    words = codes.reshape(codes.shape[0], -1, 8 * k, 1)
    bits = ((words >> torch.arange(32, device=codes.device, dtype=torch.int32)) & 1)
    bits = bits.reshape(words.shape[0], words.shape[1], 256 * k)
    index = torch.zeros((words.shape[0], words.shape[1], 256), dtype=torch.long, device=codes.device)
    for n in range(12):
        index += bits[..., ((255 - at) * k + n) % (256 * k)].long() << n
    # a weight is the float32 product rounded to bf16, by definition
    return torch.mul(lut[index.reshape(words.shape[0], -1)], scales[:, None]).bfloat16().double()


def _exact_layer(s):
    case, n = s["case"], s["case"]["inter"]
    (uc, us, ul), (dc, ds, dl) = s["up"], s["down"]
    ids, w = s["ids"].tolist(), s["w"].double().tolist()
    out = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        rows = [m for m, row in enumerate(ids) if e in row]
        if not rows:
            continue
        share = torch.tensor([sum(v for i, v in zip(ids[m], w[m]) if i == e) for m in rows],
                             dtype=torch.float64, device="cuda")
        at = torch.tensor(rows, dtype=torch.long, device="cuda")
        gu = torch.mm(s["x"][at].double(), _exact_weights(uc[e], us[e], ul, case["k"]).t().contiguous())
        h = share[:, None] * gu[:, :n] * torch.sigmoid(gu[:, :n]) * gu[:, n:]
        wd = _exact_weights(dc[e], ds[e], dl, case["k_down"])
        out[at] += torch.mm(h, wd.t().contiguous() if case["axis_down"] == 1 else wd)
    return out


def _exact_powers(low, high):
    return torch.tensor([2.0 ** e for e in range(low, high)], dtype=torch.float64, device="cuda")


def _exact_held(x):
    """What bf16 rows in 8 bits stand for."""
    parts, powers = [], _exact_powers(-133, 122)
    for part in torch.split(x.double(), 32, dim=1):
        top = torch.frexp(part.abs().amax(1, keepdim=True)).exponent - 1  # floor of the logarithm
        step = powers[top.long().clamp(min=-127) + 127]
        parts.append((part / step).round().clamp(-127, 127) * step)
    return torch.cat(parts, dim=1)


def _exact_values(s):
    """[g, u] as the backward pass has them."""
    rows, n = s["dh"].shape
    if s["case"]["op"] == "swiglu_pass":
        return _exact_held(s["gu"].reshape(2 * rows, n)).reshape(rows, 2 * n)
    if "gu" in s:
        return s["gu"].double()
    step = _exact_powers(-133, 122)[s["exponents"].long()[:, torch.arange(n, device="cuda") // 32]]
    return (s["codes"].double() * step).reshape(rows, 2 * n)


def _exact_swiglu_values(gu):
    g, u = gu.chunk(2, dim=1)
    return g * torch.sigmoid(g) * u


def _exact_gradient(dh, gu):
    g, u = gu.chunk(2, dim=1)
    sig, dh = torch.sigmoid(g), dh.double()
    return torch.cat([dh * u * (sig + g * sig * torch.sigmoid(-g)), dh * (g * sig)], dim=1)


def _exact_swiglu(s):
    return _exact_swiglu_values(s["gu"].double())


def _exact_swiglu_pass(s):
    return {"h": _exact_swiglu_values(s["gu"].double()), "dgu": _exact_gradient(s["dh"], _exact_values(s))}


def _exact_swiglu_gradient(s):
    gu = _exact_values(s)
    out = {"dgu": _exact_gradient(s["dh"], gu)}
    return out | {"h": _exact_swiglu_values(gu)} if s["case"]["again"] else out


def _exact_keep(s):
    return _exact_held(s["x"])


def _exact_adapters_gradient_kept(s):
    case, ids = s["case"], s["ids"].tolist()
    group = torch.arange(case["in"], device="cuda") // 32
    x = s["codes"].double() * _exact_powers(-133, 122)[s["exponents"].long()[:, group]]
    dy, dx = s["dy"].double(), s["base"].double()
    da = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(s["b"].shape, dtype=torch.float64, device="cuda")
    for a in range(case["count"]):
        rows = torch.tensor([m for m, i in enumerate(ids) if i == a], dtype=torch.long, device="cuda")
        if len(rows):
            scale = float(s["scales"][a])
            g = scale * torch.mm(dy[rows], s["b"][a].double().t().contiguous())
            dx[rows] += torch.mm(g, s["a"][a].double())
            da[a] = torch.mm(g.t().contiguous(), x[rows])
            db[a] = scale * torch.mm(s["u"][rows].double().t().contiguous(), dy[rows])
    return {"dx": dx, "da": da, "db": db}


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)
