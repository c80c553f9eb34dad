"""Workloads of the grouped operators: low-rank adapters of many requests
beside a shared projection, tokens sorted by expert and back, and the experts'
trellis-coded products.

Each case is one call (or the two calls a user makes in a row) with inputs
drawn from a seed. `run` computes it in plain float32 torch operations, or,
where `own` is set, through the package's entry points. `exact` computes the
same in float64, written from the definitions below.

Definitions (a = ids[m]; rows with a outside [0, count) take no adapter):
  adapters            u[m] = A[a] x[m],  y[m] = base[m] + s[a] B[a]^T u[m]
                      (A [count][rank][in], B [count][rank][out])
  adapters_gradient   g[m] = s[a] B[a] dy[m],  dx[m] = base[m] + A[a]^T g[m],
                      dA[a] = sum_m g[m] x[m]^T,  dB[a] = s[a] sum_m u[m] dy[m]^T
  dispatch            slots i = (token, choice) sorted by ids[i], equal ids in
                      slot order; slots with an id outside [0, experts) last
                      and dropped; out[place(i)] = x[token(i)]
  combine             out[m] = sum_j w[m][j] y[place(m, j)]
  combine_gradient    dy[place(m, j)] = w[m][j] dout[m],
                      dw[m][j] = <dout[m], y[place(m, j)]>
  experts             y[s] = W_e x[s] for the rows s of expert e, W_e decoded
                      from its trellis codes and rounded to bf16
"""
from __future__ import annotations

import torch

own = False

_ADAPTED = ((5120, 17408), (17408, 5120), (2048, 2048), (512, 4111), (1024, 300), (768, 5000))
# (axis, in, out): on axis 1 `in` is a multiple of 256, on axis 0 `out` is
_EXPERTS = ((1, 2048, 1536), (1, 1024, 768), (1, 512, 300), (1, 768, 1000),
            (0, 1536, 2048), (0, 768, 1024), (0, 300, 512), (0, 1000, 768))


def listed():
    return [
        # one request decodes a token beside the up projection of the MLP
        {"name": "adapters_token", "op": "adapters", "rows": 1, "in": 5120, "out": 17408,
         "rank": 16, "count": 8, "runs": False, "keep": False},
        # a full decode batch beside the down projection, nearly every request with its own adapter
        {"name": "adapters_decode", "op": "adapters", "rows": 32, "in": 17408, "out": 5120,
         "rank": 16, "count": 32, "runs": False, "keep": False},
        # packed prompts of a few requests, or the forward pass of training (the inner rows kept)
        {"name": "adapters_prompt", "op": "adapters", "rows": 4096, "in": 5120, "out": 17408,
         "rank": 16, "count": 4, "runs": True, "keep": True},
        # backward over a short, odd batch of a small projection
        {"name": "adapters_gradient_small", "op": "adapters_gradient", "rows": 203, "in": 512,
         "out": 4111, "rank": 8, "count": 3, "runs": True},
        # backward of one training batch: two adapters on the up projection
        {"name": "adapters_gradient", "op": "adapters_gradient", "rows": 4096, "in": 5120,
         "out": 17408, "rank": 32, "count": 2, "runs": True},
        # a decode batch on its way to the experts
        {"name": "dispatch_decode", "op": "dispatch", "tokens": 32, "top_k": 8, "experts": 128,
         "width": 2048},
        # a prompt on its way to the experts
        {"name": "dispatch_prompt", "op": "dispatch", "tokens": 8192, "top_k": 8, "experts": 128,
         "width": 2048},
        # a decode batch on its way back
        {"name": "combine_decode", "op": "combine", "tokens": 32, "top_k": 8, "experts": 128,
         "width": 2048, "weighted": True},
        # gradient of the way back over a prompt of odd length
        {"name": "combine_gradient", "op": "combine_gradient", "tokens": 4097, "top_k": 8,
         "experts": 128, "width": 2048},
        # a decode batch through the experts' stacked gate and up projections
        {"name": "experts_decode", "op": "experts", "tokens": 32, "top_k": 8, "experts": 64,
         "axis": 1, "in": 2048, "out": 1536, "k": 3},
        # a prompt through the same
        {"name": "experts_prompt", "op": "experts", "tokens": 2048, "top_k": 8, "experts": 64,
         "axis": 1, "in": 2048, "out": 1536, "k": 2},
        # the transposed product: the gradient of the case above, or an axis-0 down projection
        {"name": "experts_prompt_axis0", "op": "experts", "tokens": 2048, "top_k": 8,
         "experts": 64, "axis": 0, "in": 1536, "out": 2048, "k": 4},
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread over the logarithm."""
    return min(hi, int(lo * ((hi + 1) / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters_gradient", "dispatch", "combine",
                     "combine_gradient", "experts", "experts"])
    if op in ("adapters", "adapters_gradient"):
        i, o = rng.choice(_ADAPTED)
        c = {"op": op, "rows": _log(rng, 1, 4096), "in": i, "out": o,
             "rank": rng.choice([4, 8, 13, 16, 24, 32, 64]), "count": _log(rng, 1, 40),
             "runs": rng.random() < 0.5}
        if op == "adapters":
            c["keep"] = rng.random() < 0.5
        return c
    if op == "experts":
        axis, i, o = rng.choice(_EXPERTS)
        return {"op": op, "tokens": _log(rng, 1, 2048), "top_k": rng.randint(1, 8),
                "experts": _log(rng, 8, 64), "axis": axis, "in": i, "out": o,
                "k": rng.choice([2, 3, 4])}
    width = _log(rng, 64, 4096)
    c = {"op": op, "tokens": _log(rng, 1, 8192), "top_k": rng.randint(1, 8),
         "experts": _log(rng, 8, 256), "width": width if rng.random() < 0.3 else -(-width // 64) * 64}
    if op == "combine":
        c["weighted"] = rng.random() < 0.7
    return c


# ---- inputs -------------------------------------------------------------------


def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _normal(g, *shape, std=1.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda")
    return t.normal_(0.0, std, generator=g)


def _choices(g, case):
    """Router choices: top_k distinct experts per token, some of them more
    popular, and a few slots dropped (a full expert, a padded token)."""
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    score = _normal(g, t, e) + _normal(g, 1, e, std=0.7)
    ids = score.topk(k, dim=1).indices.to(torch.int32)
    drop = torch.rand((t, k), device="cuda", generator=g) < 0.02
    return torch.where(drop, torch.full_like(ids, -1), ids).contiguous()


def _sorted(ids, experts):
    """offsets [experts + 1], order [slots], position [slots] of the slots."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(experts, device=key.device)[None, :]).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.arange(key.numel(), device=key.device)
    live = place < offsets[-1]
    position = torch.empty_like(place)
    position[order] = torch.where(live, place, torch.full_like(place, -1))
    order = torch.where(live, order, torch.full_like(order, -1))
    return (offsets.to(torch.int32), order.to(torch.int32),
            position.to(torch.int32).reshape(ids.shape))


def prepare(case, seed):
    g = _generator(case, seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op in ("adapters", "adapters_gradient"):
        m, i, o, r, n = (case[x] for x in ("rows", "in", "out", "rank", "count"))
        if case["runs"]:  # packed sequences: each request's rows are adjacent
            cuts = torch.randint(0, m + 1, (n,), device="cuda", generator=g).sort().values
            run = torch.searchsorted(cuts, torch.arange(m, device="cuda"), right=True)
            name = torch.randint(-1 if n > 2 else 0, n, (n + 1,), device="cuda", generator=g)
            ids = name[run]
        else:
            ids = torch.randint(0, n, (m,), device="cuda", generator=g)
            if m > 4:
                ids = torch.where(torch.rand(m, device="cuda", generator=g) < 0.05, -1, ids)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["x"] = _normal(g, m, i).to(torch.bfloat16)
        s["a"] = _normal(g, n, r, i, std=i ** -0.5).to(torch.bfloat16)
        s["b"] = _normal(g, n, r, o, std=r ** -0.5).to(torch.bfloat16)
        s["scales"] = torch.rand(n, device="cuda", generator=g) * 1.5 + 0.5
        if op == "adapters":
            s["base"] = _normal(g, m, o).to(torch.bfloat16)  # the shared projection's output
        else:
            s["dy"] = _normal(g, m, o).to(torch.bfloat16)
            s["base"] = _normal(g, m, i).to(torch.bfloat16)  # the projection's share of dx
            s["u"] = _inner(s["x"], s["a"], s["ids"])        # kept by the forward pass
        return s
    ids = _choices(g, case)
    s["ids"] = ids
    if op == "dispatch":
        s["x"] = _normal(g, case["tokens"], case["width"]).to(torch.bfloat16)
        s["out"] = torch.zeros((ids.numel(), case["width"]), dtype=torch.bfloat16, device="cuda")
        return s
    offsets, order, position = _sorted(ids, case["experts"])
    if op == "experts":
        rows = case["out"] if case["axis"] == 1 else case["in"]
        cols = case["in"] if case["axis"] == 1 else case["out"]
        e, k = case["experts"], case["k"]
        words = torch.randint(-2 ** 31, 2 ** 31, (e, rows, cols * k // 32), dtype=torch.int64,
                              device="cuda", generator=g)
        s["codes"] = words.to(torch.int32)
        s["scales"] = torch.rand((e, rows), device="cuda", generator=g) + 0.5
        s["lut"] = _normal(g, 4096)
        s["x"] = _normal(g, ids.numel(), case["in"]).to(torch.bfloat16)
        s["offsets"] = offsets
        s["most"] = int((offsets[1:] - offsets[:-1]).max())
        s["y"] = torch.zeros((ids.numel(), case["out"]), dtype=torch.bfloat16, device="cuda")
        return s
    s["offsets"], s["order"], s["position"] = offsets, order, position
    s["y"] = _normal(g, ids.numel(), case["width"]).to(torch.bfloat16)
    s["w"] = torch.softmax(_normal(g, *ids.shape), dim=1)
    if op == "combine_gradient":
        s["dout"] = _normal(g, case["tokens"], case["width"]).to(torch.bfloat16)
        s["dy"] = torch.zeros_like(s["y"])
    return s


# ---- the plain forms ------------------------------------------------------------


def _spread(v, ids, count):
    """[rows, count, rank] with v[m] at adapter ids[m] and zeros elsewhere."""
    mine = ids.long()[:, None] == torch.arange(count, device=ids.device)[None, :]
    return torch.where(mine[:, :, None], v, torch.zeros_like(v))


def _inner(x, a, ids):
    """u[m] = A[ids[m]] x[m] in float32 (0 where a row has no adapter)."""
    count, rank, width = a.shape
    every = (x.float() @ a.float().reshape(count * rank, width).t()).reshape(-1, count, rank)
    return _spread(every, ids, count).sum(1)


def _run_adapters(s):
    a, b, ids = s["a"].float(), s["b"].float(), s["ids"]
    count, rank, width = b.shape
    u = _inner(s["x"], s["a"], ids)
    scaled = _spread(u[:, None, :] * s["scales"][None, :, None], ids, count)
    delta = scaled.reshape(-1, count * rank) @ b.reshape(count * rank, width)
    y = (s["base"].float() + delta).to(torch.bfloat16)
    return {"y": y, "u": u} if s["case"]["keep"] else {"y": y}


def _run_adapters_gradient(s):
    a, b, ids = s["a"].float(), s["b"].float(), s["ids"]
    count, rank, _ = a.shape
    dy, x = s["dy"].float(), s["x"].float()
    every = (dy @ b.reshape(count * rank, -1).t()).reshape(-1, count, rank)
    g = _spread(every * s["scales"][None, :, None], ids, count).reshape(-1, count * rank)
    u = _spread(s["u"][:, None, :] * s["scales"][None, :, None], ids, count)
    u = u.reshape(-1, count * rank)
    dx = s["base"].float() + g @ a.reshape(count * rank, -1)
    return {"dx": dx.to(torch.bfloat16),
            "da": (g.t() @ x).reshape(a.shape).to(torch.bfloat16),
            "db": (u.t() @ dy).reshape(b.shape).to(torch.bfloat16)}


def _run_dispatch(s):
    offsets, order, position = _sorted(s["ids"], s["case"]["experts"])
    rows = s["x"][(order.long().clamp(min=0)) // s["case"]["top_k"]]
    out = torch.where((order >= 0)[:, None], rows, s["out"])
    return {"offsets": offsets, "order": order, "position": position, "out": out}


def _run_combine(s):
    pos = s["position"].long()
    live = (pos >= 0).float()
    w = s["w"] * live if s["case"]["weighted"] else live
    rows = s["y"][pos.clamp(min=0)].float()
    return (rows * w[:, :, None]).sum(1).to(torch.bfloat16)


def _run_combine_gradient(s):
    order, pos, k = s["order"].long(), s["position"].long(), s["case"]["top_k"]
    slot = order.clamp(min=0)
    dout = s["dout"].float()
    dy = (dout[slot // k] * s["w"].reshape(-1)[slot][:, None]).to(torch.bfloat16)
    dy = torch.where((order >= 0)[:, None], dy, s["dy"])
    dots = (s["y"][pos.clamp(min=0)].float() * dout[:, None, :]).sum(2)
    return {"dy": dy, "dw": torch.where(pos >= 0, dots, torch.zeros_like(dots))}


def _weights(codes, scales, lut, k):
    """[experts, rows, cols] float32 values of the bf16 weights."""
    e, rows, words = codes.shape
    w = (codes.long() & 0xFFFFFFFF).reshape(e, rows, words // (8 * k), 8 * k)
    bit = (255 - torch.arange(256, device=codes.device)) * k
    at = bit // 32
    both = w[..., at] | (w[..., (at + 1) % (8 * k)] << 32)
    window = (both >> (bit % 32)) & 4095
    return (lut[window] * scales[:, :, None, None]).to(torch.bfloat16).float().reshape(e, rows, -1)


def _run_experts(s):
    case, offsets = s["case"], s["offsets"].long()
    e, total = case["experts"], s["x"].shape[0]
    w = _weights(s["codes"], s["scales"], s["lut"], case["k"])
    if case["axis"] == 1:
        w = w.transpose(1, 2).contiguous()
    place = torch.arange(max(1, s["most"]), device="cuda")
    src = (offsets[:-1, None] + place[None, :]).clamp(max=total - 1)
    live = place[None, :] < (offsets[1:] - offsets[:-1])[:, None]
    x = torch.where(live[:, :, None], s["x"].float()[src], torch.zeros((), device="cuda"))
    y = torch.bmm(x, w)
    row = torch.arange(total, device="cuda")
    of = (row[:, None] >= offsets[None, 1:]).sum(1)
    mine = of.clamp(max=e - 1)
    at = (row - offsets[mine]).clamp(max=max(1, s["most"]) - 1)
    return torch.where((of < e)[:, None], y[mine, at].to(torch.bfloat16), s["y"])


def _own(s):
    from dequant_gemm_trellis_amd import synth, trellis

    case, op = s["case"], s["case"]["op"]
    if op == "adapters":
        y, u = trellis.adapters(s["x"], s["ids"], s["a"], s["b"], s["scales"], base=s["base"],
                                keep_inner=case["keep"])
        return {"y": y, "u": u} if case["keep"] else {"y": y}
    if op == "adapters_gradient":
        dx, da, db = trellis.adapters_backward(s["dy"], s["x"], s["u"], s["ids"], s["a"], s["b"],
                                               s["scales"], base=s["base"])
        return {"dx": dx, "da": da, "db": db}
    if op == "dispatch":
        route = trellis.route(s["ids"], case["experts"])
        out = trellis.dispatch(s["x"], route, out=s["out"])
        return {"offsets": route.offsets, "order": route.order, "position": route.position,
                "out": out}
    if op == "experts":
        shape = synth.Shape(case["axis"], 256, 12, case["k"], case["in"], case["out"])
        return trellis.experts(s["x"], s["offsets"], s["codes"], s["scales"], s["lut"], shape,
                               y=s["y"])
    route = trellis.Route(s["offsets"], s["order"], s["position"])
    if op == "combine":
        return trellis.combine(s["y"], s["w"] if case["weighted"] else None, route)
    dy, dw = trellis.combine_backward(s["dout"], s["y"], s["w"], route, dy=s["dy"])
    return {"dy": dy, "dw": dw}


def run(state):
    if own:
        return _own(state)
    return globals()["_run_" + state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------


def work(case):
    op = case["op"]
    if op in ("adapters", "adapters_gradient"):
        m, i, o, r = case["rows"], case["in"], case["out"], case["rank"]
        used = min(case["count"], m)
        if op == "adapters":
            return {"bytes": 2 * (m * i + 2 * m * o + used * r * (i + o)) + 4 * m
                    + (4 * m * r if case["keep"] else 0),
                    "flops": 2 * m * r * (i + o)}
        return {"bytes": 2 * (m * o + 3 * m * i + used * r * (i + o) + case["count"] * r * (i + o))
                + 4 * m * (r + 1),
                "flops": 4 * m * r * (i + o)}
    slots = case["tokens"] * case["top_k"]
    if op == "experts":
        used = min(case["experts"], slots)
        return {"bytes": used * case["in"] * case["out"] * case["k"] // 8
                + 2 * slots * (case["in"] + case["out"]),
                "flops": 2 * slots * case["in"] * case["out"]}
    row = 2 * case["width"]
    if op == "dispatch":
        return {"bytes": row * (case["tokens"] + slots) + 12 * slots, "flops": 0}
    if op == "combine":
        return {"bytes": row * (case["tokens"] + slots) + 8 * slots,
                "flops": 2 * slots * case["width"]}
    return {"bytes": row * (case["tokens"] + 2 * slots) + 12 * slots,
            "flops": 3 * slots * case["width"]}


# ---- the definitions in float64 ---------------------------------------------------


def _exact_adapters(s):
    case, ids = s["case"], s["ids"].tolist()
    x, y = s["x"].double(), s["base"].double()
    u = torch.zeros((case["rows"], case["rank"]), dtype=torch.float64, device="cuda")
    for a in range(case["count"]):
        rows = torch.tensor([m for m, i in enumerate(ids) if i == a], dtype=torch.long, device="cuda")
        if len(rows):
            inner = torch.mm(x[rows], s["a"][a].double().t().contiguous())
            u[rows] = inner
            y[rows] += float(s["scales"][a]) * torch.mm(inner, s["b"][a].double())
    return {"y": y, "u": u} if case["keep"] else {"y": y}


def _exact_adapters_gradient(s):
    case, ids = s["case"], s["ids"].tolist()
    x, dy, dx = s["x"].double(), s["dy"].double(), s["base"].double()
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


def _exact_combine(s):
    pos = s["position"].tolist()
    y = torch.zeros((len(pos), s["y"].shape[1]), dtype=torch.float64, device="cuda")
    for j in range(s["case"]["top_k"]):
        live = torch.tensor([m for m, p in enumerate(pos) if p[j] >= 0], dtype=torch.long, device="cuda")
        at = torch.tensor([p[j] for p in pos if p[j] >= 0], dtype=torch.long, device="cuda")
        if len(live):
            share = s["w"][live, j].double()[:, None] if s["case"]["weighted"] else 1.0
            y[live] += share * s["y"][at].double()
    return y


def _exact_combine_gradient(s):
    pos = s["position"].tolist()
    dy, dw = s["dy"].double(), torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    for j in range(s["case"]["top_k"]):
        live = torch.tensor([m for m, p in enumerate(pos) if p[j] >= 0], dtype=torch.long, device="cuda")
        at = torch.tensor([p[j] for p in pos if p[j] >= 0], dtype=torch.long, device="cuda")
        if len(live):
            d = s["dout"][live].double()
            dy[at] = s["w"][live, j].double()[:, None] * d
            dw[live, j] = (d * s["y"][at].double()).sum(1)
    return {"dy": dy, "dw": dw}


def _exact_experts(s):
    case, k = s["case"], s["case"]["k"]
    cut = s["offsets"].tolist()
    y = s["y"].double()
    at = torch.arange(256, device="cuda")
    for e in range(case["experts"]):
        if cut[e] == cut[e + 1]:
            continue
        words = s["codes"][e].reshape(s["codes"].shape[1], -1, 8 * k, 1)
        bits = ((words >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1)
        bits = bits.reshape(words.shape[0], words.shape[1], 256 * k)
        index = torch.zeros((words.shape[0], words.shape[1], 256), dtype=torch.long, device="cuda")
        for n in range(12):
            index += bits[..., ((255 - at) * k + n) % (256 * k)].long() << n
        # a weight is the float32 product rounded to bf16, by definition
        w = torch.mul(s["lut"][index.reshape(words.shape[0], -1)], s["scales"][e][:, None])
        w = w.bfloat16().double()
        x = s["x"][cut[e]:cut[e + 1]].double()
        y[cut[e]:cut[e + 1]] = torch.mm(x, w.t().contiguous() if case["axis"] == 1 else w)
    return y


def _exact_dispatch(s):
    """Values are moved, not computed: each sorted row is its token's."""
    ids, out = s["ids"].reshape(-1).tolist(), s["out"].double()
    live = [n for n, i in enumerate(ids) if 0 <= i < s["case"]["experts"]]
    live.sort(key=lambda n: ids[n])  # equal ids keep their order
    token = torch.tensor(live, dtype=torch.long, device="cuda") // s["case"]["top_k"]
    out[:len(live)] = s["x"].double()[token]
    return {"offsets": None, "order": None, "position": None, "out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)
