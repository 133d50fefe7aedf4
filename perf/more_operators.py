"""What the operators of a layer with routed experts are measured on.

Three operators that take the place of a dense feed-forward part: a router and
the products of its experts, whose weights are quantised (Q4_K, and Q6_K for
some down projections):

- ``route``:  each token's best experts and their weights from the router's
  logits, and the (token, expert) pairs grouped by expert;
- ``gate_up``: silu(gate x) * (up x) of every pair, each expert's matrices over
  the ragged number of tokens that chose it;
- ``down``:   each token's weighted sum of its experts' down projections, with
  the residual.

``run`` computes the plain form (elementary torch operations in 32 bits) or,
where ``own`` is true, makes the framework's calls.  ``exact`` computes the
same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of one user: 8 of 128 experts (latency)
        {"name": "route decode 1", "op": "route", "tokens": 1, "valid": 1, "experts": 128, "top_k": 8, "renorm": True,
         "scale": 1.0, "coarse": False, "masked": False},
        # one decode step in a batch padded to 208, logits from a 16-bit product (ties), experts switched off
        {"name": "route decode 208", "op": "route", "tokens": 208, "valid": 187, "experts": 60, "top_k": 4,
         "renorm": False, "scale": 2.5, "coarse": True, "masked": True},
        # a prompt's step over 8192 tokens
        {"name": "route prompt 8192", "op": "route", "tokens": 8192, "valid": 8192, "experts": 128, "top_k": 8,
         "renorm": True, "scale": 1.0, "coarse": False, "masked": False},
        # one decode step of one user: 8 of 128 narrow experts (latency)
        {"name": "gate up decode 1", "op": "gate_up", "tokens": 1, "experts": 128, "top_k": 8, "cols": 2048,
         "rows": 768},
        # one decode step of 12 users: 2 of 8 wide experts
        {"name": "gate up decode 12", "op": "gate_up", "tokens": 12, "experts": 8, "top_k": 2, "cols": 4096,
         "rows": 12288},
        # one decode step of 64 users: some 4 tokens to an expert
        {"name": "gate up decode 64", "op": "gate_up", "tokens": 64, "experts": 128, "top_k": 8, "cols": 2048,
         "rows": 768},
        # a short prompt: some 50 tokens to an expert
        {"name": "gate up prompt 513", "op": "gate_up", "tokens": 513, "experts": 60, "top_k": 6, "cols": 2560,
         "rows": 1280},
        # a prompt's step over 4096 tokens: some 512 tokens to an expert
        {"name": "gate up prompt 4096", "op": "gate_up", "tokens": 4096, "experts": 32, "top_k": 4, "cols": 2560,
         "rows": 1536},
        # one decode step of one user, down projections in Q6_K (latency)
        {"name": "down decode 1 q6", "op": "down", "tokens": 1, "experts": 128, "top_k": 8, "cols": 768, "rows": 2048,
         "format": "q6_k", "residual": True},
        # one decode step of 64 users
        {"name": "down decode 64", "op": "down", "tokens": 64, "experts": 128, "top_k": 8, "cols": 768, "rows": 2048,
         "format": "q4_k", "residual": True},
        # a short prompt, Q6_K
        {"name": "down prompt 513 q6", "op": "down", "tokens": 513, "experts": 60, "top_k": 6, "cols": 1280,
         "rows": 2560, "format": "q6_k", "residual": False},
        # a prompt's step over 4096 tokens
        {"name": "down prompt 4096", "op": "down", "tokens": 4096, "experts": 32, "top_k": 4, "cols": 1536,
         "rows": 2560, "format": "q4_k", "residual": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("route", "gate_up", "gate_up", "down", "down"))
    experts = rng.choice((8, 16, 24, 32, 60, 64, 128, 160, 256))
    top_k = rng.randint(1, min(8, experts // 4))
    tokens = _spread(rng, 1, 4095)
    if op == "route":
        tokens = _spread(rng, 1, 8191)
        return {"op": op, "tokens": tokens, "valid": tokens if rng.random() < 0.7 else rng.randint(0, tokens),
                "experts": experts, "top_k": top_k, "renorm": rng.random() < 0.6,
                "scale": rng.choice((1.0, 1.0, 2.5)), "coarse": rng.random() < 0.4, "masked": rng.random() < 0.3}
    wide, narrow = 256 * rng.randint(3, 16), _spread(rng, 200, 4000)
    if op == "down":
        narrow = 256 * _spread(rng, 1, 12)
    # no more weights and no more products than the largest listed cases have
    narrow = min(narrow, 100_000_000 // (experts * wide), 15_000_000_000 // (tokens * top_k * wide))
    if op == "gate_up":
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "cols": wide, "rows": max(narrow, 64)}
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "cols": max(256, narrow // 256 * 256),
            "rows": wide - rng.choice((0, 0, 0, 3, 100)), "format": rng.choice(("q4_k", "q4_k", "q6_k")),
            "residual": rng.random() < 0.7}


# ------------------------------------------------- routing: by the case alone
def _chosen(case):
    """The experts of each token [tokens][top_k], the best first; some experts are several times as popular as others."""
    r = np.random.default_rng([case["tokens"], case["experts"], case["top_k"], case["cols"], case["rows"]])
    popular = r.normal(size=case["experts"]) * 0.7
    score = popular + r.gumbel(size=(case["tokens"], case["experts"]))
    return np.argsort(-score, axis=1, kind="stable")[:, :case["top_k"]]


# ------------------------------------------------------------------- prepare
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _bytes(g, hi, *shape):
    return torch.randint(0, hi, shape, generator=g, device="cuda", dtype=torch.uint8)


def _halves(v):
    """The bytes of 16-bit floats, an axis of two more."""
    return v.half().contiguous().view(torch.uint8).view(*v.shape, 2)


def _q4k(g, rows, cols):
    """A packed Q4_K matrix: superblocks of 144 bytes (scale and min as 16-bit floats, 12 bytes of 6-bit scales and
    mins, 128 bytes of quants) whose mins come near the middle of the quants, as in a trained matrix."""
    n = rows * cols // 256
    w = torch.empty((n, 144), dtype=torch.uint8, device="cuda")
    d = (torch.rand((n,), generator=g, device="cuda") + 0.5) * (cols ** -0.5 / 184)
    w[:, 0:2], w[:, 2:4] = _halves(d), _halves(d * 7.5)
    sc = _bytes(g, 48, n, 8) + 12
    m = sc + _bytes(g, 9, n, 8) - 4
    w[:, 4:8] = sc[:, :4] | ((sc[:, 4:] >> 4) << 6)
    w[:, 8:12] = m[:, :4] | ((m[:, 4:] >> 4) << 6)
    w[:, 12:16] = (sc[:, 4:] & 15) | ((m[:, 4:] & 15) << 4)
    w[:, 16:] = _bytes(g, 256, n, 128)
    return w.view(-1)


def _q6k(g, rows, cols):
    """A Q6_K matrix in the layout that the framework's kernels read: a row's superblocks of 208 bytes (16 signed
    scales, then for each 64 weights 32 bytes of low nibbles and 16 of high bit pairs), its scales d, zeros up to a
    multiple of 16 bytes."""
    nb = cols // 256
    pitch = (210 * nb + 15) // 16 * 16
    w = torch.zeros((rows, pitch), dtype=torch.uint8, device="cuda")
    w[:, :208 * nb] = _bytes(g, 256, rows, 208 * nb)
    d = (torch.rand((rows, nb), generator=g, device="cuda") + 0.5) * (cols ** -0.5 / 1400)
    w[:, 208 * nb:210 * nb] = _halves(d).view(rows, -1)
    return w.view(-1)


def _grouped(expert, experts):
    """(place, order, offsets) of the pairs with the experts `expert` [tokens][top_k]; negative: none."""
    flat = expert.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    order = torch.sort(key, stable=True).indices
    has = key[order] < experts
    place = torch.empty_like(order)
    place[order] = torch.where(has, torch.arange(len(order), device="cuda"), torch.full_like(order, -1))
    counts = (key[:, None] == torch.arange(experts, device="cuda")).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = torch.where(has, order, torch.full_like(order, -1))
    return place.view(expert.shape).to(torch.int32), order.to(torch.int32), offsets.to(torch.int32)


def _prepare_route(case, seed):
    g, t, e = _gen(seed), case["tokens"], case["experts"]
    logits = _randn(g, t, e) * 1.5 + _randn(g, e)
    if case["coarse"]:
        logits = logits.bfloat16().float()
    if case["masked"]:
        off = torch.rand((t, e), generator=g, device="cuda")
        logits[off < 0.5 * torch.rand((t, 1), generator=g, device="cuda")] = -math.inf
        logits[::17] = -math.inf                                  # tokens with no expert, and with one
        logits[::17, seed % e] = torch.where(torch.arange(len(logits[::17]), device="cuda") % 2 == 0, -math.inf, 0.5)
    state = {"case": case, "logits": logits, "valid": torch.tensor([case["valid"]], dtype=torch.int32, device="cuda")}
    if own:
        import q4_weight_matmul_gb300 as q4k
        state["out"] = q4k.q4k_moe_route_out(t, case["top_k"], e)
        state["workspace"] = q4k.q4k_moe_workspace(t, case["top_k"], e)
    return state


def _prepare_products(case, seed):
    g, t, e, k = _gen(seed), case["tokens"], case["experts"], case["top_k"]
    rows, cols = case["rows"], case["cols"]
    expert = torch.from_numpy(_chosen(case)).cuda().to(torch.int32)
    place, order, offsets = _grouped(expert, e)
    weight = torch.softmax(_randn(g, t, k), -1).sort(-1, descending=True).values.contiguous()
    state = {"case": case, "expert": expert, "weight": weight, "place": place, "order": order, "offsets": offsets}
    if case["op"] == "gate_up":
        state.update(x=_randn(g, t, cols), gate=_q4k(g, e * rows, cols), up=_q4k(g, e * rows, cols),
                     out=torch.empty((t * k, rows), dtype=torch.float32, device="cuda"))
    else:
        u = _randn(g, t * k, cols)
        state.update(h=u * torch.sigmoid(u) * _randn(g, t * k, cols),
                     w=_q4k(g, e * rows, cols) if case["format"] == "q4_k" else _q6k(g, e * rows, cols),
                     residual=_randn(g, t, rows) if case["residual"] else None,
                     out=torch.empty((t, rows), dtype=torch.float32, device="cuda"))
    if own:
        import q4_weight_matmul_gb300 as q4k
        state["route"] = q4k.MoeRoute(expert, weight, place, order, offsets)
        wide = (cols, rows) if case["op"] == "gate_up" else (rows, cols)
        state["workspace"] = q4k.q4k_moe_workspace(t, k, e, *wide)
    return state


def prepare(case, seed):
    return (_prepare_route if case["op"] == "route" else _prepare_products)(case, seed)


# ----------------------------------------------------------------- plain form
def _weights(packed, first, rows, cols, fmt):
    """Rows first .. first + rows - 1 of a packed matrix in 32 bits."""
    nb = cols // 256
    if fmt == "q4_k":
        b = packed.view(-1, 144)[first * nb:(first + rows) * nb]
        half = b[:, :4].contiguous().view(torch.float16).float()
        s, z, x = b[:, 4:8], b[:, 8:12], b[:, 12:16]
        sc = torch.cat([s & 63, (x & 15) | ((s >> 6) << 4)], 1).float() * half[:, :1]
        m = torch.cat([z & 63, (x >> 4) | ((z >> 6) << 4)], 1).float() * half[:, 1:]
        q = b[:, 16:].view(-1, 4, 1, 32)
        q = torch.cat([q & 15, q >> 4], 2).view(-1, 8, 32).float()
        return (q * sc[..., None] - m[..., None]).view(rows, cols)
    pitch = (210 * nb + 15) // 16 * 16
    b = packed.view(-1, pitch)[first:first + rows]
    d = b[:, 208 * nb:210 * nb].contiguous().view(torch.float16).float()
    b = b[:, :208 * nb].reshape(rows, nb, 208)
    sc = b[..., :16].contiguous().view(torch.int8).float() * d[..., None]
    c = b[..., 16:].reshape(rows, nb, 4, 48)
    low = torch.cat([c[..., :32] & 15, c[..., :32] >> 4], -1).view(rows, nb, 16, 16)
    pair = c[..., 32:].unsqueeze(-2)
    high = torch.cat([(pair >> s) & 3 for s in (0, 2, 4, 6)], -2).view(rows, nb, 16, 16) ^ 2
    q = (low | (high << 4)).float() - 32
    return (q * sc[..., None]).view(rows, cols)


def _plain_route(s):
    case, logits, k = s["case"], s["logits"], s["case"]["top_k"]
    best, expert = torch.sort(logits, dim=-1, descending=True, stable=True)
    best, expert = best[:, :k], expert[:, :k]
    live = torch.arange(logits.shape[0], device="cuda")[:, None] < s["valid"]
    has = (best > -math.inf) & live
    top = torch.where(has[:, :1], best[:, :1], torch.zeros_like(best[:, :1]))
    weight = torch.where(has, torch.exp(best - top), torch.zeros_like(best))
    total = weight.sum(-1, keepdim=True) if case["renorm"] else torch.exp(logits - top).sum(-1, keepdim=True)
    weight = torch.where(has, weight / total * case["scale"], torch.zeros_like(weight))
    expert = torch.where(has, expert, torch.full_like(expert, -1)).to(torch.int32)
    place, order, offsets = _grouped(expert, case["experts"])
    place = torch.where(live, place, torch.full_like(place, -2))
    return {"expert": expert, "weight": weight, "place": place, "order": order, "offsets": offsets}


def _plain_gate_up(s):
    case, at = s["case"], s["offsets"].tolist()
    token = s["order"].long() // case["top_k"]
    h = torch.empty((len(token), case["rows"]), dtype=torch.float32, device="cuda")
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if a < b:
            x = s["x"][token[a:b]]
            g = torch.matmul(x, _weights(s["gate"], e * case["rows"], case["rows"], case["cols"], "q4_k").t())
            u = torch.matmul(x, _weights(s["up"], e * case["rows"], case["rows"], case["cols"], "q4_k").t())
            h[a:b] = g / (1 + torch.exp(-g)) * u
    return h


def _plain_down(s):
    case, at = s["case"], s["offsets"].tolist()
    z = torch.empty((s["h"].shape[0], case["rows"]), dtype=torch.float32, device="cuda")
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if a < b:
            w = _weights(s["w"], e * case["rows"], case["rows"], case["cols"], case["format"])
            z[a:b] = torch.matmul(s["h"][a:b], w.t())
    y = torch.zeros_like(z[:case["tokens"]]) if s["residual"] is None else s["residual"]
    for j in range(case["top_k"]):
        y = y + s["weight"][:, j:j + 1] * z[s["place"][:, j].long()]
    return y


# ----------------------------------------------------------------------- run
def _own_route(s):
    import q4_weight_matmul_gb300 as q4k
    case = s["case"]
    return q4k.q4k_moe_route(s["logits"], case["top_k"], renormalize=case["renorm"], scale=case["scale"],
                             n_tokens=s["valid"], out=s["out"], workspace=s["workspace"])._asdict()


def _own_gate_up(s):
    import q4_weight_matmul_gb300 as q4k
    return q4k.q4k_moe_gate_up(s["x"], s["gate"], s["up"], s["case"]["rows"], s["route"], out=s["out"],
                               workspace=s["workspace"])


def _own_down(s):
    import q4_weight_matmul_gb300 as q4k
    return q4k.q4k_moe_down(s["h"], s["w"], s["case"]["rows"], s["route"], residual=s["residual"],
                            q6k=s["case"]["format"] == "q6_k", out=s["out"], workspace=s["workspace"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "gate_up": _own_gate_up, "down": _own_down}[op](state)
    return {"route": _plain_route, "gate_up": _plain_gate_up, "down": _plain_down}[op](state)


# ---------------------------------------------------------------------- work
def work(case):
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if case["op"] == "route":
        return {"bytes": case["valid"] * e * 4 + t * k * 16 + 4 * (e + 2), "flops": 4 * case["valid"] * e}
    rows, cols = case["rows"], case["cols"]
    used = len(np.unique(_chosen(case)))
    pairs, index = t * k, t * k * 4 + 4 * (e + 1)
    if case["op"] == "gate_up":
        return {"bytes": 2 * used * rows * (cols // 256) * 144 + 4 * (t * cols + pairs * rows) + index,
                "flops": 2 * pairs * rows * cols * 2}
    matrix = rows * (cols // 256) * (144 if case["format"] == "q4_k" else 210)
    return {"bytes": used * matrix + 4 * (pairs * cols + t * rows * (2 if case["residual"] else 1)) + 2 * index,
            "flops": 2 * pairs * rows * cols}


# --------------------------------------------------------------------- exact
def _fields(packed, first, rows, cols, fmt):
    """Rows of a packed matrix in 64 bits, sub-block by sub-block."""
    nb = cols // 256
    out = torch.empty((rows, nb, 256), dtype=torch.float64, device="cuda")
    if fmt == "q4_k":
        b = packed.view(-1, nb, 144)[first:first + rows].to(torch.int64)
        d, dmin = (packed.view(torch.float16).view(-1, nb, 72)[first:first + rows, :, i].double() for i in (0, 1))
        for j in range(8):
            if j < 4:
                sc, m = b[..., 4 + j] % 64, b[..., 8 + j] % 64
            else:
                sc = b[..., 8 + j] % 16 + b[..., j] // 64 * 16
                m = b[..., 8 + j] // 16 + b[..., 4 + j] // 64 * 16
            q = b[..., 16 + 32 * (j // 2):48 + 32 * (j // 2)]
            q = q // 16 if j % 2 else q % 16
            out[..., 32 * j:32 * j + 32] = (d * sc)[..., None] * q - (dmin * m)[..., None]
        return out.view(rows, cols)
    pitch = (210 * nb + 15) // 16 * 16
    b = packed.view(-1, pitch)[first:first + rows]
    d = packed.view(torch.float16).view(-1, pitch // 2)[first:first + rows, 104 * nb:105 * nb].double()
    b = b[:, :208 * nb].reshape(rows, nb, 208).to(torch.int64)
    for j in range(16):
        sc = b[..., j] - 256 * (b[..., j] > 127)
        c, f = 16 + 48 * (j // 4), j % 4
        low = b[..., c + 16 * (f % 2):c + 16 * (f % 2) + 16] // 16 ** (f // 2) % 16
        high = (b[..., c + 32:c + 48] // 4 ** f + 2) % 4
        out[..., 16 * j:16 * j + 16] = (d * sc)[..., None] * (low + 16 * high - 32)
    return out.view(rows, cols)


def _exact_route(case, s):
    logits = s["logits"].double().cpu().numpy()
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    expert, weight = np.full((t, k), -1, np.int32), np.zeros((t, k))
    for i in range(min(case["valid"], t)):
        best = [j for j in sorted(range(e), key=lambda j: (-logits[i, j], j))[:k] if logits[i, j] > -np.inf]
        if best:
            p = np.exp(logits[i] - logits[i, best[0]])
            expert[i, :len(best)] = best
            weight[i, :len(best)] = p[best] / (p[best].sum() if case["renorm"] else p.sum()) * case["scale"]
    place, order, at = np.full(t * k, -1, np.int32), [], [0]
    place[case["valid"] * k:] = -2
    for j in range(e):
        order += np.flatnonzero(expert.reshape(-1) == j).tolist()
        at.append(len(order))
    place[order] = np.arange(len(order))
    order = np.array(order + [-1] * (t * k - len(order)), np.int32)
    cuda = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    return {"expert": cuda(expert), "weight": cuda(weight), "place": cuda(place.reshape(t, k)), "order": cuda(order),
            "offsets": cuda(np.array(at, np.int32))}


def _exact_products(case, s):
    rows, cols, k = case["rows"], case["cols"], case["top_k"]
    chosen = _chosen(case)
    gate_up = case["op"] == "gate_up"
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    if not gate_up and s["residual"] is not None:
        out += s["residual"].double()
    n = 0
    for e in range(case["experts"]):
        token, slot = np.nonzero(chosen == e)
        if not len(token):
            continue
        mine, t = slice(n, n + len(token)), torch.from_numpy(token).cuda()
        n += len(token)
        if gate_up:
            x = s["x"][t].double()
            g, u = (x @ _fields(s[m], e * rows, rows, cols, "q4_k").t() for m in ("gate", "up"))
            out[mine] = g * torch.sigmoid(g) * u
        else:
            z = s["h"][mine].double() @ _fields(s["w"], e * rows, rows, cols, case["format"]).t()
            out[t] += z * s["weight"][t, torch.from_numpy(slot).cuda()].double()[:, None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_route if case["op"] == "route" else _exact_products)(case, s)
