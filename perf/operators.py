"""What the attention-block operators are measured on.

Three operators that stand between the quantised projections of a decoder
layer:

- ``heads``:  RMS norm of every query and key head, position rotation, and the
  store of the keys and values into a paged cache, from the projections' fp32
  outputs;
- ``attend``: attention of the new tokens of many requests (one token each
  when decoding, a few when verifying drafts, a chunk when reading a prompt)
  over that cache;
- ``lora``:   the low-rank adapters of many requests added to the outputs of
  projections that share one input.

``run`` computes the plain form (elementary torch operations in 32 bits) or,
where ``own`` is true, makes the framework's calls.  ``exact`` computes the
same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
THETA = 1.0e6


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of one user: 32 query and 8 key heads of 128 (latency)
        {"name": "heads decode 1", "op": "heads", "tokens": 1, "requests": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "page": 16, "dtype": "f16"},
        # one decode step of 61 users at unrelated positions, narrow heads, pairs of neighbours rotated
        {"name": "heads decode 61", "op": "heads", "tokens": 61, "requests": 61, "heads": 28, "kv_heads": 4, "dim": 64,
         "rot": 32, "interleaved": True, "page": 64, "dtype": "bf16"},
        # a prompt's step over 8192 tokens
        {"name": "heads prompt 8192", "op": "heads", "tokens": 8192, "requests": 2, "heads": 32, "kv_heads": 8,
         "dim": 128, "rot": 128, "interleaved": False, "page": 64, "dtype": "bf16"},
        # one decode step of one user about 1k tokens in (latency)
        {"name": "attend decode 1", "op": "attend", "requests": 1, "new": 1, "context": 1021, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "dtype": "f16", "out": "f32"},
        # one decode step of 64 users, contexts of many lengths up to 8192
        {"name": "attend decode 64", "op": "attend", "requests": 64, "new": 1, "context": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 32, "window": 0, "dtype": "bf16", "out": "f32"},
        # one decode step of one user at the end of a very long context
        {"name": "attend decode 131072", "op": "attend", "requests": 1, "new": 1, "context": 131072, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "dtype": "f16", "out": "f32"},
        # drafts of up to 5 tokens verified for 8 users, 7 query heads to a key head, a sliding window
        {"name": "attend drafts 8x5", "op": "attend", "requests": 8, "new": 5, "context": 4001, "heads": 28,
         "kv_heads": 4, "dim": 128, "page": 16, "window": 2048, "dtype": "f16", "out": "f32"},
        # a chunk of 512 prompt tokens over what the cache has of that prompt
        {"name": "attend chunk 512", "op": "attend", "requests": 1, "new": 512, "context": 4096, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "dtype": "f16", "out": "f16"},
        # two long prompts, chunks of up to 2048 tokens
        {"name": "attend chunks 2x2048", "op": "attend", "requests": 2, "new": 2048, "context": 16384, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "dtype": "bf16", "out": "bf16"},
        # one decode step of one user: adapters beside the query, key and value projections (latency)
        {"name": "lora decode 1 qkv", "op": "lora", "tokens": 1, "requests": 1, "adapters": 1, "rank": 16,
         "cols": 2560, "rows": "4096+1024+1024", "dtype": "f16"},
        # one decode step of 64 users with 17 adapters beside the gate and up projections
        {"name": "lora decode 64 gate up", "op": "lora", "tokens": 64, "requests": 64, "adapters": 17, "rank": 64,
         "cols": 2560, "rows": "9728+9728", "dtype": "bf16"},
        # a prompt step of 5 users beside the down projection
        {"name": "lora prompt 2049 down", "op": "lora", "tokens": 2049, "requests": 5, "adapters": 4, "rank": 32,
         "cols": 9728, "rows": "2560", "dtype": "f16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over the logarithm."""
    v = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))
    return v + 1 if v == 3072 else v


HEADS = ((32, 8, 128), (16, 8, 128), (28, 4, 128), (40, 8, 128), (8, 8, 128), (16, 1, 128), (32, 8, 64), (12, 4, 64))


def draw(rng):
    op = rng.choice(("heads", "attend", "attend", "attend", "lora"))
    dtype = rng.choice(("f16", "bf16"))
    heads, kv_heads, dim = rng.choice(HEADS)
    if op == "heads":
        tokens = _spread(rng, 1, 8191)
        return {"op": op, "tokens": tokens, "requests": tokens if tokens <= 128 else rng.randint(1, 9), "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "rot": rng.choice((dim, dim, dim // 2)),
                "interleaved": rng.random() < 0.3, "page": rng.choice((16, 32, 64, 128)), "dtype": dtype}
    if op == "attend":
        kind = rng.choice(("decode", "decode", "drafts", "chunk"))
        new = {"decode": 1, "drafts": rng.randint(2, 9), "chunk": _spread(rng, 33, 2047)}[kind]
        requests = _spread(rng, 1, 96) if kind != "chunk" else rng.randint(1, 3)
        most = min(131071, (400_000 if kind != "chunk" else 32_768) // requests)
        context = _spread(rng, max(new, min(65, most)), max(most, new))
        # the plain form holds every score: keep requests x heads x new x context within the largest case's
        context = max(new, min(context, 2_100_000_000 // (requests * heads * new)))
        return {"op": op, "requests": requests, "new": new, "context": context, "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "page": rng.choice((16, 32, 64, 128)), "window": rng.choice((0, 0, 0, 511, 1500)),
                "dtype": dtype, "out": dtype if kind == "chunk" else rng.choice(("f32", "f32", dtype))}
    tokens = _spread(rng, 1, 2048)
    cols = 256 * rng.randint(3, 38)
    rows = "+".join(str(_spread(rng, 250, 9728)) for _ in range(rng.randint(1, 3)))
    if cols == 3072:
        cols += 256
    return {"op": op, "tokens": tokens, "requests": tokens if tokens <= 128 else rng.randint(1, 9),
            "adapters": min(tokens, rng.randint(1, 20)), "rank": 8 * rng.randint(1, 8), "cols": cols, "rows": rows,
            "dtype": dtype}


# ------------------------------------------------- lengths: by the case alone
def _case_rng(case):
    return random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))


def _parts(case):
    """How the tokens of a `heads` or `lora` case are shared out among its requests."""
    n, t = case["requests"], case["tokens"]
    if n >= t:
        return [1] * t
    cuts = sorted(_case_rng(case).sample(range(1, t), n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [t])]


def _lengths(case):
    """(new tokens, keys in the cache) of each request of an `attend` case; the first has the most of both."""
    r = _case_rng(case)
    new = [case["new"]] + [r.randint(1, case["new"]) for _ in range(case["requests"] - 1)]
    low = max(1, case["context"] // 8)
    kv = [case["context"]] + [max(q, r.randint(low, case["context"])) for q in new[1:]]
    return new, kv


def _adapters(case):
    """The adapter of each token of a `lora` case, -1 where it has none; every adapter is used where tokens allow."""
    r = _case_rng(case)
    of_request = [i if i < case["adapters"] else r.randint(-1, case["adapters"] - 1) for i in range(case["requests"])]
    if case["requests"] > 1:
        r.shuffle(of_request)
    return [a for a, n in zip(of_request, _parts(case)) for _ in range(n)]


# ------------------------------------------------------------------- prepare
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _prepare_heads(case, seed):
    g, t, d = _gen(seed), case["tokens"], case["dim"]
    dtype, page, hk = DTYPES[case["dtype"]], case["page"], case["kv_heads"]
    r = random.Random(seed)
    pos, cells, base = [], [], 0
    for n in _parts(case):
        start = r.randint(0, 32768 - n)
        pos += range(start, start + n)
        first = start % page                                      # a request's tokens lie in its own pages
        cells += [base * page + first + i for i in range(n)]
        base += (first + n + page - 1) // page
    pages = base + 3
    place = torch.randperm(pages, generator=g, device="cuda")     # where each page lies in the cache
    cell = _ints(cells, torch.int64)
    slot = (place[cell // page] * page + cell % page).to(torch.int32)
    freq = THETA ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    angle = torch.arange(32768, device="cuda", dtype=torch.float64)[:, None] * freq
    return {"case": case, "q": _randn(g, t, case["heads"], d), "k": _randn(g, t, hk, d), "v": _randn(g, t, hk, d),
            "q_weight": 1 + _randn(g, d, std=0.2), "k_weight": 1 + _randn(g, d, std=0.2),
            "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(), "pos": _ints(pos), "slot": slot,
            "k_cache": _randn(g, pages, hk, page, d, dtype=dtype), "v_cache": _randn(g, pages, hk, page, d, dtype=dtype),
            "q_out": torch.empty((t, case["heads"], d), dtype=dtype, device="cuda")}


def _prepare_attend(case, seed):
    g, dtype, page = _gen(seed), DTYPES[case["dtype"]], case["page"]
    new, kv = _lengths(case)
    per = [-(-n // page) for n in kv]
    most, total = max(per), sum(per) + 5
    place = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(kv), most), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = place[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    shape = (total, case["kv_heads"], page, case["dim"])
    state = {"case": case, "q": _randn(g, starts[-1], case["heads"], case["dim"], dtype=dtype, std=1.4),
             "k_cache": _randn(g, *shape, dtype=dtype, std=1.4), "v_cache": _randn(g, *shape, dtype=dtype),
             "table": table, "cu_q": _ints(starts), "kv_len": _ints(kv),
             "out": torch.empty((starts[-1], case["heads"], case["dim"]), dtype=DTYPES[case["out"]], device="cuda")}
    if own:
        import q4_weight_matmul_gb300 as q4k
        state["workspace"] = q4k.q4k_paged_attn_workspace(state["q"], state["k_cache"], table, max_q=case["new"],
                                                          out_dtype=state["out"].dtype)
    return state


def _prepare_lora(case, seed):
    g, dtype, t = _gen(seed), DTYPES[case["dtype"]], case["tokens"]
    rows, n, r, cols = [int(v) for v in case["rows"].split("+")], case["adapters"], case["rank"], case["cols"]
    ids = _adapters(case)
    order = sorted(range(t), key=lambda i: ids[i])
    starts = [i for i in range(t) if i == 0 or ids[order[i]] != ids[order[i - 1]]]
    state = {"case": case, "x": _randn(g, t, cols), "ids": _ints(ids, torch.int64), "order": _ints(order),
             "seg_start": _ints(starts + [t]), "seg_adapter": _ints([ids[order[i]] for i in starts]),
             "scale": torch.rand(n, generator=g, device="cuda") + 0.5,
             "a": [_randn(g, n, r, cols, dtype=dtype, std=cols ** -0.5) for _ in rows],
             "b": [_randn(g, n, m, r, dtype=dtype, std=0.1) for m in rows],
             "base": [_randn(g, t, m) for m in rows],
             "y": [torch.empty((t, m), dtype=torch.float32, device="cuda") for m in rows]}
    if own:
        import q4_weight_matmul_gb300 as q4k
        state["workspace"] = q4k.q4k_lora_workspace(t, r, len(rows))
    return state


def prepare(case, seed):
    return {"heads": _prepare_heads, "attend": _prepare_attend, "lora": _prepare_lora}[case["op"]](case, seed)


# ----------------------------------------------------------------- plain form
def _norm_rotate(x, weight, cos, sin, case):
    """x [tokens][heads][dim] in 32 bits: normed per head, the first `rot` values rotated."""
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    rot = case["rot"]
    cos, sin = cos[:, None], sin[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_heads(s):
    case, dtype = s["case"], s["k_cache"].dtype
    cos, sin = s["cos_sin"][s["pos"].long()].chunk(2, -1)
    q = _norm_rotate(s["q"], s["q_weight"], cos, sin, case).to(dtype)
    k = _norm_rotate(s["k"], s["k_weight"], cos, sin, case).to(dtype)
    page, off = s["slot"].long() // case["page"], s["slot"].long() % case["page"]
    s["k_cache"][page, :, off] = k
    s["v_cache"][page, :, off] = s["v"].to(dtype)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    case = s["case"]
    q, table, cu, kv_len = s["q"], s["table"].long(), s["cu_q"].long(), s["kv_len"].long()
    n, hk, d, new = table.shape[0], case["kv_heads"], case["dim"], case["new"]
    g = case["heads"] // hk
    k = s["k_cache"][table].transpose(1, 2).reshape(n, hk, -1, d).float()
    v = s["v_cache"][table].transpose(1, 2).reshape(n, hk, -1, d).float()
    at = (cu[:-1, None] + torch.arange(new, device="cuda")).clamp_max(q.shape[0] - 1)
    qs = q[at].float().reshape(n, new, hk, g, d).permute(0, 2, 1, 3, 4).reshape(n, hk, new * g, d)
    p = torch.matmul(qs, k.transpose(2, 3)).mul_(d ** -0.5).view(n, hk, new, g, -1)
    where = (kv_len - (cu[1:] - cu[:-1]))[:, None] + torch.arange(new, device="cuda")         # a row's own position
    key = torch.arange(k.shape[2], device="cuda")
    seen = (key <= where[..., None]) & (key < kv_len[:, None, None])
    if case["window"]:
        seen &= key > where[..., None] - case["window"]
    p.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hk, new * g, -1), v).view(n, hk, new, g, d) / total.clamp_min(1e-30)
    o = o.permute(0, 2, 1, 3, 4).reshape(n, new, case["heads"], d)
    token = torch.arange(q.shape[0], device="cuda")
    req = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    return o[req, token - cu[req]].to(DTYPES[case["out"]])


def _plain_lora(s):
    n, r = s["case"]["adapters"], s["case"]["rank"]
    mine = s["ids"][:, None] == torch.arange(n, device="cuda")
    weight = (mine * s["scale"])[..., None]
    out = []
    h = [torch.matmul(s["x"], a.float().view(n * r, -1).t()).view(-1, n, r) * weight for a in s["a"]]
    out = [torch.addmm(base, z.view(-1, n * r), b.float().transpose(1, 2).reshape(n * r, -1))
           for z, b, base in zip(h, s["b"], s["base"])]
    return out


# ----------------------------------------------------------------------- run
def _own_heads(s):
    import q4_weight_matmul_gb300 as q4k
    q = q4k.q4k_qk_norm_rope(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pos"], s["slot"], s["cos_sin"],
                             q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                             interleaved=s["case"]["interleaved"], q_out=s["q_out"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    import q4_weight_matmul_gb300 as q4k
    return q4k.q4k_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu_q"], s["kv_len"],
                              max_q=s["case"]["new"], window=s["case"]["window"], out=s["out"],
                              workspace=s["workspace"])


def _own_lora(s):
    import q4_weight_matmul_gb300 as q4k
    return q4k.q4k_lora_add(s["x"], s["a"], s["b"], s["base"], s["order"], s["seg_start"], s["seg_adapter"],
                            s["scale"], y=s["y"], workspace=s["workspace"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"heads": _own_heads, "attend": _own_attend, "lora": _own_lora}[op](state)
    return {"heads": _plain_heads, "attend": _plain_attend, "lora": _plain_lora}[op](state)


# ---------------------------------------------------------------------- work
def work(case):
    if case["op"] == "heads":
        values = case["tokens"] * case["dim"] * (case["heads"] + 2 * case["kv_heads"])
        return {"bytes": values * (4 + 2) + case["tokens"] * (case["rot"] * 4 + 8) + 8 * case["dim"],
                "flops": values * 6}
    if case["op"] == "attend":
        new, kv = _lengths(case)
        keys = pairs = 0
        for q, n in zip(new, kv):
            w = case["window"] or n
            first = max(0, n - q - w + 1)                        # the first key that the first row sees
            keys += n - first
            # row i sits at n - q + i and sees min(n - q + i + 1, w) keys
            full = max(0, min(q, w - (n - q)))                   # rows that the window does not cut
            pairs += full * (n - q) + full * (full + 1) // 2 + (q - full) * w
        cell = case["kv_heads"] * case["dim"]
        rows = sum(new) * case["heads"] * case["dim"]
        return {"bytes": keys * cell * 2 * 2 + rows * (2 + (4 if case["out"] == "f32" else 2))
                + 4 * sum(-(-n // case["page"]) for n in kv) + 8 * len(kv),
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    ids, r = _adapters(case), case["rank"]
    used, having = len(set(ids) - {-1}), sum(a >= 0 for a in ids)
    rows = [int(v) for v in case["rows"].split("+")]
    return {"bytes": case["tokens"] * (case["cols"] * 4 + sum(rows) * 8 + 4)
            + 2 * used * r * (case["cols"] * len(rows) + sum(rows)),
            "flops": 2 * having * r * (case["cols"] * len(rows) + sum(rows))}


# --------------------------------------------------------------------- exact
def _exact_heads(case, s):
    pos = s["pos"].long()
    table = s["cos_sin"].double()
    half = case["rot"] // 2

    def turn(x, w):
        x = x.double()
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["dim"] + EPS) * w.double()
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        z = torch.complex(x[..., first], x[..., second])
        z = z * torch.complex(table[pos, :half], table[pos, half:])[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k, v = turn(s["k"], s["k_weight"]), s["v"].double()
    k_flat, v_flat = k_cache.transpose(1, 2).reshape(-1, *k.shape[1:]), v_cache.transpose(1, 2).reshape(-1, *k.shape[1:])
    k_flat[s["slot"].long()], v_flat[s["slot"].long()] = k, v
    back = lambda f, c: f.view(c.shape[0], c.shape[2], c.shape[1], c.shape[3]).transpose(1, 2).contiguous()  # noqa: E731
    return {"q": turn(s["q"], s["q_weight"]), "k_cache": back(k_flat, k_cache), "v_cache": back(v_flat, v_cache)}


def _exact_attend(case, s):
    new, kv = _lengths(case)
    g, page = case["heads"] // case["kv_heads"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (q, n) in enumerate(zip(new, kv)):
        cells = torch.arange(n, device="cuda")
        pages = s["table"][i].long()[cells // page]
        row, key = torch.arange(n - q, n, device="cuda")[:, None], cells[None]
        seen = key <= row
        if case["window"]:
            seen = seen & (row - key < case["window"])
        for h in range(case["kv_heads"]):
            ks, vs = s["k_cache"][pages, h, cells % page].double(), s["v_cache"][pages, h, cells % page].double()
            for j in range(h * g, h * g + g):
                z = s["q"][at:at + q, j].double() @ ks.t() / math.sqrt(case["dim"])
                z = torch.softmax(torch.where(seen, z, torch.full_like(z, -math.inf)), -1)
                out[at:at + q, j] = z @ vs
        at += q
    return out


def _exact_lora(case, s):
    out = [b.double() for b in s["base"]]
    ids = _adapters(case)
    for n in sorted(set(ids) - {-1}):
        at = _ints([i for i, a in enumerate(ids) if a == n], torch.int64)
        for y, a, b in zip(out, s["a"], s["b"]):
            y[at] += (s["x"][at].double() @ a[n].double().t()) @ b[n].double().t() * float(s["scale"][n].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"heads": _exact_heads, "attend": _exact_attend, "lora": _exact_lora}[case["op"]](case, s)
