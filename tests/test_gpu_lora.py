"""q4k_lora_add against the 64-bit oracle: |y - exact| <= 1e-5 * (|base| +
|scale| sum |B||A||x|), the header's bound (fp32 sums of up to 9728 products
in parts of at most a few hundred, products exact to 2^-21 or better)."""
import numpy as np
import pytest
import torch

import q4_weight_matmul_gb300 as q4k
from oracle import attention as O

pytestmark = pytest.mark.gpu


def make(seed, ids, n, rank, cols, rows, dtype):
    g = torch.Generator().manual_seed(seed)
    f = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"x": f(len(ids), cols), "scale": torch.rand(n, generator=g) + 0.5, "ids": ids,
            "a": [(f(n, rank, cols) * cols ** -0.5).to(dtype) for _ in rows],
            "b": [(f(n, m, rank) * 0.3).to(dtype) for m in rows], "base": [f(len(ids), m) for m in rows]}


def run(d, base="given", **kw):
    c = {k: ([t.cuda() for t in v] if isinstance(v, list) and k != "ids" else v.cuda()) for k, v in d.items()
         if k != "ids"}
    b = [None] * len(d["a"]) if base is None else c["base"]
    y = q4k.q4k_lora_add(c["x"], c["a"], c["b"], b, *q4k.q4k_lora_segments(d["ids"]), c["scale"],
                         y=b if base == "in place" else None, **kw)
    return y


def check(y, d, base="given"):
    f = lambda t: t.float().numpy()  # noqa: E731
    for m in range(len(d["a"])):
        want, mag = O.lora_add(f(d["x"]), f(d["a"][m]), f(d["b"][m]), None if base is None else f(d["base"][m]),
                               d["ids"], f(d["scale"]))
        got = y[m].cpu().double().numpy()
        assert np.all(np.abs(got - want) <= 1e-5 * mag), float(np.max(np.abs(got - want) / np.maximum(mag, 1e-300)))


def ids_of(seed, tokens, n, none=True):
    return [int(v) for v in np.random.default_rng(seed).integers(-1 if none else 0, n, tokens)]


CASES = [  # tokens, adapters, rank, cols, rows
    (1, 1, 8, 256, [1]),
    (1, 3, 16, 2560, [4096, 1024, 1024]),
    (2, 2, 64, 512, [97]),
    (7, 4, 24, 768, [130, 33]),
    (16, 1, 128, 1024, [515]),
    (33, 5, 40, 2560, [1024, 256, 256, 8]),
    (64, 17, 64, 2560, [641]),
    (100, 100, 8, 256, [40, 44]),
    (129, 2, 32, 9728, [250]),
    (300, 3, 120, 512, [323]),
    (700, 6, 16, 1280, [1000, 999]),
    (1100, 3, 32, 512, [97]),
    (1301, 5, 64, 768, [130, 33]),
    (1025, 14, 8, 1024, [70]),
    (400, 300, 8, 256, [33]),                       # more segments than one warp looks at
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_the_oracle(case, dtype):
    q4k.build()
    tokens, n, rank, cols, rows = CASES[case]
    d = make(case, ids_of(case, tokens, n, tokens > 1), n, rank, cols, rows, dtype)
    check(run(d), d)
    assert q4k.q4k_device_error() == 0


@pytest.mark.parametrize("tokens", [1, 5, 90])
def test_without_base_in_place_and_without_adapters(tokens):
    q4k.build()
    d = make(40, ids_of(40, tokens, 3, tokens > 1), 3, 16, 512, [260, 61], torch.float16)
    check(run(d, None), d, None)
    check(run(d, "in place"), d)
    d["ids"] = [-1] * tokens
    for base in ("given", "in place", None):
        y = run(d, base)
        for m in range(2):
            want = torch.zeros_like(d["base"][m]) if base is None else d["base"][m]
            assert torch.equal(y[m].cpu(), want)
    c = make(41, [-1] * tokens, 0, 16, 512, [60], torch.float16)      # no adapter is loaded at all
    assert torch.equal(run(c)[0].cpu(), c["base"][0])
    assert q4k.q4k_device_error() == 0


def test_large_and_small_activations():
    """Activations over 60 binades in one row, and rows of zeros."""
    q4k.build()
    d = make(42, [0, 1, 0, 1, -1], 2, 32, 512, [200], torch.bfloat16)
    d["x"] *= 2.0 ** torch.randint(-40, 20, d["x"].shape, generator=torch.Generator().manual_seed(1)).float()
    d["x"][2] = 0
    check(run(d), d)


def banded(seed, tokens, dtype):
    """Activations over 110 binades, by columns; one adapter sees only the small ones, one all, and one has ranks that
    see a band of columns each, so that its products spread as far, beside outputs that take only some of the ranks."""
    d = make(seed, ids_of(seed, tokens, 3), 3, 32, 512, [200, 61], dtype)
    r = np.random.default_rng(seed)
    e = r.integers(-60, 51, 512)
    d["x"] *= torch.from_numpy(2.0 ** e).float()
    d["ids"][0] = 0
    for a, b in zip(d["a"], d["b"]):
        a[0, :, torch.from_numpy(e > -35)] = 0
        low = torch.from_numpy(-60 + 100 * np.arange(32) // 32)[:, None]
        band = torch.from_numpy(e)[None]
        a[2][(band < low) | (band > low + 12)] = 0
        b[2][torch.from_numpy(r.random(b[2].shape) < 0.9)] = 0
    return d


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens", [1, 4, 16, 60, 300])
def test_small_activations_beside_large_ones(tokens, dtype):
    """The bound is against sum |B||A||x|: where A, or B, is zero at the large values, the small ones still count in full."""
    q4k.build()
    d = banded(48 + tokens, tokens, dtype)
    check(run(d, None), d, None)
    assert q4k.q4k_device_error() == 0


def test_one_large_value_in_front():
    q4k.build()
    for dtype in (torch.float16, torch.bfloat16):
        for tokens in (1, 20):
            d = make(49, [0] * tokens, 1, 8, 256, [8], dtype)
            d["x"][:, 0], d["x"][:, 1:] = 2.0 ** 30, 1.2345678
            d["a"][0][:, :, 0], d["a"][0][:, :, 2:] = 0, 0
            check(run(d, None), d, None)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens", [1, 3, 70])
def test_infinite_and_largest_activations(tokens, dtype):
    """An infinite activation gives what the definition gives, an infinity where all products agree; the largest finite
    ones (beyond what bfloat16 and tf32 round to) count as what they are; other tokens take nothing from either."""
    q4k.build()
    r = np.random.default_rng(tokens)
    d = make(50, [0] * tokens, 1, 16, 512, [67, 40], dtype)
    for a, b in zip(d["a"], d["b"]):
        a[:] = (a.abs().clamp(2.0 ** -6, 2.0 ** -2) * 2.0 ** -3).to(dtype)      # positive: A x has x's sign
        side = torch.from_numpy(np.where(r.random(b.shape[1]) < 0.5, -1.0, 1.0))[None, :, None]
        b[:] = ((b.abs() + 0.05) * side).to(dtype)                              # of one sign in a row: so have its terms
    value = {0: np.inf, 1: -np.inf, 2: float(np.finfo(np.float32).max), 3: float.fromhex("-0x1.fffep127")}
    for t in range(tokens):
        if t % 7 in value:
            d["x"][t, (97 * t + 5) % 512] = value[t % 7]
    y = run(d)
    f = lambda t: t.float().numpy()  # noqa: E731
    for m in range(2):
        with np.errstate(invalid="ignore"):
            want, mag = O.lora_add(f(d["x"]), f(d["a"][m]), f(d["b"][m]), f(d["base"][m]), d["ids"], f(d["scale"]))
        got = y[m].cpu().double().numpy()
        assert np.all(np.isinf(want[0])) and not np.any(np.isnan(want))
        far = np.isinf(want)
        assert np.array_equal(got[far], want[far])
        assert np.all(np.abs(got[~far] - want[~far]) <= 1e-5 * mag[~far])
    assert q4k.q4k_device_error() == 0


def test_indices_out_of_range_are_reported():
    q4k.build()
    d = make(43, [0, 0, 1, 1, 2, 2], 3, 16, 512, [70], torch.float16)
    c = {k: v.cuda() for k, v in d.items() if isinstance(v, torch.Tensor)}
    order, start, ad = q4k.q4k_lora_segments(d["ids"])
    order[1], ad[2] = 6, 3
    y = [torch.full((6, 70), 5.0, device="cuda")]
    q4k.q4k_lora_add(c["x"], [d["a"][0].cuda()], [d["b"][0].cuda()], [d["base"][0].cuda()], order, start, ad,
                     c["scale"], y=y)
    assert q4k.q4k_device_error() == 6 and q4k.q4k_device_error() == 0
    got = y[0].cpu()
    assert torch.all(got[1] == 5)                                   # no place of the order names token 1
    assert torch.equal(got[4:], d["base"][0][4:])                   # adapter 3 of 3: none
    f = lambda t: t.float().numpy()  # noqa: E731
    want, mag = O.lora_add(f(d["x"]), f(d["a"][0]), f(d["b"][0]), f(d["base"][0]), d["ids"], f(d["scale"]))
    for t in (0, 2, 3):
        assert np.all(np.abs(got[t].double().numpy() - want[t]) <= 1e-5 * mag[t])


@pytest.mark.parametrize("tokens", [3, 200])
def test_repeats_streams_and_graphs(tokens):
    q4k.build()
    d = make(44, ids_of(44, tokens, 4), 4, 32, 1024, [300, 300], torch.float16)
    c = {k: ([t.cuda() for t in v] if isinstance(v, list) else v.cuda()) for k, v in d.items() if k != "ids"}
    seg = q4k.q4k_lora_segments(d["ids"])
    ws = q4k.q4k_lora_workspace(tokens, 32, 2)
    ref = q4k.q4k_lora_add(c["x"], c["a"], c["b"], c["base"], *seg, c["scale"], workspace=ws)
    again = q4k.q4k_lora_add(c["x"], c["a"], c["b"], c["base"], *seg, c["scale"], workspace=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = q4k.q4k_lora_add(c["x"], c["a"], c["b"], c["base"], *seg, c["scale"])
    s.synchronize()
    y = [torch.zeros_like(t) for t in ref]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        q4k.q4k_lora_add(c["x"], c["a"], c["b"], c["base"], *seg, c["scale"], y=y, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    for m in range(2):
        assert torch.equal(ref[m], again[m]) and torch.equal(ref[m], other[m]) and torch.equal(ref[m], y[m])


@pytest.mark.parametrize("tokens", [3, 200])
def test_stream_argument_while_the_current_stream_is_busy(tokens):
    """Workspace and outputs made by the call belong to ``stream``: the current stream's next allocation gets neither."""
    q4k.build()
    d = make(47, ids_of(47, tokens, 4), 4, 32, 1024, [300, 300], torch.float16)
    c = {k: ([t.cuda() for t in v] if isinstance(v, list) else v.cuda()) for k, v in d.items() if k != "ids"}
    seg = q4k.q4k_lora_segments(d["ids"])
    need = q4k.q4k_lora_workspace(tokens, 32, 2).numel()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    torch.cuda._sleep(2_000_000)
    s.wait_stream(torch.cuda.current_stream())         # both streams start when every call has returned
    for _ in range(8):
        outs.append(q4k.q4k_lora_add(c["x"], c["a"], c["b"], c["base"], *seg, c["scale"], stream=s))
        torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    s.synchronize()
    for y in outs:
        check(y, d)
    assert q4k.q4k_device_error() == 0


def test_no_tokens_and_refusals():
    q4k.build()
    d = make(45, [], 2, 16, 512, [70], torch.float16)
    assert run(d)[0].shape == (0, 70)
    d = make(46, [0, 1], 2, 16, 512, [70], torch.float16)
    x, a, b, base, scale = d["x"].cuda(), d["a"][0].cuda(), d["b"][0].cuda(), d["base"][0].cuda(), d["scale"].cuda()
    order, start, ad = q4k.q4k_lora_segments(d["ids"])
    ok = dict(x=x, a=[a], b=[b], base=[base], order=order, seg_start=start, seg_adapter=ad, scale=scale)
    q4k.q4k_lora_add(**ok)
    for bad, err in ((dict(x=x.half()), TypeError), (dict(a=[a.float()]), TypeError), (dict(b=[b.bfloat16()]), TypeError),
                     (dict(a=[a, a]), ValueError), (dict(a=[a[:, :8]]), ValueError), (dict(base=[base[:1]]), ValueError),
                     (dict(order=order[:1]), ValueError), (dict(order=order.long()), TypeError),
                     (dict(scale=scale[:1]), ValueError), (dict(x=x[:, :256]), ValueError),
                     (dict(a=[a] * 5, b=[b] * 5, base=[base] * 5), q4k.Q4KError),
                     (dict(a=[a[:, :12].contiguous()], b=[b[:, :, :12].contiguous()]), q4k.Q4KError),
                     (dict(workspace=torch.zeros(0, dtype=torch.uint8, device="cuda")), q4k.Q4KError)):
        with pytest.raises(err):
            q4k.q4k_lora_add(**{**ok, **bad})
