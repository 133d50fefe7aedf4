"""How exact the routed experts' products are, on each of the kernels: beside the
bound of single outputs (test_gpu_moe.py), which lets half of an operand's bits
go, what is lost on average.

The measures, over the outputs of one expert's pairs, y and their exact values:
``norm`` = |y - exact| / |exact| and ``mean`` = <y - exact, exact> / <exact, exact>,
which is what all sums are too small or too large by.  Where they come from, for
weights and activations around zero, whose sums grow as the root of their length:

- activations hold 22 bits: each is off by at most 2^-23 of its superblock's (or
  row's) largest, on average a third of a square of that: norm 0.7e-7 for values
  near the largest, some 3e-7 for a normal distribution, whose largest of 2048 is
  3.5 times the rest;
- a product on the tensor cores drops what lies below its sum's last place: half
  of a place in the mean, and 1 / sqrt(12) around it.  Sums of the streaming
  kernel have 4 products: mean 1.2 2^-24.  Those of the tiles have 34 (tiles of 32
  pairs: 18), whose mean is put back by a factor; what is left around it is
  sqrt(34 / 12) 2^-23 = 2e-7 in norm, and of the mean a third at most: 3.4 2^-24;
- the ratio dmin / d within 2^-22 and its product's two parts: 2e-7 in norm.

Together sqrt(3^2 + 2^2 + 2^2) 1e-7 + 2e-7 = 6.2e-7 and fp32's sums over eight
superblocks: norm 1e-6, mean 2e-7 for a product; h is one of two products, one of
them through silu, whose relative slope is 1.2 on average: 1.5e-6 and 4.5e-7.
Activations of 11 bits are off by 2^-12 / sqrt(3) = 1.4e-4, a hundred times that
(tested on the host), sums without the factor by a mean of 3.3e-7 and 6e-7.
"""
import numpy as np
import pytest
import torch

import q4_weight_matmul_gb300 as q4k
import synth
from oracle import moe

NORM, MEAN, H_NORM, H_MEAN = 1e-6, 2e-7, 1.5e-6, 4.5e-7
ROWS, COLS = 192, 2048
# pairs of each expert: up to 8 tokens; below 10 an expert (tiles of up to 4, 8, 16 pairs); up to 24; beyond
COUNTS = {"one tile": [5, 3], "few": [16, 9, 7, 4], "small": [32, 17, 9, 16], "large": [112, 50, 129, 16]}


def around_zero(f):
    """Weights d sc (q - 7.5), of some 1 / sqrt(cols) each; Q6_K: d sc (q - 32) as drawn, smaller."""
    f = {k: v.copy() for k, v in f.items()}
    half = lambda v: v.astype(np.float16).view(np.uint16)  # noqa: E731
    d = 2e-4 * (0.5 + f["d"].view(np.float16).astype(np.float64) * 30)
    if "dmin" in f:
        f["d"], f["dmin"] = half(d), half(7.5 * half(d).view(np.float16).astype(np.float64))
        f["m"] = f["sc"].copy()
    else:
        f["d"] = half(d / 8)
    return f


def fields(experts, seed, fmt="q4_k"):
    draw = synth.q4k_fields if fmt == "q4_k" else synth.q6k_fields
    return around_zero(draw(experts * ROWS, COLS, seed))


def packed(f):
    from _gpu import pack_dev, to_dev
    if "dmin" in f:
        return pack_dev(f)
    t = to_dev(f)
    return q4k.q6k_pack(t["d"], t["sc"], t["q"])


def measures(got, want):
    got, want = got.astype(np.float64).ravel(), want.ravel()
    return np.linalg.norm(got - want) / np.linalg.norm(want), float((got - want) @ want / (want @ want))


def eleven_bits(x):
    """x as binary16 of its row's largest in [2^14, 2^15): what the first parts alone hold."""
    s = 2.0 ** (14 - np.floor(np.log2(np.abs(x).max(1, keepdims=True))))
    return ((x * s).astype(np.float16).astype(np.float64) / s).astype(np.float32)


def case(name):
    counts = COUNTS[name]
    expert = np.repeat(np.arange(len(counts)), counts).reshape(-1, 1)
    np.random.default_rng(5).shuffle(expert)
    return counts, expert, np.ones(expert.shape, np.float32)


def pieces(counts):
    ends = np.cumsum(counts)
    return [slice(e - n, e) for n, e in zip(counts, ends)]


@pytest.mark.parametrize("fmt", ["q4_k", "q6_k"])
def test_the_measures_see_activations_of_eleven_bits(fmt):
    counts, expert, weight = case("one tile")
    f, x = fields(2, 1, fmt), synth.activations(expert.size, COLS, 2)
    want = moe.down(x, f, fmt, ROWS, expert, weight, 2)[0]
    assert measures(moe.down(eleven_bits(x), f, fmt, ROWS, expert, weight, 2)[0], want)[0] > 50 * NORM
    if fmt == "q4_k":
        up = fields(2, 3)
        want = moe.gate_up(x, f, up, ROWS, expert, 2)[0]
        assert measures(moe.gate_up(eleven_bits(x), f, up, ROWS, expert, 2)[0], want)[0] > 50 * H_NORM


def route_of(expert, weight, experts):
    place, order, offsets = moe.group(expert, experts)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return q4k.MoeRoute(*(to(a) for a in (expert.astype(np.int32), weight, place, order, offsets)))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_k", "q6_k"])
@pytest.mark.parametrize("name", COUNTS)
def test_down_on_average(name, fmt):
    q4k.build()
    counts, expert, weight = case(name)
    n = len(counts)
    f, h = fields(n, 10, fmt), synth.activations(expert.size, COLS, 11)
    route = route_of(expert, weight, n)
    got = q4k.q4k_moe_down(torch.from_numpy(h).cuda(), packed(f), ROWS, route, q6k=fmt == "q6_k").cpu().numpy()
    want = moe.down(h, f, fmt, ROWS, expert, weight, n)[0]
    order = route.order.cpu().numpy()
    for e, mine in enumerate(pieces(counts)):
        norm, mean = measures(got[order[mine]], want[order[mine]])
        assert norm <= NORM and abs(mean) <= MEAN, (e, norm, mean)
    assert q4k.q4k_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", COUNTS)
def test_gate_up_on_average(name):
    q4k.build()
    counts, expert, weight = case(name)
    n = len(counts)
    gate, up, x = fields(n, 20), fields(n, 21), synth.activations(expert.size, COLS, 22)
    got = q4k.q4k_moe_gate_up(torch.from_numpy(x).cuda(), packed(gate), packed(up), ROWS, route_of(expert, weight, n))
    got, want = got.cpu().numpy(), moe.gate_up(x, gate, up, ROWS, expert, n)[0]
    for e, mine in enumerate(pieces(counts)):
        norm, mean = measures(got[mine], want[mine])
        assert norm <= H_NORM and abs(mean) <= H_MEAN, (e, norm, mean)
    assert q4k.q4k_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_k", "q6_k"])
@pytest.mark.parametrize("name", COUNTS)
def test_single_activations(name, fmt):
    """Rows with one activation of 24 bits: every bit but the last two counts, and
    the factor of the tiles' sums is all error here.

    In steps of 2^-24: the activation 2; the sum's products drop at most one last
    place (2) each, of which up to six are not zero (hi and lo of the activation,
    of its sum, and of the min); the factor 10; d or d sc times the sum, and its
    addition, 3.  Q4_K: dmin / d, times m, in two parts: 4 + 2 + 2; the sum's parts
    2; the oracle's weight 1.  Q6_K: the low parts' product, which is left out, 4.
    So 36 of
    |x| (|d| (|sc q - c| + c) + |dmin| m), c up to 8.1 sc the middle that both parts
    have taken off in the tiles, and 31 of |x d sc (q - 32)|.
    """
    q4k.build()
    counts, expert, weight = case(name)
    n = len(counts)
    r = np.random.default_rng(30)
    f, w = (lambda g: (g, packed(g)))(fields(n, 31, fmt))
    at = r.integers(0, COLS, expert.size)
    value = (r.choice((-1.0, 1.0), expert.size) * (2 ** 23 + r.integers(0, 2 ** 23, expert.size)) * 2.0 ** r.integers(-40, 10, expert.size))
    h = np.zeros((expert.size, COLS), np.float32)
    h[np.arange(expert.size), at] = value
    got = q4k.q4k_moe_down(torch.from_numpy(h).cuda(), w, ROWS, route_of(expert, weight, n), q6k=fmt == "q6_k").cpu().numpy()
    want = moe.down(h, f, fmt, ROWS, expert, weight, n)[0]
    place, seen = moe.group(expert, n)[0][:, 0], 0
    for t in range(expert.size):
        rows = slice(int(expert[t, 0]) * ROWS, (int(expert[t, 0]) + 1) * ROWS)
        k, x = at[place[t]], abs(value[place[t]])
        of = lambda a, g: a[rows, k // g].astype(np.float64)  # noqa: E731
        half = lambda a: np.abs(a[rows, k // 256].view(np.float16).astype(np.float64))  # noqa: E731
        if fmt == "q4_k":
            size = half(f["d"]) * of(f["sc"], 32) * (np.abs(of(f["q"], 1) - 8.1) + 8.1) + half(f["dmin"]) * of(f["m"], 32)
            size = 36 * size
        else:
            size = 31 * half(f["d"]) * np.abs(of(f["sc"], 16) * (of(f["q"], 1) - 32))
        assert np.all(np.abs(got[t] - want[t]) <= 2.0 ** -24 * x * size + 1e-300), t
        first = np.float64(eleven_bits(h[place[t]:place[t] + 1])[0, k])
        seen += bool(np.any(np.abs(want[t]) * abs(abs(first) / x - 1) > 2.0 ** -24 * x * size))
    assert seen > 0.9 * expert.size                                   # first parts alone would not have passed
    assert q4k.q4k_device_error() == 0
