"""The routed experts' products where they can go wrong: numbers of pairs around
the tiles' sizes on each of the kernels, scales and mins of any magnitude and
sign, most experts and most choices, long rows, arrays that pass 2^31, values
that are not finite, workspaces that several calls share.

Tolerances: the bounds that include/q4k.h states (``oracle/moe.py``); where the
same call is made twice, the same bits.
"""
import numpy as np
import pytest
import torch

import q4_weight_matmul_gb300 as q4k
import synth
from oracle import moe
from test_gpu_moe import choose, dev, matrices, route_of

pytestmark = pytest.mark.gpu

# pairs of each expert: below 10, up to 24, and above 24 on average (the streaming kernel, tiles of 32 pairs, of 112)
FEW = [0, 1, 2, 7, 8, 9, 15, 16, 17, 24, 0, 0]
SMALL = [1, 15, 16, 17, 31, 32, 33, 0, 64, 65, 97, 2, 3, 0, 0, 5, 6, 30, 12, 48]
LARGE = [0, 1, 15, 16, 17, 111, 112, 113, 224, 225, 128, 100]


@pytest.fixture(scope="module", autouse=True)
def built():
    q4k.build()
    yield
    assert q4k.q4k_device_error() == 0


def with_counts(counts, seed):
    expert = np.repeat(np.arange(len(counts)), counts)
    np.random.default_rng(seed).shuffle(expert)
    expert = expert.reshape(-1, 1)
    return expert, np.random.default_rng(seed + 1).normal(size=expert.shape).astype(np.float32)


def check_gate_up(gf, gate, uf, up, rows, x, expert, weight, experts):
    want, tol = moe.gate_up(x, gf, uf, rows, expert, experts)
    out = torch.full((expert.size + 1, rows), 7.5, device="cuda")
    q4k.q4k_moe_gate_up(dev(x), gate, up, rows, route_of(expert, weight, experts), out=out[:-1])
    assert np.all(np.abs(out.cpu().numpy()[:len(want)] - want) <= tol)
    assert torch.all(out[len(want):] == 7.5)


def check_down(f, w, fmt, rows, h, expert, weight, experts, res=None):
    want, tol = moe.down(h, f, fmt, rows, expert, weight, experts, res)
    out = torch.full((len(expert) + 1, rows), -3.25, device="cuda")
    q4k.q4k_moe_down(dev(h), w, rows, route_of(expert, weight, experts), residual=None if res is None else dev(res),
                     q6k=fmt == "q6_k", out=out[:-1])
    assert np.all(np.abs(out.cpu().numpy()[:-1] - want) <= tol)
    assert torch.all(out[-1] == -3.25)


@pytest.mark.parametrize("counts", [FEW, SMALL, LARGE], ids=["few", "small", "large"])
@pytest.mark.parametrize("cols,rows", [(256, 127), (512, 129), (1280, 257)])
def test_pairs_around_the_tiles(counts, cols, rows):
    expert, weight = with_counts(counts, 30)
    n, e = expert.size, len(counts)
    (gf, gate), (uf, up) = (matrices(e, rows, cols, [i, 31, cols]) for i in (1, 2))
    check_gate_up(gf, gate, uf, up, rows, 0.02 * synth.activations(n, cols, 32), expert, weight, e)
    h = synth.activations(n, cols, 33)
    for fmt in ("q4_k", "q6_k"):
        check_down(*matrices(e, rows, cols, [3, 31, cols], fmt), fmt, rows, h, expert, weight, e, synth.residual(n, rows, 34))


def scales_of(f, what, rng):
    """The fields with scales and mins of a kind; each kind has both signs."""
    f = {k: v.copy() for k, v in f.items()}
    sign = rng.choice((-1.0, 1.0), size=f["d"].shape)
    half = lambda v: v.astype(np.float16).view(np.uint16)  # noqa: E731
    d = 0.01 * sign * rng.uniform(0.5, 1.5, size=sign.shape)
    if what == "zeros":
        d *= rng.random(d.shape) < 0.5
    elif what == "subnormal":
        d *= 2.0 ** -12                                              # some 2^-19; binary16 is normal from 2^-14
    f["d"] = half(d)
    if "dmin" not in f:
        if what == "zeros":
            f["sc"][:, ::3] = 0
            f["q"][:, ::5] = 32
        elif what == "extremes":
            f["sc"][:] = rng.choice((-128, 127), size=f["sc"].shape)
            f["q"][:] = rng.choice((0, 63), size=f["q"].shape)
        return f
    other = rng.choice((-1.0, 1.0), size=d.shape)
    ratio = {"zeros": rng.choice((0.0, 1.0), size=d.shape), "subnormal": rng.choice((1.0, 1e4), size=d.shape),
             "extremes": rng.choice((15.9, 16.0, 16.1, 33.0, 1000.0), size=d.shape), "mins": 0.0 * d + 2000}[what]
    f["dmin"] = half(other * np.abs(d) * ratio + (0.01 * other if what == "zeros" else 0) * (rng.random(d.shape) < 0.3))
    if what == "mins":                                               # dmin / d from 2^13 to beyond 2^24, and d = 0
        f["d"] = half(sign * 2.0 ** rng.choice((-14, -20, -24, -40), size=d.shape))
        f["dmin"] = half(other * 2.0 ** rng.choice((-1, 3, 10), size=d.shape))
    elif what == "extremes":
        f["sc"][:] = rng.choice((0, 1, 63), size=f["sc"].shape)
        f["m"][:] = rng.choice((0, 1, 63), size=f["m"].shape)
        f["q"][:] = rng.choice((0, 15), size=f["q"].shape)
    return f


@pytest.mark.parametrize("counts", [[3, 5, 0, 9], [16, 17, 3, 28], [40, 113, 9, 90]], ids=["few", "small", "large"])
@pytest.mark.parametrize("what", ["zeros", "subnormal", "extremes", "mins"])
def test_scales_of_any_kind(counts, what):
    cols, rows = 768, 140
    expert, weight = with_counts(counts, 40)
    n, e, rng = expert.size, len(counts), np.random.default_rng(41)
    from _gpu import pack_dev, to_dev
    f = [scales_of(synth.q4k_fields(e * rows, cols, [42, i]), what, rng) for i in range(3)]
    small = 1e-3 if what == "mins" else 0.05
    check_gate_up(f[0], pack_dev(f[0]), f[1], pack_dev(f[1]), rows, np.float32(small) * synth.activations(n, cols, 43), expert,
                  weight, e)
    h = synth.activations(n, cols, 44)
    check_down(f[2], pack_dev(f[2]), "q4_k", rows, h, expert, weight, e)
    if what != "mins":
        f6 = scales_of(synth.q6k_fields(e * rows, cols, 45), what, rng)
        t = to_dev(f6)
        check_down(f6, q4k.q6k_pack(t["d"], t["sc"], t["q"]), "q6_k", rows, h, expert, weight, e)


@pytest.mark.parametrize("tokens", [1, 40, 250, 600])
def test_most_experts_and_choices(tokens):
    """512 experts, 32 of them a token: below 10 pairs an expert, up to 24, above."""
    e, k, cols, rows = 512, 32, 256, 8
    (gf, gate), (uf, up), (f, w) = (matrices(e, rows, cols, [i, 50]) for i in (1, 2, 3))
    logits = np.random.default_rng(51).normal(size=(tokens, e)).astype(np.float32)
    expert, weight = moe.route(logits, k)[:2]
    got = q4k.q4k_moe_route(dev(logits), k)
    assert np.array_equal(got.expert.cpu().numpy(), expert)
    check_gate_up(gf, gate, uf, up, rows, 0.02 * synth.activations(tokens, cols, 52), expert, weight, e)
    check_down(f, w, "q4_k", rows, synth.activations(tokens * k, cols, 53), expert, weight.astype(np.float32), e)


@pytest.mark.parametrize("tokens", [2, 24, 90])
def test_long_rows(tokens):
    cols, rows, e = 16384, 20, 2
    (gf, gate), (uf, up) = (matrices(e, rows, cols, [i, 60]) for i in (1, 2))
    expert, weight = choose(tokens, e, 1, "any", 61)
    check_gate_up(gf, gate, uf, up, rows, 0.005 * synth.activations(tokens, cols, 62), expert, weight, e)
    for fmt in ("q4_k", "q6_k"):
        check_down(*matrices(e, rows, cols, [3, 60], fmt), fmt, rows, synth.activations(tokens, cols, 63), expert, weight, e)


@pytest.mark.parametrize("tokens", [12, 70, 300])
def test_values_that_are_not_finite_stay_in_their_rows(tokens):
    e, k, cols, rows = 4, 1, 512, 100
    (_, gate), (_, up), (_, w) = (matrices(e, rows, cols, [i, 70]) for i in (1, 2, 3))
    (_, w6) = matrices(e, rows, cols, [4, 70], "q6_k")
    expert, weight = choose(tokens, e, k, "any", 71)
    route, x = route_of(expert, weight, e), 0.02 * synth.activations(tokens, cols, 72)
    bad = x.copy()
    bad[1, 7], bad[5, 300], bad[8] = np.nan, np.inf, -np.inf
    place = route.place.cpu().numpy()[:, 0]
    wrong = np.isin(np.arange(tokens), (1, 5, 8))
    good, got = (q4k.q4k_moe_gate_up(dev(v), gate, up, rows, route).cpu().numpy()[place] for v in (x, bad))
    assert np.array_equal(got[~wrong], good[~wrong]) and not np.isfinite(got[wrong]).any()
    for m, six in ((w, False), (w6, True)):
        at = np.argsort(place)                                       # h lies in the order of the positions
        good, got = (q4k.q4k_moe_down(dev(v[at]), m, rows, route, q6k=six).cpu().numpy() for v in (x, bad))
        assert np.array_equal(got[~wrong], good[~wrong]) and not np.isfinite(got[wrong]).any()


def test_magnitudes_of_any_size():
    """Rows from 1e-30 to 1e30 beside each other, on each kernel."""
    e, cols, rows = 2, 512, 64
    for tokens in (10, 40, 150):
        h = synth.activations(tokens, cols, 75) * (10.0 ** np.linspace(-30, 30, tokens, dtype=np.float32))[:, None]
        expert, weight = choose(tokens, e, 1, "any", 76)
        place = route_of(expert, weight, e).place.cpu().numpy()[:, 0]
        for fmt in ("q4_k", "q6_k"):
            check_down(*matrices(e, rows, cols, [77], fmt), fmt, rows, h[np.argsort(place)], expert, weight, e)


def test_a_larger_workspace_full_of_anything():
    """A workspace made for more tokens serves fewer, and nothing has to be cleared."""
    e, k, hidden, width = 6, 2, 512, 256
    (_, gate), (_, up), (_, w) = (matrices(e, *s, [80, i]) for i, s in enumerate(((width, hidden), (width, hidden),
                                                                                   (hidden, width))))
    work = q4k.q4k_moe_workspace(2000, k, e, hidden, width)
    for tokens in (1, 9, 31, 60, 500):
        logits, x = torch.randn((tokens, e), device="cuda"), dev(0.02 * synth.activations(tokens, hidden, 81))
        work.fill_(255)

        def layer(work=None):
            route = q4k.q4k_moe_route(logits, k, workspace=work)
            h = q4k.q4k_moe_gate_up(x, gate, up, width, route, workspace=work)
            return q4k.q4k_moe_down(h, w, hidden, route, x, workspace=work)

        assert torch.equal(layer(work), layer())


def test_graphs_of_different_steps_share_a_workspace():
    e, k, hidden, width = 4, 2, 512, 512
    (_, gate), (_, up), (_, w) = (matrices(e, hidden, hidden, [85, i]) for i in range(3))
    work, steps = q4k.q4k_moe_workspace(300, k, e, hidden, width), []
    for tokens in (300, 3, 40, 1):
        logits, x = torch.randn((tokens, e), device="cuda"), dev(0.02 * synth.activations(tokens, hidden, 86))

        def layer(work=None):
            route = q4k.q4k_moe_route(logits, k, workspace=work)
            h = q4k.q4k_moe_gate_up(x, gate, up, width, route, workspace=work)
            return q4k.q4k_moe_down(h, w, hidden, route, x, workspace=work)

        want = layer()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = layer(work)
        steps.append((graph, y, want, logits, x))
    for i in (0, 1, 2, 3, 1, 0, 3, 2):
        steps[i][1].zero_()
        steps[i][0].replay()
        assert torch.equal(steps[i][1], steps[i][2])


@pytest.mark.parametrize("tokens", [16, 2900])
def test_matrices_of_more_than_four_gigabytes(tokens):
    """512 experts of 16500 x 1024: 4.9 GB; what the last experts give."""
    e, k, cols, rows, seen = 512, 2, 1024, 16500, 40
    w = torch.zeros(e * rows * (cols // 256) * 144, dtype=torch.uint8, device="cuda")
    last = w.view(e, rows, -1)[-2:, -seen:]
    f, packed = matrices(2, seen, cols, 90)
    last.copy_(packed.view(2, seen, -1))
    expert = np.stack([np.arange(tokens) % (e - 2), np.full(tokens, e - 2) + np.arange(tokens) % 2], 1)
    weight = np.ones(expert.shape, np.float32)
    x, route = 0.02 * synth.activations(tokens, cols, 91), route_of(expert, weight, e)
    h = q4k.q4k_moe_gate_up(dev(x), w, w, rows, route)[-tokens:, -seen:].cpu().numpy()
    want, tol = moe.gate_up(x, f, f, seen, expert[:, 1:] - (e - 2), 2)
    assert np.all(np.abs(h - want) <= tol)
    y = q4k.q4k_moe_down(dev(np.repeat(x, 2, 0)), w, rows, route)[:, -seen:].cpu().numpy()
    at = route.place.cpu().numpy()[:, 1]
    mine = np.repeat(x, 2, 0)[at]                                    # the rows of h that the second choices have
    order = np.argsort(moe.group(expert[:, 1:] - (e - 2), 2)[0][:, 0])
    want, tol = moe.down(mine[order], f, "q4_k", seen, expert[:, 1:] - (e - 2), weight[:, 1:], 2)
    assert np.all(np.abs(y - want) <= tol)


def test_results_of_more_than_two_to_the_31_values():
    """570000 tokens, 2 of 5 experts, 2000 outputs: 2.28e9 values; the first and last rows."""
    tokens, e, k, cols, rows = 570000, 5, 2, 256, 2000
    (gf, gate), (uf, up), (f, w) = (matrices(e, rows, cols, [95, i]) for i in range(3))
    logits = torch.randn((tokens, e), generator=torch.Generator(device="cuda").manual_seed(96), device="cuda")
    x = torch.randn((tokens, cols), generator=torch.Generator(device="cuda").manual_seed(97), device="cuda") * 0.02
    route = q4k.q4k_moe_route(logits, k)
    h = q4k.q4k_moe_gate_up(x, gate, up, rows, route)
    expert, place = route.expert.cpu().numpy(), route.place.cpu().numpy()
    some = np.r_[0:20, tokens // 2:tokens // 2 + 20, tokens - 20:tokens]
    want, tol = moe.gate_up(x.cpu().numpy()[some], gf, uf, rows, expert[some], e)
    mine = moe.group(expert[some], e)[0]
    got = h[torch.from_numpy(place[some].astype(np.int64)).cuda()].cpu().numpy()
    assert np.all(np.abs(got - want[mine]) <= tol[mine])
    del h
    hd = torch.randn((tokens * k, cols), generator=torch.Generator(device="cuda").manual_seed(98), device="cuda")
    y = q4k.q4k_moe_down(hd, w, rows, route)
    rows_of = hd[torch.from_numpy(place[some].astype(np.int64)).cuda()].cpu().numpy()
    ours = np.zeros((mine.size, cols), np.float32)
    ours[mine.reshape(-1)] = rows_of.reshape(-1, cols)
    want, tol = moe.down(ours, f, "q4_k", rows, expert[some], route.weight.cpu().numpy()[some], e)
    assert np.all(np.abs(y[torch.from_numpy(some).cuda()].cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("tokens", [5, 300])
def test_a_place_behind_the_last_pair_is_reported(tokens):
    """The rows behind offsets[experts] of a workspace hold anything."""
    e, k, cols, rows = 3, 2, 256, 40
    _, w = matrices(e, rows, cols, 110)
    expert, weight = choose(tokens, e, k, "any", 111)
    expert[1] = -1
    good, h = route_of(expert, weight, e), dev(synth.activations(tokens * k, cols, 112))
    work = q4k.q4k_moe_workspace(tokens, k, e, rows, cols)
    work.fill_(255)
    want = q4k.q4k_moe_down(h, w, rows, good, workspace=work)
    assert q4k.q4k_device_error() == 0
    place = good.place.clone()
    place[1, 0] = int(good.offsets[-1])
    got = q4k.q4k_moe_down(h, w, rows, good._replace(place=place), workspace=work)
    assert q4k.q4k_device_error() == 6
    assert torch.equal(got, want) and torch.all(want[1] == 0)


@pytest.mark.parametrize("tokens,experts,top_k,hidden,width", [
    (12, 8, 2, 4096, 2048), (64, 128, 8, 2048, 768), (256, 64, 4, 2048, 768), (700, 16, 4, 2560, 1280)])
def test_the_same_bits_every_time(tokens, experts, top_k, hidden, width):
    """Steps with many items for every CTA, three hundred times."""
    from q4_weight_matmul_gb300.expert_block import random_experts
    g = torch.Generator(device="cuda").manual_seed(120)
    x = torch.randn((tokens, hidden), generator=g, device="cuda")
    route = q4k.q4k_moe_route(torch.randn((tokens, experts), generator=g, device="cuda"), top_k)
    for six in (False, True):
        block = random_experts(hidden, width, experts, top_k, six)
        work = q4k.q4k_moe_workspace(tokens, top_k, experts, hidden, width)

        def both():
            h = q4k.q4k_moe_gate_up(x, block.gate, block.up, width, route, workspace=work)
            return h, q4k.q4k_moe_down(h, block.down, hidden, route, x, six, workspace=work)

        want = both()
        differ = [torch.stack([(a != b).any() for a, b in zip(both(), want)]).any() for _ in range(300)]
        assert not torch.stack(differ).any()


@pytest.mark.parametrize("tokens", [12, 72, 300])
def test_scales_that_are_not_finite_spoil_their_rows(tokens):
    """NaN and infinities as d and dmin of single superblocks: the outputs of
    those rows are not finite for the pairs of that expert; all others stay."""
    from _gpu import pack_dev, to_dev
    e, cols, rows, bad = 4, 768, 100, 1
    expert, weight = with_counts([tokens // e] * e, 73)
    route, x = route_of(expert, weight, e), dev(0.02 * synth.activations(tokens, cols, 74))
    order = route.order.cpu().numpy()
    hit = expert[:, 0] == bad
    spoiled = {3: ("d", np.nan), 10: ("d", np.inf), 17: ("d", -np.inf), 24: ("dmin", np.nan), 31: ("dmin", np.inf),
               38: ("dmin", -np.inf), 45: ("d", np.nan), 99: ("d", np.nan)}

    def spoil(f):
        f = {n: v.copy() for n, v in f.items()}
        for i, (row, (name, value)) in enumerate(spoiled.items()):
            if name in f:
                f[name][bad * rows + row, i % (cols // 256)] = np.array(value, np.float16).view(np.uint16)
        return f

    def check(good, got, pairs, names):
        wrong = np.zeros(got.shape, bool)
        for row, (name, _) in spoiled.items():
            if name in names:
                wrong[pairs, row] = True
        assert np.array_equal(got[~wrong], good[~wrong])
        assert not np.isfinite(got[wrong]).any()

    (gf, gate), (uf, up), (df, w) = (matrices(e, rows, cols, [i, 78]) for i in (1, 2, 3))
    good = q4k.q4k_moe_gate_up(x, gate, up, rows, route).cpu().numpy()
    for g, u in ((pack_dev(spoil(gf)), up), (gate, pack_dev(spoil(uf)))):
        check(good, q4k.q4k_moe_gate_up(x, g, u, rows, route).cpu().numpy(), hit[order], ("d", "dmin"))
    good = q4k.q4k_moe_down(x, w, rows, route).cpu().numpy()
    check(good, q4k.q4k_moe_down(x, pack_dev(spoil(df)), rows, route).cpu().numpy(), hit, ("d", "dmin"))
    f6, w6 = matrices(e, rows, cols, [4, 78], "q6_k")
    t = to_dev(spoil(f6))
    good = q4k.q4k_moe_down(x, w6, rows, route, q6k=True).cpu().numpy()
    got = q4k.q4k_moe_down(x, q4k.q6k_pack(t["d"], t["sc"], t["q"]), rows, route, q6k=True).cpu().numpy()
    check(good, got, hit, ("d",))


@pytest.mark.parametrize("six", [False, True], ids=["q4_k", "q6_k"])
@pytest.mark.parametrize("tokens", [5, 40, 300])
def test_pairs_before_the_first_expert_are_reported(tokens, six):
    """offsets[0] > 0: no expert has the positions before it, and what a
    workspace holds there is not added up."""
    e, k, cols, rows = 3, 2, 256, 40
    f, w = matrices(e, rows, cols, 113, "q6_k" if six else "q4_k")
    (gf, gate), (uf, up) = (matrices(e, rows, cols, [i, 113]) for i in (1, 2))
    expert, weight = choose(tokens, e, k, "any", 114)
    good, h = route_of(expert, weight, e), synth.activations(tokens * k, cols, 115)
    work = q4k.q4k_moe_workspace(tokens, k, e, max(rows, cols), cols)
    first = int(good.offsets[1]) - 1                                 # all but one of the first expert's pairs
    for start in {1, max(1, first)}:
        offsets = good.offsets.clone()
        offsets[0] = start
        bad = good._replace(offsets=offsets)
        left = weight.copy()
        left.reshape(-1)[good.order.cpu().numpy()[:start]] = 0
        want, tol = moe.down(h, f, "q6_k" if six else "q4_k", rows, expert, left, e)
        work.fill_(255)
        got = q4k.q4k_moe_down(dev(h), w, rows, bad, q6k=six, workspace=work).cpu().numpy()
        assert q4k.q4k_device_error() == 6
        assert np.all(np.abs(got - want) <= tol)
        x = 0.02 * synth.activations(tokens, cols, 116)
        want, tol = moe.gate_up(x, gf, uf, rows, expert, e)
        out = torch.full((tokens * k, rows), 7.5, device="cuda")
        q4k.q4k_moe_gate_up(dev(x), gate, up, rows, bad, out=out)
        assert q4k.q4k_device_error() == 6
        assert torch.all(out[:start] == 7.5)
        assert np.all(np.abs(out.cpu().numpy() - want)[start:] <= tol[start:])
