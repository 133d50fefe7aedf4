"""The routed experts' operators against the 64-bit oracle.

Tolerances.  Routing: indices are exact; a weight is a quotient of fp32
exponentials: the argument l - top is rounded once (2^-24 |l - top| of the
weight, and exp(-x) x < 0.4), expf is within 2 steps, a lane adds at most 16
terms, five more steps add the lanes: (0.4 + 4 + 21 + 3) * 2^-24 < 3e-6.
Products: the bound that include/q4k.h states (``oracle/moe.py``).
"""
import numpy as np
import pytest
import torch

import q4_weight_matmul_gb300 as q4k
import synth
from _gpu import pack_dev, to_dev
from oracle import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    q4k.build()
    yield
    assert q4k.q4k_device_error() == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def route_of(expert, weight, experts, tokens=None):
    place, order, offsets = moe.group(expert, experts, tokens)
    return q4k.MoeRoute(*(dev(a) for a in (expert.astype(np.int32), weight.astype(np.float32), place, order, offsets)))


# ------------------------------------------------------------------ routing
def logits_of(tokens, experts, kind, seed):
    r = np.random.default_rng(seed)
    v = r.normal(size=(tokens, experts)).astype(np.float32) * 2
    if kind == "ties":
        v = np.round(v)
        v[r.random(v.shape) < 0.1] = -0.0
    elif kind == "masked":
        v[r.random(v.shape) < 0.7] = -np.inf
        v[::3] = -np.inf
        v[::6, experts // 2] = np.finfo(np.float32).min
        v[1::4, 0] = np.nan
    elif kind == "extreme":
        v[::4] = 3e38
        v[1::4, ::2] = np.inf
        v[2::4] *= 1e30
        v[3::4] = np.float32(1e-45) * r.integers(-3, 4, size=v[3::4].shape)
    return v


@pytest.mark.parametrize("tokens,experts,top_k,renorm,scale,valid,kind", [
    (1, 1, 1, True, 1.0, None, "plain"), (1, 128, 8, True, 1.0, None, "plain"), (3, 8, 2, False, 2.5, 2, "ties"),
    (31, 60, 4, False, 1.0, None, "masked"), (33, 33, 32, True, 1.0, None, "ties"),
    (128, 512, 32, False, 0.5, 100, "plain"), (129, 512, 32, False, 1.0, None, "masked"),
    (129, 64, 6, True, 1.0, 0, "plain"), (200, 257, 7, True, -1.0, 199, "extreme"),
    (1000, 128, 8, True, 1.0, 937, "ties"), (4865, 32, 4, False, 1.0, None, "masked"),
    (9800, 8, 2, True, 1.0, 9799, "ties"), (77, 160, 6, False, 1.0, None, "extreme")])
def test_route(tokens, experts, top_k, renorm, scale, valid, kind):
    logits = logits_of(tokens, experts, kind, [tokens, experts])
    n = None if valid is None else torch.tensor([valid], dtype=torch.int32, device="cuda")
    got = q4k.q4k_moe_route(dev(logits), top_k, renormalize=renorm, scale=scale, n_tokens=n)
    expert, weight, place, order, offsets = moe.route(logits, top_k, renorm, scale, valid)
    for name, want in (("expert", expert), ("offsets", offsets), ("order", order), ("place", place)):
        assert np.array_equal(getattr(got, name).cpu().numpy(), want), name
    off = np.abs(got.weight.cpu().numpy() - weight)
    assert off.max() <= 3e-6 * abs(scale)


def test_route_twice_captured_and_with_other_sizes():
    """A captured call follows the logits and the number of tokens; it leaves
    nothing of the call before."""
    work = q4k.q4k_moe_workspace(300, 4, 40)
    out = q4k.q4k_moe_route_out(300, 4, 40)
    logits, n = torch.empty((300, 40), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    logits.normal_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        q4k.q4k_moe_route(logits, 4, n_tokens=n, out=out, workspace=work)
    for live, seed in ((300, 1), (17, 2), (0, 3), (299, 4)):
        v = logits_of(300, 40, "masked", seed)
        logits.copy_(dev(v))
        n.fill_(live)
        graph.replay()
        torch.cuda.synchronize()
        want = moe.route(v, 4, n_tokens=live)
        for got, w in zip((out.expert, out.place, out.order, out.offsets), (want[0], *want[2:])):
            assert np.array_equal(got.cpu().numpy(), w)


def test_route_on_another_stream_and_bad_count():
    v = logits_of(500, 64, "plain", 5)
    logits = dev(v)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)                              # the current stream is busy
    got = q4k.q4k_moe_route(logits, 6, stream=stream)
    stream.synchronize()
    want = moe.route(v, 6)
    assert np.array_equal(got.order.cpu().numpy(), want[3])
    for bad, live in ((-5, 0), (501, 500)):
        got = q4k.q4k_moe_route(logits, 6, n_tokens=torch.tensor([bad], dtype=torch.int32, device="cuda"))
        assert q4k.q4k_device_error() == 6
        assert np.array_equal(got.place.cpu().numpy(), moe.route(v, 6, n_tokens=live)[2])


# ----------------------------------------------------------------- products
def choose(tokens, experts, top_k, how, seed):
    r = np.random.default_rng(seed)
    expert = np.argsort(r.random((tokens, experts)) + 0.3 * r.normal(size=experts), axis=1)[:, :top_k]
    if how == "one":                                           # every token has the same experts
        expert = np.tile(np.arange(experts - top_k, experts), (tokens, 1))
    elif how == "holes":                                       # pairs and whole tokens without an expert
        expert[r.random(expert.shape) < 0.4] = -1
        expert[::5] = -1
    elif how == "none":
        expert[:] = -1
    return expert, r.normal(size=expert.shape).astype(np.float32)


SHAPES = [  # tokens, experts, top_k, cols, rows, how
    (1, 1, 1, 256, 1, "any"), (1, 8, 2, 512, 70, "any"), (1, 32, 8, 2304, 33, "any"), (7, 4, 2, 768, 129, "any"),
    (8, 16, 4, 512, 128, "holes"), (9, 3, 1, 1024, 200, "one"), (17, 2, 2, 512, 260, "any"), (33, 40, 3, 256, 96, "any"),
    (64, 4, 1, 512, 64, "one"), (65, 9, 4, 768, 135, "holes"), (129, 3, 2, 512, 257, "any"), (150, 2, 1, 1280, 40, "one"),
    (300, 5, 2, 512, 130, "holes"), (400, 2, 1, 256, 128, "any"), (5, 6, 3, 256, 32, "none"), (40, 300, 2, 256, 20, "any")]


def matrices(experts, rows, cols, seed, fmt="q4_k"):
    if fmt == "q4_k":
        f = synth.q4k_fields(experts * rows, cols, seed)
        return f, pack_dev(f)
    f = synth.q6k_fields(experts * rows, cols, seed)
    d = to_dev(f)
    return f, q4k.q6k_pack(d["d"], d["sc"], d["q"])


@pytest.mark.parametrize("tokens,experts,top_k,cols,rows,how", SHAPES)
def test_gate_up(tokens, experts, top_k, cols, rows, how):
    (gf, gate), (uf, up) = (matrices(experts, rows, cols, [i, tokens, cols]) for i in (1, 2))
    x = 0.02 * synth.activations(tokens, cols, 3)
    expert, weight = choose(tokens, experts, top_k, how, 4)
    want, tol = moe.gate_up(x, gf, uf, rows, expert, experts)
    out = torch.full((tokens * top_k + 1, rows), 7.5, device="cuda")
    got = q4k.q4k_moe_gate_up(dev(x), gate, up, rows, route_of(expert, weight, experts), out=out[:-1])
    n = len(want)
    assert np.all(np.abs(got.cpu().numpy()[:n] - want) <= tol)
    assert torch.all(out[n:] == 7.5)                           # rows behind the last pair, and behind the tensor


@pytest.mark.parametrize("fmt", ["q4_k", "q6_k"])
@pytest.mark.parametrize("tokens,experts,top_k,cols,rows,how", SHAPES)
def test_down(tokens, experts, top_k, cols, rows, how, fmt):
    f, w = matrices(experts, rows, cols, [5, tokens, cols], fmt)
    h = synth.activations(tokens * top_k, cols, 6)
    expert, weight = choose(tokens, experts, top_k, how, 7)
    with_residual = tokens % 2 == 1
    res = synth.residual(tokens, rows, 8) if with_residual else None
    want, tol = moe.down(h, f, fmt, rows, expert, weight, experts, res)
    out = torch.full((tokens + 1, rows), -3.25, device="cuda")
    got = q4k.q4k_moe_down(dev(h), w, rows, route_of(expert, weight, experts), residual=None if res is None else dev(res),
                           q6k=fmt == "q6_k", out=out[:-1])
    assert np.all(np.abs(got.cpu().numpy() - want) <= tol)
    assert torch.all(out[-1] == -3.25)


def test_rows_behind_the_last_token_stay():
    tokens, live, experts, rows, cols = 21, 13, 4, 96, 512
    f, w = matrices(experts, rows, cols, 9)
    h = synth.activations(tokens * 2, cols, 10)
    expert, weight = choose(tokens, experts, 2, "any", 11)
    expert[live:] = -1
    expert[3] = -1
    want, tol = moe.down(h, f, "q4_k", rows, expert, weight, experts)
    h[2 * live - 2:] = np.nan                                  # rows that no pair has
    y = torch.full((tokens, rows), 2.0, device="cuda")
    q4k.q4k_moe_down(dev(h), w, rows, route_of(expert, weight, experts, live), out=y)
    y = y.cpu().numpy()
    assert np.all(np.abs(y[:live] - want[:live]) <= tol[:live]) and np.all(y[live:] == 2.0) and np.all(y[3] == 0.0)


@pytest.mark.parametrize("tokens", [3, 200])
def test_residual_in_place_bits_and_streams(tokens):
    """The same bits again, with y as the residual, on another stream, and from
    a graph that shares its workspace with another."""
    experts, rows, cols, k = 4, 200, 512, 2
    (gf, gate), (uf, up), (df, w) = (matrices(experts, *s, [12, i]) for i, s in
                                     enumerate(((512, cols), (512, cols), (rows, 512))))
    x = dev(0.02 * synth.activations(tokens, 512, 13))
    expert, weight = choose(tokens, experts, k, "any", 14)
    route = route_of(expert, weight, experts)
    res = dev(synth.residual(tokens, rows, 15))
    work = q4k.q4k_moe_workspace(tokens, k, experts, 512, 512)

    def both(y, work=None, stream=None):
        h = q4k.q4k_moe_gate_up(x, gate, up, 512, route, workspace=work, stream=stream)
        return h, q4k.q4k_moe_down(h, w, rows, route, residual=y, out=y, workspace=work, stream=stream)

    h0, y0 = both(res.clone())
    h1, y1 = both(res.clone(), work)
    assert torch.equal(h0, h1) and torch.equal(y0, y1)
    stream = torch.cuda.Stream()
    y2 = res.clone()
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)
    h2, _ = both(y2, stream=stream)
    stream.synchronize()
    assert torch.equal(h0, h2) and torch.equal(y0, y2)
    ys, graphs = [res.clone(), res.clone()], []
    torch.cuda.synchronize()
    for y in ys:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            both(y, work)
    for _ in range(2):
        for y, g in zip(ys, graphs):
            y.copy_(res)
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], y0) and torch.equal(ys[1], y0)


def test_a_captured_step_follows_the_routing():
    tokens, experts, k, cols, rows = 24, 8, 2, 512, 64
    (gf, gate), (uf, up) = (matrices(experts, rows, cols, [16, i]) for i in (1, 2))
    x, xd = np.zeros((tokens, cols), np.float32), torch.zeros((tokens, cols), device="cuda")
    logits = torch.zeros((tokens, experts), device="cuda")
    out = q4k.q4k_moe_route_out(tokens, k, experts)
    h, work = torch.zeros((tokens * k, rows), device="cuda"), q4k.q4k_moe_workspace(tokens, k, experts, cols, rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4k.q4k_moe_route(logits, k, out=out, workspace=work)
        q4k.q4k_moe_gate_up(xd, gate, up, rows, out, out=h, workspace=work)
    for kind, seed in (("plain", 1), ("masked", 2), ("ties", 3)):
        v = logits_of(tokens, experts, kind, seed)
        x = 0.02 * synth.activations(tokens, cols, seed)
        logits.copy_(dev(v)), xd.copy_(dev(x))
        graph.replay()
        want, tol = moe.gate_up(x, gf, uf, rows, moe.route(v, k)[0], experts)
        assert np.all(np.abs(h.cpu().numpy()[:len(want)] - want) <= tol)


def test_bad_indices_are_reported_and_skipped():
    tokens, experts, k, cols, rows = 12, 3, 2, 256, 40
    (gf, gate), (uf, up) = (matrices(experts, rows, cols, [17, i]) for i in (1, 2))
    (df, w) = matrices(experts, rows, cols, 18)
    expert, weight = choose(tokens, experts, k, "any", 19)
    good = route_of(expert, weight, experts)
    x, hd = dev(0.02 * synth.activations(tokens, cols, 20)), dev(synth.activations(tokens * k, cols, 21))
    h, y = q4k.q4k_moe_gate_up(x, gate, up, rows, good), q4k.q4k_moe_down(hd, w, rows, good)
    assert q4k.q4k_device_error() == 0

    def changed(name, at, value):
        t = getattr(good, name).clone()
        t.view(-1)[at] = value
        return good._replace(**{name: t})

    for value in (-1, tokens * k, 2 ** 31 - 1, -2 ** 31):
        got = q4k.q4k_moe_gate_up(x, gate, up, rows, changed("order", 5, value))
        assert q4k.q4k_device_error() == 6
        assert torch.equal(torch.cat([got[:5], got[6:]]), torch.cat([h[:5], h[6:]])) and torch.all(got[5] == 0)
    for value in (tokens * k, 2 ** 31 - 1, -3):
        got = q4k.q4k_moe_down(hd, w, rows, changed("place", 7, value))
        assert q4k.q4k_device_error() == 6
        assert torch.equal(torch.cat([got[:3], got[4:]]), torch.cat([y[:3], y[4:]]))
    for at, value in ((0, -4), (3, 2 ** 31 - 1), (1, -2 ** 31), (1, 2 ** 30)):
        q4k.q4k_moe_gate_up(x, gate, up, rows, changed("offsets", at, value))
        assert q4k.q4k_device_error() == 6
        q4k.q4k_moe_down(hd, w, rows, changed("offsets", at, value))
        assert q4k.q4k_device_error() == 6


def test_wide_activations():
    """Values of very different magnitude in a row, rows of zeros, rows of very
    large and very small values."""
    tokens, experts, k, cols, rows = 40, 2, 1, 768, 72
    (gf, gate), (uf, up) = (matrices(experts, rows, cols, [22, i]) for i in (1, 2))
    x = synth.activations(tokens, cols, 23)
    x[0] = 0
    x[1] *= 1e-12
    x[2] *= 1e8
    x[3] *= np.float32(10.0) ** np.random.default_rng(24).integers(-7, 1, cols)
    x[4:, :256] *= 1e-4
    expert, weight = choose(tokens, experts, k, "any", 25)
    want, tol = moe.gate_up(x, gf, uf, rows, expert, experts)
    got = q4k.q4k_moe_gate_up(dev(x), gate, up, rows, route_of(expert, weight, experts)).cpu().numpy()
    assert np.all(np.abs(got - want) <= tol)
    for fmt in ("q4_k", "q6_k"):
        f, w = matrices(experts, rows, cols, 26, fmt)
        want, tol = moe.down(x, f, fmt, rows, expert, weight, experts)
        # h lies in the order of the positions: x serves as it is
        got = q4k.q4k_moe_down(dev(x), w, rows, route_of(expert, weight, experts), q6k=fmt == "q6_k").cpu().numpy()
        assert np.all(np.abs(got - want) <= tol)


def test_refused_arguments():
    experts, k, cols, rows = 4, 2, 512, 64
    _, w = matrices(experts, rows, cols, 27)
    expert, weight = choose(5, experts, k, "any", 28)
    route = route_of(expert, weight, experts)
    x, h = torch.zeros((5, cols), device="cuda"), torch.zeros((10, cols), device="cuda")
    gate_up, down = q4k.q4k_moe_gate_up, q4k.q4k_moe_down
    with pytest.raises(TypeError):
        q4k.q4k_moe_route(torch.zeros((5, experts)), k, out=route)
    with pytest.raises(TypeError):
        q4k.q4k_moe_route(torch.zeros((5, experts), device="cuda").half(), k, out=route)
    with pytest.raises(ValueError):
        q4k.q4k_moe_route(torch.zeros((5, experts + 1), device="cuda"), k, out=route)
    with pytest.raises(ValueError):
        q4k.q4k_moe_route(torch.zeros((5, experts), device="cuda"), 1, out=route)
    with pytest.raises(ValueError):
        q4k.q4k_moe_route(torch.zeros((experts, 5), device="cuda").t(), k, out=route)
    with pytest.raises(q4k.Q4KError):
        q4k.q4k_moe_route(torch.zeros((5, experts), device="cuda"), k, scale=float("inf"))
    with pytest.raises(TypeError):
        gate_up(x.double(), w, w, rows, route)
    with pytest.raises(ValueError):
        gate_up(x, w[:-144], w, rows, route)
    with pytest.raises(ValueError):
        gate_up(x[:, ::2], w, w, rows, route)
    with pytest.raises(ValueError):
        gate_up(x[:4], w, w, rows, route)
    with pytest.raises(ValueError):
        gate_up(x, w, w, rows, route, out=torch.zeros((9, rows), device="cuda"))
    with pytest.raises(TypeError):
        gate_up(x, w, w, rows, route._replace(order=route.order.long()))
    with pytest.raises(ValueError):
        down(h[:9], w, rows, route)
    with pytest.raises(ValueError):
        down(h, w, rows, route, q6k=True)
    with pytest.raises(ValueError):
        down(h, w, rows, route, residual=torch.zeros((5, rows + 1), device="cuda"))
    with pytest.raises(q4k.Q4KError):
        down(h, w, rows, route, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    empty = q4k.q4k_moe_route(torch.zeros((0, experts), device="cuda"), k)
    assert gate_up(x[:0], w, w, rows, empty).shape == (0, rows) and down(h[:0], w, rows, empty).shape == (0, rows)
