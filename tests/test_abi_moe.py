"""Host-side validation of the routed experts' calls: every refusal comes
before any CUDA launch, so no GPU is needed."""
import ctypes

import numpy as np
import pytest

import q4_weight_matmul_gb300 as q4k
from oracle import moe

OK, INVALID, ALIGN, UNSUPPORTED = 0, 1, 2, 3
P = ctypes.c_void_p(0x100000)
ODD16, ODD4 = ctypes.c_void_p(0x100008), ctypes.c_void_p(0x100002)


@pytest.fixture(scope="module")
def lib():
    q4k.build()
    return q4k.lib()


def plan(**kw):
    d = dict(expert=P, weight=P, place=P, order=P, offsets=P, tokens=5, top_k=2, experts=8)
    d.update(kw)
    return ctypes.byref(q4k.MoePlan(*(d[n] for n, _ in q4k.MoePlan._fields_)))


BAD_PLAN = [(dict(tokens=-1), INVALID), (dict(tokens=2 ** 40), INVALID), (dict(top_k=0), INVALID),
            (dict(top_k=9), INVALID), (dict(top_k=33, experts=64), INVALID), (dict(experts=0), INVALID),
            (dict(experts=513), INVALID), (dict(expert=None), INVALID), (dict(weight=None), INVALID),
            (dict(place=None), INVALID), (dict(order=None), INVALID), (dict(offsets=None), INVALID),
            (dict(expert=ODD4), ALIGN), (dict(weight=ODD4), ALIGN), (dict(place=ODD4), ALIGN),
            (dict(order=ODD4), ALIGN), (dict(offsets=ODD4), ALIGN)]


def call(fn, d, kw):
    d.update(kw)
    return fn(*d.values(), None)


def test_route_refusals(lib):
    def route(**kw):
        return call(lib.q4k_moe_route, dict(logits=P, plan=plan(), renorm=1, scale=1.0, n=P, ws=P, bytes=1 << 40), kw)

    for bad, status in BAD_PLAN:
        assert route(plan=plan(**bad)) == status, bad
    for bad, status in [(dict(plan=None), INVALID), (dict(logits=None), INVALID), (dict(ws=None), INVALID),
                        (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
                        (dict(logits=ODD16), ALIGN), (dict(ws=ODD16), ALIGN), (dict(n=ODD4), ALIGN),
                        (dict(plan=plan(tokens=5000), bytes=16), INVALID),
                        (dict(plan=plan(tokens=0, expert=None), logits=None, ws=None), OK)]:
        assert route(**bad) == status, bad


def test_product_refusals(lib):
    def gate_up(**kw):
        return call(lib.q4k_moe_gate_up, dict(plan=plan(), gate=P, up=P, rows=64, cols=512, x=P, h=P, ws=P,
                                              bytes=1 << 40), kw)

    def down(**kw):
        return call(lib.q4k_moe_down, dict(plan=plan(), w=P, format=0, rows=64, cols=512, h=P, residual=P, y=P, ws=P,
                                           bytes=1 << 40), kw)

    for fn in gate_up, down:
        for bad, status in BAD_PLAN:
            assert fn(plan=plan(**bad)) == status, bad
        for bad, status in [(dict(plan=None), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
                            (dict(cols=300), INVALID), (dict(h=None), INVALID), (dict(ws=None), INVALID),
                            (dict(h=ODD16), ALIGN), (dict(ws=ODD16), ALIGN), (dict(rows=0, h=None), OK),
                            (dict(rows=2 ** 24, plan=plan(experts=512)), UNSUPPORTED),
                            (dict(plan=plan(tokens=0, order=None), h=None, ws=None), OK)]:
            assert fn(**bad) == status, bad
    for bad, status in [(dict(gate=None), INVALID), (dict(up=None), INVALID), (dict(x=None), INVALID),
                        (dict(gate=ODD16), ALIGN), (dict(up=ODD16), ALIGN), (dict(x=ODD16), ALIGN)]:
        assert gate_up(**bad) == status, bad
    for bad, status in [(dict(w=None), INVALID), (dict(y=None), INVALID), (dict(format=2), INVALID),
                        (dict(format=-1), INVALID), (dict(w=ODD16), ALIGN), (dict(residual=ODD16), ALIGN),
                        (dict(y=ODD16), ALIGN), (dict(bytes=16), INVALID)]:
        assert down(**bad) == status, bad


def test_workspace_serves_fewer_tokens_and_each_call(lib):
    ws = lib.q4k_moe_workspace_bytes
    assert ws(0, 2, 8, 256, 256) > 0 and ws(5, 2, 8, 0, 0) > 0
    assert ws(-1, 2, 8, 256, 256) == 0 and ws(5, 9, 8, 256, 256) == 0 and ws(5, 2, 513, 256, 256) == 0
    need = [ws(t, 4, 32, 1024, 512) for t in range(1, 3000)]
    assert need == sorted(need)
    for t in (1, 7, 130, 2000):
        assert ws(t, 4, 32, 1024, 512) >= ws(t, 4, 32, 0, 0)


def test_oracle_groups_by_counting():
    place, order, offsets = moe.group(np.array([[2, 0], [0, 2], [-1, -1], [1, 0], [7, 7]]), 3, tokens=4)
    assert offsets.tolist() == [0, 3, 4, 6] and order.tolist() == [1, 2, 7, 6, 0, 3] + [-1] * 4
    assert place.tolist() == [[4, 0], [1, 5], [-1, -1], [3, 2], [-2, -2]]


def test_oracle_route_by_hand():
    inf = np.inf
    logits = np.array([[1.0, 3.0, 3.0, 2.0], [-inf, np.nan, 0.0, -inf], [-inf] * 4, [inf, 0.0, inf, 1.0], [9, 8, 7, 6]])
    expert, weight, place, order, offsets = moe.route(logits, 3, n_tokens=4)
    assert expert.tolist() == [[1, 2, 3], [2, -1, -1], [-1] * 3, [0, 2, 3], [-1] * 3]
    e = np.exp(-1.0)
    assert np.allclose(weight, [[1 / (2 + e), 1 / (2 + e), e / (2 + e)], [1, 0, 0], [0] * 3, [0.5, 0.5, 0], [0] * 3])
    assert place[4].tolist() == [-2] * 3 and offsets.tolist() == [0, 1, 2, 5, 7]
    assert moe.route(logits[:1], 1, renormalize=False, scale=2.0)[1][0, 0] == pytest.approx(
        2 / (2 + e + np.exp(-2.0)))
