"""The feed-forward part with routed experts (router, choice, gated products,
weighted down projections) against the same chain in 64 bits.

Tolerance, from the bounds of the calls: the router's rows have eight weights
that are not zero, so that its product in fp32 is off by at most 8 2^-24 sum
|r x| =: dl, so the choice is exact where the chosen and
the other logits lie further apart than 2 dl (asserted on the inputs), and a
weight is off by at most 2 dl of itself and 3e-6.  h is off by gate_up's bound
dh.  y is off by down's own bound, by sum_j w_j |W| dh (and 1e-4 of that: the
bound is stated for the h that it was given), and by what the weights are off
times |z|.
"""
import numpy as np
import pytest
import torch

import q4_weight_matmul_gb300 as q4k
import synth
from oracle import moe, q4k as O4, q6k as O6
from q4_weight_matmul_gb300.attention_block import Workspaces
from q4_weight_matmul_gb300.expert_block import ExpertBlock
from test_gpu_moe import matrices

pytestmark = pytest.mark.gpu
HIDDEN, WIDTH, EXPERTS, TOP_K = 512, 256, 12, 3


def tame(f):
    """Weights of about 1 / sqrt(cols) around zero."""
    f["d"] = (f["d"].view(np.float16).astype(np.float32) * 2e-2).astype(np.float16).view(np.uint16)
    if "dmin" in f:
        f["dmin"] = f["d"].copy()
        f["m"] = (f["sc"].astype(np.int32) * 15 // 2 % 64).astype(np.uint8)
    return f


def make(six):
    q4k.build()
    from _gpu import pack_dev, to_dev
    gate, up = (tame(synth.q4k_fields(EXPERTS * WIDTH, HIDDEN, [100, i])) for i in (1, 2))
    if six:
        down = tame(synth.q6k_fields(EXPERTS * HIDDEN, WIDTH, [100, 3]))
        t = to_dev(down)
        packed = q4k.q6k_pack(t["d"], t["sc"], t["q"])
    else:
        down = tame(synth.q4k_fields(EXPERTS * HIDDEN, WIDTH, [100, 3]))
        packed = pack_dev(down)
    r = np.random.default_rng(101)
    router = np.zeros((EXPERTS, HIDDEN), np.float32)
    for row in router:
        row[r.choice(HIDDEN, 8, replace=False)] = r.normal(size=8) * 8 ** -0.5
    block = ExpertBlock(torch.from_numpy(router).cuda(), pack_dev(gate), pack_dev(up), packed, WIDTH, TOP_K, six, scale=1.5)
    return block, router, gate, up, down


def reference(x, router, gate, up, down, six):
    """(y, tolerance) of the block for ``x`` (also the residual)."""
    x64, r64 = x.astype(np.float64), router.astype(np.float64)
    logits = x64 @ r64.T
    dl = (8 * 2.0 ** -24 * (np.abs(x64) @ np.abs(r64).T)).max(1)
    best = -np.sort(-logits, axis=1)[:, :TOP_K + 1]
    assert np.all(np.diff(-best, axis=1).min(1) > 2 * dl)                  # the inputs leave no choice open
    expert, weight, place = moe.route(logits, TOP_K, True, 1.5)[:3]
    h, dh = moe.gate_up(x, gate, up, WIDTH, expert, EXPERTS)
    fmt = "q6_k" if six else "q4_k"
    y, tol = moe.down(h.astype(np.float32), down, fmt, HIDDEN, expert, weight, EXPERTS, x)
    dh = dh + 2.0 ** -24 * np.abs(h)                                       # h.astype above
    mag = (lambda f, v: O6.gemv_q6k(f, v)[1]) if six else O4.magnitude_norm
    for e in range(EXPERTS):
        w = {k: v[e * HIDDEN:(e + 1) * HIDDEN] for k, v in down.items()}
        for t, j in zip(*np.nonzero(expert == e)):
            i, p = place[t, j], abs(weight[t, j])
            tol[t] += (1 + 1e-4) * p * mag(w, dh[i:i + 1].astype(np.float32))[0] * (1 + 1e-6)
            tol[t] += (2 * dl[t] * p + 3e-6 * 1.5) * mag(w, np.abs(h[i:i + 1]).astype(np.float32))[0]
    return y, tol


@pytest.mark.parametrize("six", [False, True], ids=["q4_k", "q6_k"])
def test_steps_of_all_kinds(six):
    """A prompt, a short one, decode steps of a batch and of one user, and a batch that is padded."""
    block, *rest = make(six)
    for tokens, live in ((150, 150), (60, 60), (11, 11), (1, 1), (16, 13), (90, 0)):
        x = synth.activations(tokens, HIDDEN, [102, tokens])
        want, tol = reference(x, *rest, six)
        want[live:], tol[live:] = x[live:], 0                              # rows without a token: the residual's
        n = None if live == tokens else torch.tensor([live], dtype=torch.int32, device="cuda")
        y = block(torch.from_numpy(x).cuda(), n_tokens=n).cpu().numpy()
        assert np.all(np.abs(y - want) <= tol), (tokens, live)
    assert q4k.q4k_device_error() == 0


def test_captured_steps_and_streams():
    """Graphs (with workspaces of their own, and with given ones) and direct calls on two streams beside each other."""
    block, *_ = make(False)
    for tokens, work in ((1, None), (14, Workspaces()), (200, None)):
        x = torch.from_numpy(synth.activations(tokens, HIDDEN, [103, tokens])).cuda()
        want = block(x, work=work).clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = block(x, work=work)
        side = torch.cuda.Stream()
        for _ in range(3):
            got.zero_()
            side.wait_stream(torch.cuda.current_stream())
            graph.replay()
            with torch.cuda.stream(side):
                other = block(x)
            direct = block(x)
            torch.cuda.synchronize()
            assert torch.equal(got, want) and torch.equal(direct, want) and torch.equal(other, want)
        assert set(block.work) >= {side.cuda_stream}
    with pytest.raises(RuntimeError):                                      # a graph never makes the workspaces it is given
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            block(x, work=Workspaces())
    torch.cuda.synchronize()
    assert q4k.q4k_device_error() == 0


def test_a_captured_step_follows_its_inputs():
    block, *rest = make(False)
    x, n = torch.zeros((20, HIDDEN), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    work = Workspaces()
    block(x, n_tokens=n, work=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x, n_tokens=n, work=work)
    for live in (20, 7, 0, 19):
        v = synth.activations(20, HIDDEN, [104, live])
        x.copy_(torch.from_numpy(v)), n.fill_(live)
        graph.replay()
        want, tol = reference(v, *rest, False)
        want[live:], tol[live:] = v[live:], 0
        assert np.all(np.abs(y.cpu().numpy() - want) <= tol)
    assert q4k.q4k_device_error() == 0


def test_the_layers_command_runs(capsys):
    import sys
    from q4_weight_matmul_gb300 import attention_block
    old, sys.argv = sys.argv, ["x", "--requests", "4", "--prompt", "50", "--steps", "3", "--hidden", "512", "--heads", "4",
                               "--kv-heads", "1", "--experts", "16", "--top-k", "4", "--width", "256"]
    try:
        attention_block.main()
    finally:
        sys.argv = old
    out = capsys.readouterr().out
    assert "decode step 2" in out and "nan" not in out
