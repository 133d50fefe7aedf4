"""The attention block (projections, adapters, head norms, cache, attention,
output projection) against the same chain in 64 bits, for prompts and the
decode steps that follow them.

Bound: the chain rounds q, k, v and, for chunks, the attention's weights and
result to binary16 (2^-11 each, relative), with fp32 stages of 1e-4 relative
between them; a score moves by the sum of q's and k's roundings, so an output
by twice that: under 16 roundings of 2^-11 of the output's norm.
"""
import numpy as np
import pytest
import torch

import q4_weight_matmul_gb300 as q4k
from oracle import attention as A
from q4_weight_matmul_gb300.attention_block import AttentionBlock, Pages, Workspaces
import synth
from _gpu import pack_dev

pytestmark = pytest.mark.gpu
HIDDEN, HEADS, KV, DIM, RANK = 512, 8, 2, 64, 16
ROWS = {"q": (HEADS * DIM, HIDDEN), "k": (KV * DIM, HIDDEN), "v": (KV * DIM, HIDDEN), "o": (HIDDEN, HEADS * DIM)}


def make():
    q4k.build()
    fields = {n: synth.q4k_fields(r, c, [70, i]) for i, (n, (r, c)) in enumerate(ROWS.items())}
    for f in fields.values():              # weights of about 1 / sqrt(cols)
        for n in ("d", "dmin"):
            f[n] = (f[n].view(np.float16).astype(np.float32) * 2e-2).astype(np.float16).view(np.uint16)
        f["m"] = (f["sc"].astype(np.int32) * 7 // 8).astype(np.uint8)
    g = torch.Generator().manual_seed(3)
    lora = {n: ((torch.randn((2, RANK, c), generator=g) * c ** -0.5).half(),
                (torch.randn((2, r, RANK), generator=g) * 0.1).half()) for n, (r, c) in ROWS.items()}
    norms = [1 + 0.2 * torch.randn(DIM, generator=g) for _ in range(2)]
    angle = np.arange(256)[:, None] * 1e4 ** (-np.arange(0, DIM, 2) / DIM)
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    scale = torch.tensor([1.5, 0.5])
    pages = Pages(40, 16, 12)
    cache = [torch.full((40, KV, 16, DIM), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2)]
    block = AttentionBlock({n: pack_dev(f) for n, f in fields.items()}, HIDDEN, HEADS, KV, DIM,
                           [n.cuda() for n in norms], torch.from_numpy(cs).cuda(), cache,
                           {n: (a.cuda(), b.cuda()) for n, (a, b) in lora.items()}, scale.cuda())
    return block, pages, fields, lora, norms, cs, scale


def reference(x, fields, lora, norms, cs, scale, adapters, past, new, start):
    """The block's output for ``x``; ``past``: {request: [keys, values]} in 64 bits, extended here."""
    from_fields = {n: weights(f) for n, f in fields.items()}
    ys = {n: x @ from_fields[n].T for n in "qkv"}
    for n in "qkv":
        ys[n] = A.lora_add(x, lora[n][0].float().numpy(), lora[n][1].float().numpy(), ys[n], adapters, scale.numpy())[0]
    pos = np.concatenate([np.arange(start[r], start[r] + n) for r, n in new.items()])
    q = A.norm_rope(ys["q"].reshape(-1, HEADS, DIM), norms[0].numpy(), 1e-6, cs, pos, DIM, False)[0]
    k = A.norm_rope(ys["k"].reshape(-1, KV, DIM), norms[1].numpy(), 1e-6, cs, pos, DIM, False)[0]
    v = ys["v"].reshape(-1, KV, DIM)
    out, t = np.zeros_like(q), 0
    for r, n in new.items():
        p = past.setdefault(r, [np.zeros((0, KV, DIM))] * 2)
        p[:] = [np.concatenate([p[0], k[t:t + n]]), np.concatenate([p[1], v[t:t + n]])]
        for i in range(n):
            for h in range(HEADS):
                kk, vv = p[0][:start[r] + i + 1, h // (HEADS // KV)], p[1][:start[r] + i + 1, h // (HEADS // KV)]
                z = kk @ q[t + i, h] * DIM ** -0.5
                w = np.exp(z - z.max())
                out[t + i, h] = w @ vv / w.sum()
        t += n
    o = out.reshape(len(x), -1)
    y = o @ from_fields["o"].T + x
    return A.lora_add(o, lora["o"][0].float().numpy(), lora["o"][1].float().numpy(), y, adapters, scale.numpy())[0]


def weights(f):
    rows, cols = f["q"].shape
    d = np.repeat(f["d"].view(np.float16).astype(np.float64), 256, axis=1)
    dmin = np.repeat(f["dmin"].view(np.float16).astype(np.float64), 256, axis=1)
    sc, m = (np.repeat(f[n].astype(np.float64), 32, axis=1) for n in ("sc", "m"))
    return d * sc * f["q"] - dmin * m


def test_prompts_and_decode_steps():
    block, pages, fields, lora, norms, cs, scale = make()
    r = np.random.default_rng(9)
    adapter, past, start = {0: 1, 1: -1, 2: 0}, {}, {0: 0, 1: 0, 2: 0}
    for new in ({0: 70, 1: 3, 2: 40}, {0: 1, 1: 1, 2: 1}, {2: 1, 0: 1}, {1: 33, 0: 2}, {0: 1, 1: 1, 2: 1}):
        x = r.standard_normal((sum(new.values()), HIDDEN)).astype(np.float32)
        ids = [adapter[q] for q, n in new.items() for _ in range(n)]
        step = {k: v.cuda() for k, v in pages.step(new).items()}
        y = block(torch.from_numpy(x).cuda(), step, max(new.values()), q4k.q4k_lora_segments(ids))
        want = reference(x.astype(np.float64), fields, lora, norms, cs, scale, ids, past, new, dict(start))
        for q, n in new.items():
            start[q] += n
        err = np.linalg.norm(y.cpu().double().numpy() - want, axis=1) / np.linalg.norm(want, axis=1)
        assert err.max() < 16 * 2.0 ** -11, (new, err.max())
    assert q4k.q4k_device_error() == 0


def run_step(block, pages, new, seed, **kw):
    """One step of the requests ``new``; what the block gave, and the call's arguments."""
    x = torch.randn((sum(new.values()), HIDDEN), generator=torch.Generator().manual_seed(seed)).cuda()
    step = {k: v.cuda() for k, v in pages.step(new).items()}
    segments = q4k.q4k_lora_segments([r % 3 - 1 for r, n in new.items() for _ in range(n)])
    return block(x, step, max(new.values()), segments, **kw), (x, step, max(new.values()), segments)


def test_workspaces_do_not_add_up():
    """Steps of many sizes keep the workspaces of the largest, not one for every size."""
    block, pages, *_ = make()
    sizes = []
    for n in (60, 3, 1, 41, 57, 1, 2, 22, 50, 9):
        run_step(block, pages, {n * 100: n, n * 100 + 1: 1}, n)
        pages.release(n * 100), pages.release(n * 100 + 1)
        assert len(block.work) == 1
        held = next(iter(block.work.values())).held
        sizes.append({k: t.numel() for k, t in held.items()})
    assert set(sizes[-1]) == {"attn", "lora"} and all(s == sizes[0] for s in sizes)       # the first step was the largest
    assert q4k.q4k_device_error() == 0


def test_streams_and_graphs_have_their_own_workspaces():
    """A first call inside a capture, the same step called directly on two streams, and the graph replayed beside them."""
    block, pages, *_ = make()
    run_step(block, pages, {0: 90, 1: 70, 2: 1}, 1)                       # something in the cache
    mine = next(iter(block.work.values())).held["attn"].data_ptr()
    for new, work in (({0: 1, 1: 1, 2: 1}, None), ({0: 40, 1: 1, 2: 2}, None), ({1: 1, 2: 1}, Workspaces())):
        want, args = run_step(block, pages, new, 2, **({"work": work} if work else {}))
        want = want.clone()
        torch.cuda.synchronize()
        graph, kept = torch.cuda.CUDAGraph(), dict(block.work)
        with torch.cuda.graph(graph):
            got = block(*args, work=work)
        assert block.work == kept                                        # nothing of the capture stays behind
        side = torch.cuda.Stream()
        for _ in range(3):
            got.zero_()
            side.wait_stream(torch.cuda.current_stream())
            graph.replay()
            with torch.cuda.stream(side):
                other = block(*args)
            direct = block(*args)
            torch.cuda.synchronize()
            assert torch.equal(got, want) and torch.equal(direct, want) and torch.equal(other, want)
        assert block.work[side.cuda_stream].held["attn"].data_ptr() != mine
    with pytest.raises(RuntimeError):                                    # a graph never makes the workspaces it is given
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            block(*args, work=Workspaces())
    torch.cuda.synchronize()
    assert q4k.q4k_device_error() == 0


def test_the_example_runs(capsys):
    import sys
    from q4_weight_matmul_gb300 import attention_block
    old, sys.argv = sys.argv, ["x", "--requests", "4", "--prompt", "50", "--steps", "3", "--hidden", "512", "--heads", "4",
                               "--kv-heads", "1"]
    try:
        attention_block.main()
    finally:
        sys.argv = old
    out = capsys.readouterr().out
    assert "decode step 2" in out and "nan" not in out
