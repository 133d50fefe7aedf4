"""q4k_qk_norm_rope against the 64-bit oracle.

Bound: one rounding to the 16-bit type (u = 2^-11 or 2^-8 of |y|, at least
half of binary16's smallest step, 2^-25) and fp32 arithmetic before it: a sum
of at most 128 squares in at most 12 levels, a square root, a division, two
weights' products and one rotation, under 32 roundings of 2^-24 of the terms:
2^-19 of their magnitude.
"""
import numpy as np
import pytest
import torch

import q4_weight_matmul_gb300 as q4k
from oracle import attention as O

pytestmark = pytest.mark.gpu
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def make(seed, tokens, heads, kv_heads, dim, page, dtype, pages=7, max_pos=512, rot=None):
    r = np.random.default_rng(seed)
    rot = dim if rot is None else rot
    f = lambda *s: r.standard_normal(s).astype(np.float32)  # noqa: E731
    d = {"q": f(tokens, heads, dim), "k": f(tokens, kv_heads, dim), "v": f(tokens, kv_heads, dim),
         "qw": 1 + 0.3 * f(dim), "kw": 1 + 0.3 * f(dim), "pos": r.integers(0, max_pos, tokens).astype(np.int32),
         "slot": r.permutation(pages * page)[:tokens].astype(np.int32)}
    angle = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, max(rot, 2), 2) / max(rot, 2))
    d["cs"] = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    g = torch.Generator().manual_seed(seed)
    d["kc"] = torch.randn((pages, kv_heads, page, dim), generator=g).to(dtype)
    d["vc"] = torch.randn((pages, kv_heads, page, dim), generator=g).to(dtype)
    return d, rot


def check(got, want, mag, dtype):
    got = got.cpu().double().numpy()
    tol = U[dtype] * np.abs(want) + 2.0 ** -19 * mag + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))


def run(d, rot, norm=True, interleaved=False, flat=False, **kw):
    c = {k: torch.from_numpy(v).cuda() for k, v in d.items() if isinstance(v, np.ndarray)}
    kc, vc = d["kc"].cuda(), d["vc"].cuda()
    q, k, v = (c[n].flatten(1) if flat else c[n] for n in "qkv")
    out = q4k.q4k_qk_norm_rope(q, k, v, kc, vc, c["pos"] if rot else None, c["slot"], c["cs"] if rot else None,
                               c["qw"] if norm else None, c["kw"] if norm else None, 1e-6, interleaved, **kw)
    return out, kc, vc


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,heads,kv_heads,dim,rot,page,norm,interleaved", [
    (1, 32, 8, 128, 128, 16, True, False),
    (3, 32, 8, 128, 128, 64, True, True),
    (37, 28, 4, 128, 64, 32, True, False),
    (5, 1, 1, 64, 64, 16, True, False),
    (130, 12, 4, 64, 24, 256, True, True),
    (9, 7, 7, 64, 8, 128, False, False),
    (6, 5, 1, 128, 0, 16, True, False),
    (6, 5, 1, 64, 0, 16, False, False),
    (300, 16, 8, 128, 120, 64, True, False),
])
def test_matches_the_oracle(tokens, heads, kv_heads, dim, rot, page, norm, interleaved, dtype):
    q4k.build()
    pages = max(7, 2 * tokens // page + 1)
    d, rot = make(tokens * 1000 + heads, tokens, heads, kv_heads, dim, page, dtype, pages, rot=rot)
    d["slot"][tokens // 2] = -1 if tokens > 2 else d["slot"][tokens // 2]
    out, kc, vc = run(d, rot, norm, interleaved, flat=tokens % 2 == 0)
    assert out.dtype == dtype and out.shape == (tokens, heads, dim)
    want, mag = O.norm_rope(d["q"], d["qw"] if norm else None, 1e-6, d["cs"], d["pos"], rot, interleaved)
    check(out, want, mag, dtype)
    want, mag = O.norm_rope(d["k"], d["kw"] if norm else None, 1e-6, d["cs"], d["pos"], rot, interleaved)
    ref_k, ref_v = d["kc"].clone(), d["vc"].clone()
    for t, s in enumerate(d["slot"]):
        if s < 0:
            continue
        check(kc[s // page, :, s % page], want[t], mag[t], dtype)
        assert torch.equal(vc[s // page, :, s % page].cpu(), torch.from_numpy(d["v"][t]).to(dtype))
        ref_k[s // page, :, s % page] = kc[s // page, :, s % page].cpu()
        ref_v[s // page, :, s % page] = vc[s // page, :, s % page].cpu()
    assert torch.equal(kc.cpu(), ref_k) and torch.equal(vc.cpu(), ref_v)      # the other cells are untouched
    assert q4k.q4k_device_error() == 0


def test_rows_of_zeros_large_values_and_nan():
    q4k.build()
    d, rot = make(5, 4, 2, 1, 64, 16, torch.float16)
    d["q"][0] = 0
    d["q"][1] *= 1e15                       # squares up to 1e31
    d["q"][2, 0, 3] = np.nan
    out, _, _ = run(d, rot)
    want, mag = O.norm_rope(d["q"], d["qw"], 1e-6, d["cs"], d["pos"], rot, False)
    got = out.cpu().double().numpy()
    assert np.all(got[0] == 0) and np.all(np.isnan(got[2, 0]))
    check(out[1], want[1], mag[1], torch.float16)
    check(out[2, 1], want[2, 1], mag[2, 1], torch.float16)      # the other head of that token
    check(out[3], want[3], mag[3], torch.float16)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,rot,interleaved", [(128, 0, False), (128, 0, True), (64, 0, False), (128, 64, False),
                                                 (128, 64, True), (64, 24, False), (128, 104, False), (64, 40, True)])
def test_infinities_and_nan_outside_the_rotation(dim, rot, interleaved, dtype):
    """Without norm, values that are not rotated are only rounded: one that is not finite changes no other."""
    q4k.build()
    d, _ = make(11, 5, 6, 2, dim, 16, dtype, rot=rot)
    r = np.random.default_rng(rot)
    for n in "qk":
        for value in (np.inf, -np.inf, np.nan):
            at = r.random(d[n].shape) < 0.1
            at[..., :rot] = False
            d[n][at] = value
        assert not np.all(np.isfinite(d[n]))
    out, kc, _ = run(d, rot, False, interleaved)
    cells = [(int(s) // 16, int(s) % 16) for s in d["slot"]]
    keys = torch.stack([kc[p, :, c] for p, c in cells])
    for n, got in (("q", out), ("k", keys)):
        want = torch.from_numpy(d[n][..., rot:]).to(dtype)
        assert torch.equal(got[..., rot:].cpu().view(torch.int16)[~want.isnan()], want.view(torch.int16)[~want.isnan()])
        assert torch.equal(got[..., rot:].cpu().isnan(), want.isnan())
        if rot:
            turned, mag = O.norm_rope(d[n][..., :rot], None, 0.0, d["cs"], d["pos"], rot, interleaved)
            check(got[..., :rot], turned, mag, dtype)
    assert q4k.q4k_device_error() == 0


def test_no_tokens_and_indices_out_of_range():
    q4k.build()
    d, rot = make(6, 0, 4, 2, 128, 16, torch.bfloat16)
    out, _, _ = run(d, rot)
    assert out.shape[0] == 0
    d, rot = make(7, 6, 4, 2, 128, 16, torch.bfloat16)
    d["pos"][1], d["pos"][2], d["slot"][3] = 512, -1, 7 * 16
    fill = torch.full((6, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, kc, vc = run(d, rot, q_out=fill)
    assert q4k.q4k_device_error() == 6 and q4k.q4k_device_error() == 0
    want, mag = O.norm_rope(d["q"], d["qw"], 1e-6, d["cs"], np.clip(d["pos"], 0, 511), rot, False)
    for t in (0, 3, 4, 5):
        check(out[t], want[t], mag[t], torch.bfloat16)
    assert torch.all(out[1:3] == 7)
    kept = torch.ones(7 * 16, dtype=torch.bool)
    kept[[int(d["slot"][t]) for t in (0, 4, 5)]] = False
    flat = lambda c: c.cpu().transpose(1, 2).reshape(7 * 16, -1)  # noqa: E731
    assert torch.equal(flat(kc)[kept], flat(d["kc"])[kept]) and torch.equal(flat(vc)[kept], flat(d["vc"])[kept])


def test_on_another_stream_and_in_a_graph():
    q4k.build()
    d, rot = make(8, 40, 32, 8, 128, 16, torch.float16)
    ref, rk, _ = run(d, rot)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out, kc, _ = run(d, rot)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(kc, rk)
    c = {k: torch.from_numpy(v).cuda() for k, v in d.items() if isinstance(v, np.ndarray)}
    kc, vc = d["kc"].cuda(), d["vc"].cuda()
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        q4k.q4k_qk_norm_rope(c["q"], c["k"], c["v"], kc, vc, c["pos"], c["slot"], c["cs"], c["qw"], c["kw"], q_out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(kc, rk)


def test_stream_argument_while_the_current_stream_is_busy():
    """The queries that the call makes belong to ``stream``: what the current stream still reads is not written over."""
    q4k.build()
    d, rot = make(13, 40, 32, 8, 128, 16, torch.float16)
    ref, rk, _ = run(d, rot)
    torch.cuda.synchronize()
    for by_handle in (False, True):
        s = torch.cuda.Stream()
        old = torch.full_like(ref, 3.0)
        torch.cuda._sleep(20_000_000)                                        # some 10 ms on the current stream
        kept = old + 1                                                       # reads `old` after that
        del old
        c = {k: torch.from_numpy(v).pin_memory() for k, v in d.items() if isinstance(v, np.ndarray)}
        with torch.cuda.stream(s):
            c = {k: v.cuda(non_blocking=True) for k, v in c.items()}
            kc, vc = d["kc"].cuda(), d["vc"].cuda()
        out = q4k.q4k_qk_norm_rope(c["q"], c["k"], c["v"], kc, vc, c["pos"], c["slot"], c["cs"], c["qw"], c["kw"],
                                   stream=s.cuda_stream if by_handle else s)
        s.synchronize()
        assert torch.equal(out.cpu(), ref.cpu()) and torch.equal(kc.cpu(), rk.cpu())
        torch.cuda.synchronize()
        assert torch.all(kept == 4.0)


def test_offsets_past_32_bits():
    """A cache of 2^31 + elements: the last page's cells lie past a 32-bit offset."""
    q4k.build()
    d, rot = make(9, 3, 8, 8, 128, 256, torch.float16)
    pages = 2 ** 31 // (8 * 256 * 128) + 2
    kc = torch.empty((pages, 8, 256, 128), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    slot = torch.tensor([pages * 256 - 1, pages * 256 - 256, (pages - 1) * 256 - 1], dtype=torch.int32, device="cuda")
    c = {k: torch.from_numpy(v).cuda() for k, v in d.items() if isinstance(v, np.ndarray)}
    q4k.q4k_qk_norm_rope(c["q"], c["k"], c["v"], kc, vc, c["pos"], slot, c["cs"], c["qw"], c["kw"])
    want, mag = O.norm_rope(d["k"], d["kw"], 1e-6, d["cs"], d["pos"], rot, False)
    for t, (page, cell) in enumerate(((pages - 1, 255), (pages - 1, 0), (pages - 2, 255))):
        check(kc[page, :, cell], want[t], mag[t], torch.float16)
        assert torch.equal(vc[page, :, cell], c["v"][t].half())
    assert q4k.q4k_device_error() == 0


def test_binding_refuses():
    q4k.build()
    d, rot = make(10, 4, 4, 2, 128, 16, torch.float16)
    c = {k: torch.from_numpy(v).cuda() for k, v in d.items() if isinstance(v, np.ndarray)}
    kc, vc = d["kc"].cuda(), d["vc"].cuda()
    ok = [c["q"], c["k"], c["v"], kc, vc, c["pos"], c["slot"], c["cs"]]

    def call(**change):
        a = list(ok)
        for k, v in change.items():
            a["q k v kc vc pos slot cs".split().index(k)] = v
        return q4k.q4k_qk_norm_rope(*a)

    for bad, err in ((dict(q=c["q"].half()), TypeError), (dict(q=d["q"]), TypeError), (dict(k=c["k"][:, :1]), ValueError),
                     (dict(kc=c["k"]), TypeError), (dict(vc=vc[:3]), ValueError), (dict(slot=c["slot"].long()), TypeError),
                     (dict(pos=c["pos"][:2]), ValueError), (dict(q=c["q"].transpose(1, 2)), ValueError),
                     (dict(kc=kc[:, :, :12].contiguous(), vc=vc[:, :, :12].contiguous()), q4k.Q4KError),
                     (dict(cs=c["cs"][:, :100].contiguous()), q4k.Q4KError)):
        with pytest.raises(err):
            call(**bad)


def test_an_argument_without_a_truth_value_is_refused():
    """Its own exception comes out, before any launch."""
    class Neither:
        def __bool__(self):
            raise ZeroDivisionError("neither")

    q4k.build()
    d, rot = make(12, 4, 4, 2, 128, 16, torch.float16)
    fill = torch.full((4, 4, 128), 7.0, dtype=torch.float16, device="cuda")
    with pytest.raises(ZeroDivisionError):
        run(d, rot, interleaved=Neither(), q_out=fill)
    with pytest.raises(RuntimeError):                                        # of more values than one: torch's own
        run(d, rot, interleaved=torch.ones(2), q_out=fill)
    assert torch.all(fill == 7)
