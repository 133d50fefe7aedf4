"""q4k_paged_attn against the 64-bit oracle.

Bounds.  fp32 out (the header's): 1e-5 of the largest |v| a row sees, times
z / 64 where z = max |scale| sum |q||k| is above 64 (a fp32 score is off by a
few 2^-24 of that, and a weight by as much of itself).  16-bit out: each weight may be rounded to the type (u of sum p|v|) and the result is
(u of |out|), u = 2^-11 or 2^-8, beside the fp32 bound and half of binary16's
smallest step.
"""
import numpy as np
import pytest
import torch

import q4_weight_matmul_gb300 as q4k
from oracle import attention as O

pytestmark = pytest.mark.gpu
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def make(seed, new, kv, heads, kv_heads, dim, page, dtype, spare=3, stale=float("nan"), std=1.4):
    """Caches whose cells past a request's keys, spare pages and unused table entries are poisoned."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-n // page) for n in kv]
    total = sum(per) + spare
    place = torch.randperm(total, generator=g)
    table = torch.full((len(kv), max(max(per, default=0), 1)), -1, dtype=torch.int32)
    kc = torch.full((total, kv_heads, page, dim), stale, dtype=dtype)
    vc = torch.full((total, kv_heads, page, dim), stale, dtype=dtype)
    at = 0
    for r, n in enumerate(kv):
        for i in range(per[r]):
            p = int(place[at])
            at += 1
            table[r, i] = p
            m = min(page, n - i * page)
            kc[p, :, :m] = (std * torch.randn((kv_heads, m, dim), generator=g)).to(dtype)
            vc[p, :, :m] = torch.randn((kv_heads, m, dim), generator=g).to(dtype)
    q = (std * torch.randn((sum(new), heads, dim), generator=g)).to(dtype)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return {"q": q, "kc": kc, "vc": vc, "table": table, "cu": cu, "kv": torch.tensor(kv, dtype=torch.int32)}


def run(d, max_q, out_dtype=torch.float32, window=0, scale=None, **kw):
    c = {k: v.cuda() for k, v in d.items()}
    return q4k.q4k_paged_attn(c["q"], c["kc"], c["vc"], c["table"], c["cu"], c["kv"], max_q, scale=scale,
                              window=window, out_dtype=out_dtype, **kw)


def check(got, d, new, kv, window=0, scale=None):
    dim = d["q"].shape[2]
    f = lambda t: t.float().numpy()  # noqa: E731
    want, pv, vmax, z = O.paged_attn(f(d["q"]), f(d["kc"]), f(d["vc"]), d["table"].numpy(), new, kv,
                                  dim ** -0.5 if scale is None else scale, window)
    tol = (1e-5 * np.maximum(1, z / 64) * vmax)[..., None] + np.zeros_like(want)
    if got.dtype != torch.float32:
        u = U[got.dtype]
        tol = tol + u * (pv + np.abs(want)) + (2.0 ** -24 if got.dtype == torch.float16 else 0.0)
    got = got.cpu().double().numpy()
    assert np.all(np.isfinite(got))
    over = np.abs(got - want) - tol
    assert np.all(over <= 0), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))


SHAPES = [  # new tokens, keys, heads, kv_heads, dim, page, window
    ([1], [1], 8, 2, 128, 16, 0),
    ([1], [64], 32, 8, 128, 16, 0),
    ([1], [1021], 32, 8, 128, 16, 0),
    ([1, 1, 1, 1, 1], [1, 17, 300, 0, 65], 28, 4, 128, 32, 0),
    ([1, 1], [700, 513], 16, 1, 64, 64, 100),
    ([1] * 33, [3 * i + 1 for i in range(33)], 8, 8, 128, 16, 0),
    ([1, 1], [130, 257], 40, 1, 128, 256, 0),          # 40 query heads on one key head
    ([5, 1, 4, 0, 3], [333, 64, 4, 50, 2], 28, 4, 128, 16, 0),    # the last row set starts before its first key
    ([5, 5], [301, 40], 12, 4, 64, 128, 33),
    ([9, 2], [130, 131], 32, 8, 64, 32, 1),            # each token sees only itself
    ([17], [17], 32, 8, 128, 16, 0),
    ([33, 1, 70], [200, 90, 70], 32, 8, 128, 16, 0),
    ([128], [128], 8, 8, 128, 128, 0),
    ([129], [385], 16, 4, 64, 64, 0),
    ([200, 77], [450, 333], 28, 4, 128, 32, 120),
    ([257], [300], 40, 8, 128, 64, 0),
    ([65, 3, 0, 90], [700, 129, 5, 91], 16, 1, 128, 16, 0),
    ([100], [60], 8, 2, 64, 16, 0),                    # 40 tokens before the first key: zeros
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("dtype,out_dtype", [(torch.float16, torch.float32), (torch.float16, torch.float16),
                                             (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)])
def test_matches_the_oracle(case, dtype, out_dtype):
    q4k.build()
    new, kv, heads, kv_heads, dim, page, window = SHAPES[case]
    d = make(case, new, kv, heads, kv_heads, dim, page, dtype)
    got = run(d, max(new), out_dtype, window)
    assert got.dtype == out_dtype
    check(got, d, new, kv, window)
    assert q4k.q4k_device_error() == 0


@pytest.mark.parametrize("new,kv", [([1], [40000]), ([3], [20001]), ([70], [5000]), ([300], [20000])])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_long_contexts(new, kv, dtype):
    q4k.build()
    d = make(77, new, kv, 4, 1, 128, 64, dtype)
    for out_dtype in (torch.float32, dtype):
        check(run(d, max(new), out_dtype), d, new, kv)
    assert q4k.q4k_device_error() == 0


@pytest.mark.parametrize("requests,new,kv", [(129, 1, 40), (700, 1, 20), (9, 40, 70), (40, 19, 60), (200, 3, 30),
                                             (1100, 2, 3)])
def test_many_requests(requests, new, kv):
    """More requests than one warp looks at, with and without several row tiles each, some of them without tokens."""
    q4k.build()
    r = np.random.default_rng(requests)
    news = [int(v) for v in r.integers(0, new + 1, requests)]
    kvs = [int(v) for v in r.integers(0, kv + 1, requests)]
    news[0], kvs[0] = new, kv
    d = make(requests, news, kvs, 8, 2, 64, 16, torch.float16)
    for out_dtype in (torch.float32, torch.float16):
        check(run(d, new, out_dtype), d, news, kvs)
    assert q4k.q4k_device_error() == 0


@pytest.mark.parametrize("new", [1, 6, 130])
def test_peaked_and_flat_scores(new):
    """Scores of several hundred (one key takes all, at the far end or the near one), and equal scores."""
    q4k.build()
    for std, scale in ((6.0, 1.0), (0.0, None), (1.0, -0.4)):
        d = make(11, [new], [900], 8, 2, 128, 32, torch.float16, std=std)
        for out_dtype in (torch.float32, torch.float16):
            check(run(d, new, out_dtype, scale=scale), d, [new], [900], scale=scale)


@pytest.mark.parametrize("new", [1, 5, 140])
def test_small_weights_add_up(new):
    """One key far above the rest, the rest together as heavy: weights of 2^-15 of the largest still count."""
    q4k.build()
    d = make(12, [new], [30000], 2, 1, 64, 64, torch.float16, std=0.0)
    d["q"][:] = 0
    d["q"][:, :, 0] = 8.0
    page = int(d["table"][0, 0])
    d["kc"][page, :, 3, 0] = 10.0            # score 80 / 8 = 10: e^10 = 22026 against 29999 ones
    check(run(d, new), d, [new], [30000])


def test_fully_poisoned_cache_beside_the_keys():
    """Infinities past the last key, and a request whose keys end inside a page shared with nobody."""
    q4k.build()
    for stale in (float("inf"), float("-inf"), float("nan")):
        for new, kv in (([1, 2], [33, 47]), ([70], [71])):
            for window in (0, 20):
                d = make(13, new, kv, 8, 2, 128, 32, torch.float16, stale=stale)
                if window:          # keys that no token sees any more: their pages may be gone
                    for r in range(len(kv)):
                        for j in range(max(0, kv[r] - new[r] - window + 1)):
                            d["kc"][int(d["table"][r, j // 32]), :, j % 32] = stale
                            d["vc"][int(d["table"][r, j // 32]), :, j % 32] = stale
                got = run(d, max(new), torch.float32, window)
                got16 = run(d, max(new), torch.float16, window)
                for n in ("kc", "vc"):
                    d[n] = torch.nan_to_num(d[n], 0.0, 0.0, 0.0)
                check(got, d, new, kv, window)
                check(got16, d, new, kv, window)
    assert q4k.q4k_device_error() == 0


def test_pages_outside_a_window_may_be_gone():
    q4k.build()
    for new in ([1], [9], [80]):
        kv, window = [500], 64
        d = make(14, new, kv, 8, 2, 128, 16, torch.bfloat16)
        gone = max(0, kv[0] - new[0] - window + 1) // 16
        full = d["table"].clone()
        d["table"][0, :gone] = -1
        got = run(d, new[0], torch.float32, window)
        assert q4k.q4k_device_error() == 0
        d["table"] = full
        check(got, d, new, kv, window)


@pytest.mark.parametrize("new", [1, 40])
def test_indices_out_of_range_are_reported(new):
    q4k.build()
    kv = [200]
    d = make(15, [new], kv, 8, 2, 64, 16, torch.float16)
    for bad in (-5, d["kc"].shape[0], 2 ** 30):
        b = {k: v.clone() for k, v in d.items()}
        b["table"][0, 3] = bad
        for out_dtype in (torch.float32, torch.float16):
            got = run(b, new, out_dtype)
            assert q4k.q4k_device_error() == 6
            zero = {k: v.clone() for k, v in d.items()}
            zero["kc"][int(d["table"][0, 3])] = 0
            zero["vc"][int(d["table"][0, 3])] = 0
            check(got, zero, [new], kv)
    b = {k: v.clone() for k, v in d.items()}
    b["kv"][0] = 10 ** 6                       # more than the table holds
    got = run(b, new)
    assert q4k.q4k_device_error() == 6 and got.shape == d["q"].shape
    b = {k: v.clone() for k, v in d.items()}
    b["cu"][1] = new + 50                      # more tokens than there are
    got = run(b, new)
    assert q4k.q4k_device_error() == 6
    assert q4k.q4k_device_error() == 0


def test_workspace_is_kept_and_results_repeat():
    q4k.build()
    shapes = [([1, 1, 1], [900, 64, 2000]), ([4], [1500]), ([150, 20], [600, 400]), ([1], [3])]
    made = [make(20 + i, n, k, 32, 8, 128, 16, torch.float16) for i, (n, k) in enumerate(shapes)]
    need = max(q4k.q4k_paged_attn_workspace(d["q"], d["kc"].cuda(), d["table"], max(n), t).numel()
               for d, (n, _) in zip(made, shapes) for t in (torch.float32, torch.float16))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = {}
    for turn in range(3):
        for i, (d, (n, k)) in enumerate(zip(made, shapes)):
            for t in (torch.float32, torch.float16):
                got = run(d, max(n), t, workspace=ws)
                if turn == 0:
                    check(got, d, n, k)
                    first[i, t] = got
                assert torch.equal(got, first[i, t]), (i, t)
    assert q4k.q4k_device_error() == 0


@pytest.mark.parametrize("new", [1, 90])
def test_on_another_stream_and_in_a_graph(new):
    q4k.build()
    d = make(30, [new], [800], 16, 4, 128, 16, torch.float16)
    for t in (torch.float32, torch.float16):
        ref = run(d, new, t)
        c = {k: v.cuda() for k, v in d.items()}
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            out = q4k.q4k_paged_attn(c["q"], c["kc"], c["vc"], c["table"], c["cu"], c["kv"], new, out_dtype=t)
        s.synchronize()
        assert torch.equal(out, ref)
        ws = q4k.q4k_paged_attn_workspace(c["q"], c["kc"], c["table"], new, t)
        out = torch.zeros_like(ref)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            q4k.q4k_paged_attn(c["q"], c["kc"], c["vc"], c["table"], c["cu"], c["kv"], new, out=out, workspace=ws)
        for _ in range(2):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
        # the lengths live on the device: a replay follows them
        c["kv"].fill_(new + 100)
        g.replay()
        torch.cuda.synchronize()
        check(out, d, [new], [new + 100])


@pytest.mark.parametrize("by_handle", [False, True])
@pytest.mark.parametrize("new,kv", [([1], [9000]), ([4, 1], [5000, 700]), ([300], [4000])])
def test_stream_argument_while_the_current_stream_is_busy(new, kv, by_handle):
    """The call makes its workspace and output for ``stream``: neither a fill that waits behind the current stream's work
    nor memory given back to that stream may reach the kernels."""
    q4k.build()
    d = make(34, new, kv, 16, 4, 128, 16, torch.float16)
    c = {k: v.cuda() for k, v in d.items()}
    for t in (torch.float32, torch.float16):
        need = q4k.q4k_paged_attn_workspace(c["q"], c["kc"], c["table"], max(new), t).numel()
        torch.cuda.empty_cache()
        dirty = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")     # what a fresh workspace would be made of
        torch.cuda.synchronize()
        del dirty
        s = torch.cuda.Stream()
        outs = []
        torch.cuda._sleep(20_000_000)                                           # some 10 ms on the current stream
        for _ in range(3):
            outs.append(q4k.q4k_paged_attn(c["q"], c["kc"], c["vc"], c["table"], c["cu"], c["kv"], max(new),
                                           out_dtype=t, stream=s.cuda_stream if by_handle else s))
            torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")          # takes what the call gave back
        s.synchronize()
        for got in outs:
            check(got, d, new, kv)
        torch.cuda.synchronize()
    assert q4k.q4k_device_error() == 0


@pytest.mark.parametrize("new", [1, 100])
def test_offsets_past_32_bits(new):
    q4k.build()
    d = make(31, [new], [300], 8, 8, 128, 256, torch.float16)
    pages = 2 ** 31 // (8 * 256 * 128) + 3
    kc = torch.empty((pages, 8, 256, 128), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    far = d["table"].clone()
    for i in range(2):
        far[0, i] = pages - 1 - i
        kc[pages - 1 - i] = d["kc"][int(d["table"][0, i])].cuda()
        vc[pages - 1 - i] = d["vc"][int(d["table"][0, i])].cuda()
    for t in (torch.float32, torch.float16):
        got = q4k.q4k_paged_attn(d["q"].cuda(), kc, vc, far.cuda(), d["cu"].cuda(), d["kv"].cuda(), new, out_dtype=t)
        check(got, d, [new], [300])
    assert q4k.q4k_device_error() == 0


@pytest.mark.parametrize("dim,dtype", [(64, torch.float16), (128, torch.float16), (128, torch.bfloat16)])
def test_sums_over_very_many_keys(dim, dtype):
    """2^28 keys, two pages again and again, with values that do not cancel: a sum that loses some 2^-23 of itself in one
    direction at every step is off by more than the result's rounding then.  The second page's scores are higher by 8; it
    comes last, near the end, or after a third of the keys, so that what was summed before has to be scaled."""
    q4k.build()
    g = torch.Generator().manual_seed(35)
    pages, new = 2 ** 28 // 256, 20
    kc, vc = torch.zeros((2, 1, 256, dim), dtype=dtype), (1 + 0.2 * torch.randn((2, 1, 256, dim), generator=g)).to(dtype)
    kc[:, 0, :, 0] = torch.randn((2, 256), generator=g).to(dtype)
    kc[1, :, :, 1] = 16.0
    q = torch.zeros((new, 1, dim), dtype=dtype)
    q[:, :, :2] = 1.0
    score = 0.5 * kc[:, 0, :, :2].double().sum(-1)                           # [page][cell]
    weight, values = score.exp(), vc[:, 0].double()
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    kv = torch.tensor([pages * 256], dtype=torch.int32, device="cuda")
    q, kc, vc = q.cuda(), kc.cuda(), vc.cuda()
    for turn in (pages, pages - 1, pages - 150, pages // 3):                 # pages from `turn` on are the second
        table = (torch.arange(pages, device="cuda") >= turn).to(torch.int32)[None]
        got = q4k.q4k_paged_attn(q, kc, vc, table, cu, kv, new, scale=0.5, out_dtype=dtype)
        times = torch.tensor([turn, pages - turn]).double()
        for i in (0, 7, new - 1):                                            # token i misses the last new - 1 - i cells
            gone = slice(256 - (new - 1 - i), 256)
            last = 0 if turn == pages else 1
            num = (times[:, None] * (weight[:, :, None] * values).sum(1)).sum(0) - (weight[last, gone, None] * values[last, gone]).sum(0)
            den = (times * weight.sum(1)).sum() - weight[last, gone].sum()
            want, most = num / den, values.abs().max()
            tol = U[dtype] * 2 * want.abs() + 1e-5 * most + (2.0 ** -24 if dtype == torch.float16 else 0.0)
            far = (got[i, 0].cpu().double() - want).abs()
            assert bool((far <= tol).all()), (turn, i, float((far / tol).max()))
    assert q4k.q4k_device_error() == 0


@pytest.mark.parametrize("new,out_dtype", [(1, torch.float32), (9, torch.float32), (20, torch.float16)])
def test_the_longest_context(new, out_dtype):
    """As many keys as a table of pages of 16 can name: the last unit ends past 2^31.  All keys are one page, scored far
    below zero, so that a cell past the last one, which reads as zeros, would outweigh them all."""
    q4k.build()
    pages = 2 ** 31 // 16 - 1
    kv = pages * 16
    kc = torch.full((1, 1, 16, 64), -1.0, dtype=torch.float16, device="cuda")
    vc = torch.arange(16, dtype=torch.float16, device="cuda")[None, None, :, None].expand(1, 1, 16, 64).contiguous()
    q = torch.ones((new, 1, 64), dtype=torch.float16, device="cuda")
    table = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    got = q4k.q4k_paged_attn(q, kc, vc, table, cu, torch.tensor([kv], dtype=torch.int32, device="cuda"), new, scale=1.0,
                             out_dtype=out_dtype)
    assert q4k.q4k_device_error() == 0
    # equal weights: the mean of 0..15; token i misses the last new - 1 - i cells, nothing beside 2^31.  Sums of 2^31
    # equal weights in fp32: each lane's are exact up to 2^24 of them, then the lanes' and pieces' are added up
    tol = 15 * 1e-5 + (2.0 ** -11 * 2 * 7.5 if out_dtype == torch.float16 else 0.0)
    assert float((got.double() - 7.5).abs().max()) <= tol


def test_no_tokens_and_refusals():
    q4k.build()
    d = make(32, [0, 0], [5, 7], 8, 2, 128, 16, torch.float16)
    assert run(d, 0).shape[0] == 0
    d = make(33, [2, 1], [50, 70], 8, 2, 128, 16, torch.float16)
    c = {k: v.cuda() for k, v in d.items()}
    ok = dict(q=c["q"], k_cache=c["kc"], v_cache=c["vc"], page_table=c["table"], cu_q=c["cu"], kv_len=c["kv"], max_q=2)
    q4k.q4k_paged_attn(**ok)
    small = torch.zeros(0, dtype=torch.uint8, device="cuda")
    for bad, err in ((dict(q=c["q"].float()), TypeError), (dict(q=c["q"][..., :64]), ValueError),
                     (dict(q=c["q"].cpu()), TypeError), (dict(page_table=c["table"].long()), TypeError),
                     (dict(page_table=c["table"][0]), ValueError), (dict(cu_q=c["cu"][:2]), ValueError),
                     (dict(kv_len=c["kv"][:1]), ValueError), (dict(window=-1), q4k.Q4KError),
                     (dict(scale=float("nan")), q4k.Q4KError), (dict(max_q=0), q4k.Q4KError),
                     (dict(out=torch.empty((3, 8, 128), device="cuda", dtype=torch.bfloat16)), q4k.Q4KError),
                     (dict(out=torch.empty((3, 8, 64), device="cuda")), ValueError),
                     (dict(workspace=small), q4k.Q4KError),
                     (dict(q=c["q"][:, :7].contiguous()), q4k.Q4KError)):
        with pytest.raises(err):
            q4k.q4k_paged_attn(**{**ok, **bad})
