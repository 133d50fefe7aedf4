"""The kernels that stream through rings in shared memory, three hundred times
on the same inputs: the same bits every time.  (A warp that gives a stage back
before its last reads of it finds the next copy's bytes there, in one call of
many.)"""
import pytest
import torch

import q4_weight_matmul_gb300 as q4k

pytestmark = pytest.mark.gpu
CALLS = 300


@pytest.fixture(scope="module", autouse=True)
def built():
    q4k.build()
    yield
    assert q4k.q4k_device_error() == 0


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(rows, cols, seed, six=False):
    g = rng(seed)
    i = lambda lo, hi, n, t=torch.uint8: torch.randint(lo, hi, (rows, n), generator=g, device="cuda", dtype=t)  # noqa: E731
    d = (0.5 + torch.rand((rows, cols // 256), generator=g, device="cuda")).half().view(torch.int16)
    if six:
        return q4k.q6k_pack(d, i(-128, 128, cols // 16, torch.int8), i(0, 64, cols))
    return q4k.q4k_pack(d, d, i(0, 64, cols // 32), i(0, 64, cols // 32), i(0, 16, cols))


def floats(*shape, seed=1):
    return torch.randn(shape, generator=rng(seed), device="cuda")


def repeat(call):
    """``call`` returns tensors; all of them hold the first call's bits in every later one."""
    want = [t.clone() for t in call()]
    assert all(bool(torch.isfinite(t.float()).all()) for t in want)
    differ = [torch.stack([(a != b).any() for a, b in zip(call(), want)]).any() for _ in range(CALLS)]
    assert int(torch.stack(differ).sum()) == 0


@pytest.mark.parametrize("six", [False, True], ids=["q4_k", "q6_k"])
@pytest.mark.parametrize("rows,cols,batch", [(9728, 2560, 1), (2560, 9728, 1), (1024, 2560, 3), (2560, 4096, 8), (4000, 4096, 4)])
def test_decode_products(rows, cols, batch, six):
    w, x, res = matrix(rows, cols, 10, six), floats(batch, cols), floats(batch, rows, seed=2)
    q8 = q4k.q8_quantize(x)
    fp, q = (q4k.q6k_gemv, q4k.q6k_gemv_q8) if six else (q4k.q4k_gemv, q4k.q4k_gemv_q8)
    repeat(lambda: [fp(w, rows, cols, x, residual=res), q(w, rows, cols, *q8, residual=res)])


@pytest.mark.parametrize("batch", [1, 2, 4])
def test_several_matrices_at_once(batch):
    rows, cols = [4096, 1024, 1000], 2560
    ws, x = [matrix(r, cols, 20 + i) for i, r in enumerate(rows)], floats(batch, cols)
    repeat(lambda: q4k.q4k_gemv_multi(ws, rows, cols, x))


@pytest.mark.parametrize("mixed", [False, True], ids=["q4_k", "with q6_k"])
@pytest.mark.parametrize("batch", [1, 4])
def test_a_list_of_jobs(batch, mixed):
    jobs, ys, x = [], [], {2560: floats(batch, 2560), 9728: floats(batch, 9728, seed=2)}
    for i, (rows, cols) in enumerate([(4096, 2560), (1024, 2560), (1000, 2560), (9728, 2560), (2560, 9728), (33, 2560)]):
        six = mixed and i % 2 == 1
        ys.append(torch.empty((batch, rows), device="cuda"))
        jobs.append({"w": matrix(rows, cols, 30 + i, six), "rows": rows, "cols": cols, "x": x[cols], "y": ys[-1],
                     "wait": i in (3, 4), **({"format": 1} if six else {})})
    seq = q4k.GemvSeq(jobs, batch)

    def call():
        for y in ys:
            y.fill_(float("nan"))
        seq()
        return ys

    repeat(call)


@pytest.mark.parametrize("dim,dtype", [(128, torch.float16), (64, torch.float16), (128, torch.bfloat16), (64, torch.bfloat16)])
@pytest.mark.parametrize("new,heads,kv_heads,kv,requests", [
    (1, 32, 8, 4000, 7), (1, 8, 8, 1500, 40), (1, 32, 8, 60000, 1), (5, 28, 4, 3001, 8), (40, 16, 4, 2000, 3)])
def test_attention(new, heads, kv_heads, kv, requests, dim, dtype):
    page, pages = 16, -(-kv // 16)
    cells = requests * pages, kv_heads, page, dim
    k, v = floats(*cells, seed=40).to(dtype), floats(*cells, seed=41).to(dtype)
    table = torch.randperm(requests * pages, generator=rng(42), device="cuda").int().view(requests, pages)
    lengths = (kv - 37 * torch.arange(requests, device="cuda")).int()
    cu = (new * torch.arange(requests + 1, device="cuda")).int()
    q = floats(requests * new, heads, dim, seed=43).to(dtype)
    work = {t: q4k.q4k_paged_attn_workspace(q, k, table, new, t) for t in (torch.float32, dtype)}
    repeat(lambda: [q4k.q4k_paged_attn(q, k, v, table, cu, lengths, new, out_dtype=t, workspace=work[t]) for t in work])


@pytest.mark.parametrize("rows,cols,tokens", [(9728, 2560, 512), (1000, 9728, 200), (2560, 4096, 77)])
def test_prompt_products(rows, cols, tokens):
    w, w6, x = matrix(rows, cols, 50), matrix(rows, cols, 51, True), floats(tokens, cols)
    q8, q16, split = q4k.q8_quantize(x), q4k.q8_quantize_h16(x), q4k.x_split_f16(x)
    repeat(lambda: [q4k.q4k_gemm(w, rows, cols, *q8), q4k.q4k_gemm_h16(w, rows, cols, *q16),
                    q4k.q4k_gemm_f16(w, rows, cols, *split), q4k.q6k_gemm_f16(w6, rows, cols, *split)])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,cols,rows,rank", [(3, 2560, 1000, 16), (700, 2560, 1024, 64), (1500, 4096, 999, 32)])
def test_adapters(tokens, cols, rows, rank, dtype):
    x, base = floats(tokens, cols), [floats(tokens, rows, seed=2)]
    a, b = [floats(3, rank, cols, seed=60).to(dtype)], [floats(3, rows, rank, seed=61).to(dtype)]
    segments = q4k.q4k_lora_segments([t * 7 % 4 - 1 for t in range(tokens)])
    scale, work = torch.full((3,), 0.5, device="cuda"), q4k.q4k_lora_workspace(tokens, rank, 1)
    repeat(lambda: q4k.q4k_lora_add(x, a, b, base, *segments, scale, workspace=work))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,rank", [(37, 16), (700, 64), (1500, 32)])
def test_what_other_tokens_left_behind_changes_no_bits(tokens, rank, dtype):
    """Tiles with fewer than 16 tokens hold, in shared memory, rows that no
    token has: a call before with activations near and beyond fp32's largest
    leaves such values there."""
    cols, rows = 2560, 1024
    x, base = floats(tokens, cols), [floats(tokens, rows, seed=2)]
    a, b = [floats(3, rank, cols, seed=60).to(dtype)], [floats(3, rows, rank, seed=61).to(dtype)]
    segments = q4k.q4k_lora_segments([t * 7 % 4 - 1 for t in range(tokens)])
    whole = q4k.q4k_lora_segments([0] * (tokens // 16 * 16))
    scale, work = torch.full((3,), 0.5, device="cuda"), q4k.q4k_lora_workspace(tokens, rank, 1)
    want = q4k.q4k_lora_add(x, a, b, base, *segments, scale, workspace=work)[0].clone()
    for left in (3.4e38, float("inf"), float("nan"), 1e-30, 0.0):
        full = torch.full_like(x[:whole[0].numel()], left)
        for _ in range(3):
            q4k.q4k_lora_add(full, a, b, [base[0][:full.shape[0]]], *whole, scale, workspace=work)
            assert torch.equal(q4k.q4k_lora_add(x, a, b, base, *segments, scale, workspace=work)[0], want), left


def calls(value):
    """One call of every kind, on random inputs, or on activations (and keys and values) of ``value``."""
    def x(*shape, seed=1):
        return floats(*shape, seed=seed) if value is None else torch.full(shape, value, device="cuda")

    rows, cols = 1000, 2560
    w, w6, made = matrix(rows, cols, 70), matrix(rows, cols, 71, True), {}
    for batch in (1, 4, 8):
        made[f"gemv {batch}"] = lambda b=batch: [q4k.q4k_gemv(w, rows, cols, x(b, cols)), q4k.q6k_gemv(w6, rows, cols, x(b, cols))]
    for tokens in (1, 7, 33, 200):
        q8 = q4k.q8_quantize(floats(tokens, cols) if value is None else torch.zeros((tokens, cols), device="cuda"))
        made[f"q8 {tokens}"] = lambda q8=q8: [q4k.q4k_gemm(w, rows, cols, *q8), q4k.q6k_gemm(w6, rows, cols, *q8)]
        made[f"f16 {tokens}"] = lambda t=tokens: [g(m, rows, cols, *q4k.x_split_f16(x(t, cols)))
                                                  for g, m in ((q4k.q4k_gemm_f16, w), (q4k.q6k_gemm_f16, w6))]
    jobs, ys = [], []
    for i in range(5):
        ys.append(torch.empty((2, rows), device="cuda"))
        jobs.append({"w": w6 if i == 2 else w, "rows": rows, "cols": cols, "x": x(2, cols), "y": ys[-1], "wait": i == 3,
                     **({"format": 1} if i == 2 else {})})
    seq = q4k.GemvSeq(jobs, 2)
    made["jobs"] = lambda keep=jobs: (seq(), [y.clone() for y in ys])[1]
    for dim in (64, 128):
        for dtype in (torch.float16, torch.bfloat16):
            fits = (lambda t, d=dtype: t.clamp(-6e4, 6e4).to(d)) if dtype == torch.float16 else (lambda t, d=dtype: t.to(d))
            for new in (1, 2, 5, 11, 19, 150):
                cells, kv = (40, 2, 16, dim), [300, 270]
                k, v, q = fits(x(*cells)), fits(x(*cells, seed=2)), fits(x(2 * new, 12, dim, seed=3))
                table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
                cu, n = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda"), torch.tensor(kv, dtype=torch.int32, device="cuda")
                made[f"attention {dim} {dtype} {new}"] = lambda a=(q, k, v, table, cu, n, new), t=dtype: [
                    q4k.q4k_paged_attn(*a, out_dtype=o) for o in (torch.float32, t)]
            for tokens, rank in ((3, 16), (37, 16), (150, 40)):
                a, b = [floats(2, rank, cols, seed=60).to(dtype)], [floats(2, rows, rank, seed=61).to(dtype)]
                base, scale = [floats(tokens, rows, seed=2)], torch.full((2,), 0.5, device="cuda")
                segments = q4k.q4k_lora_segments([t * 7 % 3 - 1 for t in range(tokens)] if value is None else [0] * tokens)
                made[f"adapters {dtype} {tokens}"] = lambda a=(x(tokens, cols), a, b, base, *segments, scale): q4k.q4k_lora_add(*a)
    experts, width = 6, 256
    g, u, d = (matrix(experts * r, c, 80 + i) for i, (r, c) in enumerate(((width, cols), (width, cols), (rows, width))))
    d6 = matrix(experts * rows, width, 84, True)
    for tokens in (1, 11, 25, 50, 300):
        route = q4k.q4k_moe_route(floats(tokens, experts, seed=4), 2)
        made[f"experts {tokens}"] = lambda t=tokens, r=route: (lambda h: [h] + [
            q4k.q4k_moe_down(h, m, rows, r, q6k=six) for m, six in ((d, False), (d6, True))])(
                q4k.q4k_moe_gate_up(1e-4 * x(t, cols), g, u, width, r))
    return made


@pytest.mark.parametrize("value", [3.4e38, float("inf"), float("nan")])
def test_what_other_calls_left_in_shared_memory_changes_no_bits(value):
    good, bad = calls(None), calls(value)
    want = {n: [t.clone() for t in c()] for n, c in good.items()}
    for n, w in want.items():
        assert all(bool(torch.isfinite(t.float()).all()) for t in w), n
    differ = []
    for before in bad:
        for n, c in good.items():
            bad[before]()
            if not all(torch.equal(a, b) for a, b in zip(c(), want[n])):
                differ.append((before, n))
    q4k.q4k_device_error()
    assert not differ


def test_two_streams_at_once():
    """Calls of every kind beside every other on another stream: they share the
    SMs, their shared memory and tensor memory, and nothing else."""
    good = calls(None)
    want = {n: [t.clone() for t in c()] for n, c in good.items()}
    names, streams = list(good), [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    differ = []
    for i, first in enumerate(names):
        got = []
        for second in names[i + 1::7]:                       # (one pair in seven)
            for stream, n in zip(streams, (first, second)):
                with torch.cuda.stream(stream):
                    got += [(n, a, b) for _ in range(4) for a, b in zip(good[n](), want[n])]
        torch.cuda.synchronize()
        differ += [(first, n) for n, a, b in got if not torch.equal(a, b)]
    assert q4k.q4k_device_error() == 0
    assert not differ
