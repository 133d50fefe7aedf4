"""The attention block of a Qwen3-shaped decoder layer on this library's
calls: quantised projections, low-rank adapters beside them, head norms with
rotation and cache store, attention over the paged cache, and the output
projection with the residual.

    python -m q4_weight_matmul_gb300.attention_block --requests 3 --prompt 300 --steps 8

reads a prompt of every request in one batch (one chunk each), then decodes
``--steps`` tokens of all of them, a CUDA graph per step shape, and prints the
time of each.  Weights and inputs are random (``--hidden 2560 --heads 32
--kv-heads 8``: the 4B shape).  With ``--experts 128`` (and ``--top-k``,
``--width``) the layer goes on with routed experts in place of a dense
feed-forward part (``expert_block.py``).
"""
from __future__ import annotations

import argparse

import torch

import q4_weight_matmul_gb300 as q4k


class Pages:
    """Which pages of the cache each request has, and one step's index arrays."""

    def __init__(self, num_pages: int, page_size: int, max_pages: int):
        self.free, self.page_size, self.max_pages = list(range(num_pages))[::-1], page_size, max_pages
        self.of, self.length = {}, {}

    def step(self, new):
        """``new``: {request: new tokens} in batch order.  Takes the pages that
        the new tokens need and returns the step's arrays (int32, host).  Where
        pages are missing it raises RuntimeError and changes nothing."""
        need = {r: -(-(self.length.get(r, 0) + n) // self.page_size) for r, n in new.items()}
        for r, n in need.items():
            if n > self.max_pages:
                raise RuntimeError(f"request {r} needs {n} pages of the {self.max_pages} that one may have")
        missing = sum(max(0, n - len(self.of.get(r, ()))) for r, n in need.items()) - len(self.free)
        if missing > 0:
            raise RuntimeError(f"{missing} pages too few are left")
        pos, slot, cu, kv, table = [], [], [0], [], []
        for r, n in new.items():
            pages, start = self.of.setdefault(r, []), self.length.get(r, 0)
            while len(pages) * self.page_size < start + n:
                pages.append(self.free.pop())
            for p in range(start, start + n):
                pos.append(p)
                slot.append(pages[p // self.page_size] * self.page_size + p % self.page_size)
            self.length[r] = start + n
            cu.append(cu[-1] + n)
            kv.append(start + n)
            table.append(pages + [-1] * (self.max_pages - len(pages)))
        make = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        return {"pos": make(pos), "slot": make(slot), "cu_q": make(cu), "kv_len": make(kv), "table": make(table)}

    def release(self, request):
        """Give the pages of a finished request back (its launches need not
        have ended: the next owner's come after them on their stream)."""
        self.free.extend(reversed(self.of.pop(request)))
        del self.length[request]


class Workspaces:
    """Scratch memory for the calls of one stream, or of one captured graph:
    one tensor for the attention, one for the adapters and one for the routed
    experts, each as large as the largest step so far.  Steps that share it must not overlap on the GPU, so
    one object serves all layers of a model that runs on one stream."""

    def __init__(self):
        self.held, self.in_graphs = {}, []

    def get(self, name, need, make, for_graph=False):
        """The tensor ``name`` of ``need`` bytes or more.  One that a graph
        was captured with stays where it is as long as this object does."""
        t = self.held.get(name)
        if t is None or t.numel() < need:
            if for_graph:
                raise RuntimeError("a step is captured with `work` only after it, or a larger one, has run with it")
            t = self.held[name] = make()
        if for_graph and not any(t is kept for kept in self.in_graphs):
            self.in_graphs.append(t)
        return t


class AttentionBlock:
    """One layer's attention block.  ``weights``: packed Q4_K ``q``, ``k``,
    ``v``, ``o``; ``norms``: head norm weights (q, k); ``adapters``: None or
    {"q"|"k"|"v"|"o": (a, b)} with a shared ``scale``."""

    def __init__(self, weights, hidden, heads, kv_heads, head_dim, norms, cos_sin, cache, adapters=None, scale=None):
        self.w, self.hidden, self.heads, self.kv_heads, self.dim = weights, hidden, heads, kv_heads, head_dim
        self.norms, self.cos_sin, (self.k_cache, self.v_cache) = norms, cos_sin, cache
        self.adapters, self.scale = adapters, scale
        self.work = {}                      # stream handle -> its Workspaces

    def _project(self, names, rows, x, residual=None):
        """The projections of ``x``: a weight pass per step for a few tokens, tensor-core products for many."""
        if x.shape[0] <= 8:
            return q4k.q4k_gemv_multi([self.w[n] for n in names], rows, x.shape[1], x,
                                      residuals=None if residual is None else [residual])
        split = q4k.x_split_f16(x)
        ys = [q4k.q4k_gemm_f16(self.w[n], r, x.shape[1], *split) for n, r in zip(names, rows)]
        return ys if residual is None else [ys[0] + residual]

    def _adapt(self, names, x, ys, segments, scratch):
        if self.adapters is None or segments is None:
            return
        a, b = [self.adapters[n][0] for n in names], [self.adapters[n][1] for n in names]
        size = x.shape[0], a[0].shape[1], len(names)
        work = scratch("lora", q4k.q4k_lora_workspace_bytes(*size), lambda: q4k.q4k_lora_workspace(*size))
        q4k.q4k_lora_add(x, a, b, ys, *segments, self.scale, y=ys, workspace=work)

    def __call__(self, x, step, max_q, segments=None, work=None):
        """``x`` [tokens][hidden] float32 (normed input, also the residual
        here); ``step``: ``Pages.step`` arrays on the device; ``segments``:
        ``q4k_lora_segments`` of the tokens' adapters; ``work``: the
        ``Workspaces`` to use.  Without it every stream has its own, and a
        call that is captured makes some for itself, which the graph keeps
        (its replays zero the attention's: a pass over some 0.6 to 40 MB)."""
        capturing = torch.cuda.is_current_stream_capturing()
        for_graph = capturing and work is not None
        if work is None:
            key = torch.cuda.current_stream().cuda_stream
            work = Workspaces() if capturing else self.work.setdefault(key, Workspaces())

        def scratch(name, need, make):
            return work.get(name, need, make, for_graph)

        rows = [self.heads * self.dim, self.kv_heads * self.dim, self.kv_heads * self.dim]
        q, k, v = qkv = self._project("qkv", rows, x)
        self._adapt("qkv", x, qkv, segments, scratch)
        q = q4k.q4k_qk_norm_rope(q, k, v, self.k_cache, self.v_cache, step["pos"], step["slot"], self.cos_sin,
                                 *self.norms)
        # a few tokens: fp32 results cost nothing; a chunk: 16-bit ones, from the tensor cores
        dtype = torch.float32 if max_q <= 8 else self.k_cache.dtype
        size = q, self.k_cache, step["table"], max_q, dtype
        space = scratch("attn", q4k.q4k_paged_attn_workspace_bytes(*size), lambda: q4k.q4k_paged_attn_workspace(*size))
        o = q4k.q4k_paged_attn(q, self.k_cache, self.v_cache, step["table"], step["cu_q"], step["kv_len"], max_q,
                               out_dtype=dtype, workspace=space).float().flatten(1)
        y = self._project("o", [self.hidden], o, residual=x)
        self._adapt("o", o, y, segments, scratch)
        return y[0]


def random_block(hidden, heads, kv_heads, head_dim, num_pages, page_size, max_pos, dtype, adapters=0, rank=16, seed=0,
                 device="cuda"):
    """A block with random weights of the given shape, and its Q4_K fields and
    adapters are not kept apart: for timing and examples."""
    g = torch.Generator(device=device).manual_seed(seed)

    def packed(rows, cols):
        nb = cols // 256
        d = (torch.rand((rows, nb), generator=g, device=device) * 2e-4).half().view(torch.int16)
        m = torch.randint(0, 64, (rows, cols // 32), generator=g, device=device, dtype=torch.uint8)
        sc = torch.randint(16, 64, (rows, cols // 32), generator=g, device=device, dtype=torch.uint8)
        q = torch.randint(0, 16, (rows, cols), generator=g, device=device, dtype=torch.uint8)
        return q4k.q4k_pack(d, d, sc, m, q)

    nq, nk = heads * head_dim, kv_heads * head_dim
    weights = {"q": packed(nq, hidden), "k": packed(nk, hidden), "v": packed(nk, hidden), "o": packed(hidden, nq)}
    f = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    freq = 1e6 ** (-torch.arange(0, head_dim, 2, device=device, dtype=torch.float64) / head_dim)
    angle = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] * freq
    cache = [torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=dtype, device=device) for _ in range(2)]
    lora = None
    if adapters:
        lora = {n: ((f(adapters, rank, c) * c ** -0.5).to(dtype), (f(adapters, r, rank) * 0.1).to(dtype))
                for n, r, c in (("q", nq, hidden), ("k", nk, hidden), ("v", nk, hidden), ("o", hidden, nq))}
    return AttentionBlock(weights, hidden, heads, kv_heads, head_dim, (1 + 0.1 * f(head_dim), 1 + 0.1 * f(head_dim)),
                          torch.cat([angle.cos(), angle.sin()], 1).float(), cache, lora,
                          torch.full((max(adapters, 1),), 2.0, device=device)[:adapters] if adapters else None)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--page", type=int, default=16)
    ap.add_argument("--experts", type=int, default=0, help="routed experts behind the attention block (0: none)")
    ap.add_argument("--top-k", type=int, default=8, help="experts of a token")
    ap.add_argument("--width", type=int, default=768, help="width of an expert")
    a = ap.parse_args()
    q4k.build()
    max_pages = -(-(a.prompt + a.steps) // a.page)
    pages = Pages(a.requests * max_pages, a.page, max_pages)
    block = random_block(a.hidden, a.heads, a.kv_heads, a.head_dim, a.requests * max_pages, a.page,
                         max_pages * a.page, torch.bfloat16, adapters=2)
    experts = None
    if a.experts:
        from q4_weight_matmul_gb300.expert_block import random_experts
        experts = random_experts(a.hidden, a.width, a.experts, a.top_k)

    def layer(x, step, max_q, segments, work=None):
        y = block(x, step, max_q, segments, work)
        return y if experts is None else experts(y, work=work)

    adapter = [r % 3 - 1 for r in range(a.requests)]              # none, the first, the second, none, ...

    def timed(fn):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        out = fn()
        end.record()
        torch.cuda.synchronize()
        return out, start.elapsed_time(end) * 1e3

    # the prompts, one chunk each (of different lengths)
    new = {r: max(1, a.prompt - 7 * r) for r in range(a.requests)}
    step = {k: v.cuda() for k, v in pages.step(new).items()}
    x = torch.randn((sum(new.values()), a.hidden), device="cuda")
    segments = q4k.q4k_lora_segments([adapter[r] for r, n in new.items() for _ in range(n)])
    y, us = timed(lambda: layer(x, step, max(new.values()), segments))
    print(f"prompt: {x.shape[0]} tokens, {us:.0f} us (first call)")

    # decoding: the step's arrays are copied into fixed buffers, the layer replays as a graph
    new = {r: 1 for r in range(a.requests)}
    x = torch.randn((a.requests, a.hidden), device="cuda")
    segments = q4k.q4k_lora_segments(adapter)
    buffers, graph, work = None, None, Workspaces()
    for i in range(a.steps):
        host = pages.step(new)
        if buffers is None:
            buffers = {k: v.cuda() for k, v in host.items()}
            y = layer(x, buffers, 1, segments, work)               # makes the workspaces
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = layer(x, buffers, 1, segments, work)
        else:
            for k, v in host.items():
                buffers[k].copy_(v)
        _, us = timed(graph.replay)
        print(f"decode step {i}: {a.requests} tokens, {us:.1f} us")
    if q4k.q4k_device_error() != 0:
        raise RuntimeError("a kernel reported an error")
    print("output norm", float(y.norm()))


if __name__ == "__main__":
    main()
