"""The feed-forward part of a decoder layer with routed experts on this
library's calls: the router's choice, the gated products of every token's
experts, and their weighted down projections with the residual.

``python -m q4_weight_matmul_gb300.attention_block --experts 128`` runs it
behind the attention block, prompts and captured decode steps alike.
"""
from __future__ import annotations

import torch

import q4_weight_matmul_gb300 as q4k
from q4_weight_matmul_gb300.attention_block import Workspaces


class ExpertBlock:
    """``router`` [experts][hidden] float32 (its logits are torch's product, in
    TF32 where the process lets torch's matmuls use it: tokens whose experts'
    logits lie close together may then go to others); ``gate``, ``up``: the experts'
    packed Q4_K matrices, [experts][width] rows of ``hidden`` weights;
    ``down``: [experts][hidden] rows of ``width``, packed Q4_K or (``q6k``)
    Q6_K in the GPU layout."""

    def __init__(self, router, gate, up, down, width, top_k, q6k=False, renormalize=True, scale=1.0):
        self.router, self.gate, self.up, self.down, self.width = router, gate, up, down, width
        self.top_k, self.q6k, self.renormalize, self.scale = top_k, q6k, renormalize, scale
        self.work = {}                      # stream handle -> its Workspaces

    def __call__(self, x, residual=None, n_tokens=None, work=None):
        """``x`` [tokens][hidden] float32 (normed input); ``residual``: what
        the experts' sum is added to, ``x`` without it; ``n_tokens``: None, or
        int32 [1] on the device: the rows of a padded batch from there on hold
        no tokens, and come back as the residual's; ``work``: the
        ``Workspaces`` to use (those of an attention block serve too).  Without
        it every stream has its own, and a call that is captured makes some for
        itself, which the graph keeps."""
        capturing = torch.cuda.is_current_stream_capturing()
        for_graph = capturing and work is not None
        if work is None:
            key = torch.cuda.current_stream().cuda_stream
            work = Workspaces() if capturing else self.work.setdefault(key, Workspaces())
        experts, hidden = self.router.shape
        size = x.shape[0], self.top_k, experts, hidden, self.width
        space = work.get("moe", q4k.q4k_moe_workspace_bytes(*size), lambda: q4k.q4k_moe_workspace(*size), for_graph)
        residual = x if residual is None else residual
        route = q4k.q4k_moe_route(x @ self.router.t(), self.top_k, self.renormalize, self.scale, n_tokens, workspace=space)
        h = q4k.q4k_moe_gate_up(x, self.gate, self.up, self.width, route, workspace=space)
        return q4k.q4k_moe_down(h, self.down, hidden, route, residual, self.q6k,
                                out=None if n_tokens is None else residual.clone(), workspace=space)


def random_experts(hidden, width, experts, top_k, q6k=False, seed=0, device="cuda"):
    """A block with random weights of the given shape: for timing and examples."""
    g = torch.Generator(device=device).manual_seed(seed)

    def matrix(rows, cols, six=False):
        i = lambda lo, hi, n, t=torch.uint8: torch.randint(lo, hi, (rows, n), generator=g, device=device, dtype=t)  # noqa: E731
        d = (torch.rand((rows, cols // 256), generator=g, device=device) * (2e-5 if six else 2e-4)).half().view(torch.int16)
        if six:
            return q4k.q6k_pack(d, i(-128, 128, cols // 16, torch.int8), i(0, 64, cols))
        return q4k.q4k_pack(d, d, i(16, 64, cols // 32), i(0, 64, cols // 32), i(0, 16, cols))

    router = torch.randn((experts, hidden), generator=g, device=device) * hidden ** -0.5
    return ExpertBlock(router, matrix(experts * width, hidden), matrix(experts * width, hidden),
                       matrix(experts * hidden, width, q6k), width, top_k, q6k)
