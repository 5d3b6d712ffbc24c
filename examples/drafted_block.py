"""One decoder block for drafted tokens, with the library's calls in the order
in which a server makes them: rotate and append the step's keys and values,
attend from every drafted token to its request's cache, route by sigmoid
scores with a balance bias and expert groups, run the experts.

    python examples/drafted_block.py

Weights are random, the projections are plain torch products.  Prints what
the step did and how long it takes.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import aware_expert_routing_gb300 as moe  # noqa: E402


class Block:
    """Attention over a paged cache, then the expert layer."""

    def __init__(self, d=2048, heads=32, kv_heads=4, head_dim=128, experts=128, k=8, d_ff=768, pages=2048, page=16,
                 max_tokens=64, requests=4, max_len=4096, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def w(*shape, scale):
            return (torch.randn(shape, generator=g, device=device) * scale).to(torch.bfloat16)

        self.d, self.heads, self.kv_heads, self.head_dim, self.d_ff, self.page = d, heads, kv_heads, head_dim, d_ff, page
        self.experts, self.k = experts, k
        self.w_qkv = w((heads + 2 * kv_heads) * head_dim, d, scale=d ** -0.5)
        self.w_out = w(d, heads * head_dim, scale=(heads * head_dim) ** -0.5)
        self.w_router = w(experts, d, scale=d ** -0.5)
        self.balance = torch.randn(experts, generator=g, device=device) * 0.05
        gate_up = w(2, experts, d_ff, d, scale=d ** -0.5)
        self.w_gate, self.w_up = gate_up[0], gate_up[1]
        self.w_down = w(experts, d, d_ff, scale=d_ff ** -0.5)
        self.rope = moe.moe_rope_table(moe.RopeParams(rot=head_dim, base=1e6), max_len, device)
        # the pages, and each request's table: pages are handed out in turn
        shape = (pages, kv_heads, page, head_dim)
        self.table = torch.arange(requests * (max_len // page), device=device, dtype=torch.int32).reshape(requests, -1) % pages
        self.cache = moe.KvCache(torch.zeros(shape, dtype=torch.bfloat16, device=device),
                                 torch.zeros(shape, dtype=torch.bfloat16, device=device), self.table)
        self.scratch = moe.alloc_attention_workspace(max_tokens, heads, self.cache, device)
        self.select = moe.SelectParams(score=moe.SCORE_SIGMOID, n_group=8, topk_group=4, group_top=2, scale=2.5)

    def step(self, x, ctx_len, q_offsets, depth, request, mask):
        """x [T][d]: the drafted tokens' hidden states.  Token t of request r is `depth[t]` positions past its
        context (its place in the tree) and the (t - q_offsets[r])-th of the request's new rows in the cache."""
        T, D = x.shape[0], self.head_dim
        qkv = (x @ self.w_qkv.T).view(T, -1, D)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        positions = ctx_len[request] + depth
        row = ctx_len[request] + torch.arange(T, device=x.device, dtype=torch.int32) - q_offsets[request]
        slots = self.table[request.long(), (row // self.page).long()].long() * self.page + row % self.page
        q_rot = torch.empty(T, self.heads, D, dtype=x.dtype, device=x.device)
        moe.moe_kv_append(q, k, v, self.rope, positions, slots, self.cache, q_rot, self.scratch)
        out = torch.empty_like(q_rot)
        moe.moe_tree_attention(q_rot, q_offsets, ctx_len, mask, self.cache, out, None, self.scratch)
        x = x + out.view(T, -1) @ self.w_out.T
        params = moe.RouteParams(B=T, d=self.d, N=self.experts, k=self.k)
        if getattr(self, "routing", None) is None or self.routing.expert_idx.shape[0] != T:
            self.routing = moe.Routing(params, x.device)
            self.ws = moe.alloc_workspace(params, self.d_ff, x.device)
        y = torch.empty_like(x)
        moe.moe_decode_layer_grouped(x, self.w_router, None, self.balance, self.w_gate, self.w_up, self.w_down, self.d_ff,
                                     params, self.select, self.routing, y, self.ws)
        return x + y


def drafted(parents, device="cuda"):
    """(q_offsets, depth, request, mask) of the requests' drafted trees, each given by its tokens' parents (-1: the
    context's last token)."""
    offsets, depth, request, masks = [0], [], [], []
    words = (max(len(p) for p in parents) + 31) // 32
    for r, p in enumerate(parents):
        at = []
        for q in p:
            at.append(at[q] + 1 if q >= 0 else 0)
        m = moe.tree_mask(p)
        masks.append(torch.nn.functional.pad(m, (0, words - m.shape[1])))
        depth += at
        request += [r] * len(p)
        offsets.append(offsets[-1] + len(p))
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
    return as_int(offsets), as_int(depth), as_int(request), torch.cat(masks).to(device).contiguous()


def main():
    block = Block()
    # four requests: a tree, a chain, a single token, a wider tree
    parents = [[-1, 0, 0, 1, 1, 2, 3], [-1, 0, 1, 2], [-1], [-1, 0, 0, 0, 1, 1, 2, 2, 3, 4]]
    q_offsets, depth, request, mask = drafted(parents)
    T = int(q_offsets[-1])
    ctx_len = torch.tensor([1500, 40, 3000, 0], dtype=torch.int32, device="cuda")
    # contexts that earlier steps have left in the cache
    block.cache.k.normal_()
    block.cache.v.normal_()
    x = torch.randn(T, block.d, device="cuda").to(torch.bfloat16)
    y = block.step(x, ctx_len, q_offsets, depth, request, mask)
    flags = moe.moe_device_status(block.scratch) | moe.moe_device_status(block.ws)
    assert flags == 0 and bool(torch.isfinite(y).all())
    print(f"{T} drafted tokens of {len(parents)} requests, {int(block.routing.T.item())} experts activated")

    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(5):
        block.step(x, ctx_len, q_offsets, depth, request, mask)
    start.record()
    for _ in range(50):
        block.step(x, ctx_len, q_offsets, depth, request, mask)
    end.record()
    end.synchronize()
    flags = moe.moe_device_status(block.scratch) | moe.moe_device_status(block.ws)
    assert flags == 0
    print(f"a step takes {start.elapsed_time(end) * 20:.1f} us, most of it the host's")


if __name__ == "__main__":
    main()
