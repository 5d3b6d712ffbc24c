"""moe_tree_attention on calls whose (row tile, key tile) pairs are many
millions, most of them one request's: a long prompt's chunk beside short
requests.  A sample of the rows is checked against a 64-bit statement."""
import math

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("aware_expert_routing_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from aware_expert_routing_gb300 import build as b
    b.build()
    moe.load()


def row(q, k, v, scale, bf16):
    """out, lse and their bounds of one query over the keys that it sees, as attention_ref.attend states them."""
    q, k, v = q.double(), k.double(), v.double()
    x = (k @ q) * scale
    p = torch.softmax(x, 0)
    out, lse, A = p @ v, torch.logsumexp(x, 0), p @ v.abs()
    es = (q.numel() + 2) * 2 * ref.U32 * scale * (k.abs() @ q.abs()).amax()
    e = 2 * es + 2.0 ** -20 + x.numel() * 2 * ref.U32
    tol_o = A * e + (ref.U16 * 1.05 * (A + out.abs()) if bf16 else 2 * ref.U32 * out.abs())
    return out, lse, tol_o, es + 2.0 ** -20 + x.numel() * 2 * ref.U32 + 4 * ref.U32 * lse.abs()


# heads, key heads, page, tokens and context of the long request.  Steps of the line: 128 rows x 128 keys and up for
# bf16, 64 x 64 for fp32, so 5.7 and 8.6 million.
@pytest.mark.parametrize("dtype,H,K,page,n,ctx", [("bf16", 128, 8, 64, 16384, 73000), ("f32", 16, 2, 16, 24576, 66000)])
def test_a_long_chunk_is_answered_and_so_are_its_neighbours(dtype, H, K, page, n, ctx):
    D, dt = 64, torch.bfloat16 if dtype == "bf16" else torch.float32
    ctxs, ns = [40, ctx, 300], [2, n, 3]
    g = torch.Generator(device=DEV).manual_seed(7)
    per = [(c + m + page - 1) // page for c, m in zip(ctxs, ns)]
    order = torch.randperm(sum(per), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(3, max(per), dtype=torch.int32, device=DEV)
    at = 0
    for r, p in enumerate(per):
        table[r, :p] = order[at:at + p]
        at += p
    ck, cv = (torch.randn(sum(per), K, page, D, generator=g, device=DEV).to(dt) for _ in range(2))
    q = (torch.randn(sum(ns), H, D, generator=g, device=DEV) * 2).to(dt)
    off = torch.tensor([0, 2, 2 + n, 5 + n], dtype=torch.int32, device=DEV)
    cache = moe.KvCache(ck, cv, table)
    ws = moe.alloc_attention_workspace(q.shape[0], H, cache, DEV)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((q.shape[0], H), float("nan"), device=DEV)
    moe.moe_tree_attention(q, off, torch.tensor(ctxs, dtype=torch.int32, device=DEV), None, cache, out, lse, ws)
    assert moe.moe_device_status(ws) == 0
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    t0 = 0
    for r in range(3):
        c, m = ctxs[r], ns[r]
        where = torch.arange(c + m, device=DEV)
        pg, at = table[r].long()[where // page], where % page
        for i in sorted({0, 1, m // 3, m // 2, m - 2, m - 1}):
            for h in (0, H // 2 + 1, H - 1):
                kh, L = h // (H // K), c + i + 1
                o, e, to, te = row(q[t0 + i, h], ck[pg[:L], kh, at[:L]], cv[pg[:L], kh, at[:L]], 1 / math.sqrt(D), dtype == "bf16")
                assert ((out[t0 + i, h].double() - o).abs() <= to).all(), (r, i, h)
                assert (lse[t0 + i, h].double() - e).abs() <= te, (r, i, h)
        t0 += m


def test_a_call_past_the_limit_is_refused_as_a_whole():
    """1000 tokens of 1024 heads (4 row tiles each) over 525008 key tiles: above 2^31 pairs.  The flag, and nothing
    written, the short request's output included."""
    H, D, page, ctx = 1024, 64, 128, 67_200_000
    ck, cv = (torch.zeros(1, H, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.zeros(2, ctx // page + 9, dtype=torch.int32, device=DEV)      # all of them the one page
    cache = moe.KvCache(ck, cv, table)
    q = torch.ones(1001, H, D, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, float("nan"))
    ws = moe.alloc_attention_workspace(1001, H, cache, DEV)
    off, lens = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1, 1001], [5, ctx]))
    moe.moe_tree_attention(q, off, lens, None, cache, out, None, ws)
    assert moe.moe_device_status(ws) == moe.FLAG_BAD_INDEX
    assert bool(out.isnan().all())
