"""Cases of the operators around the expert layer: rotating and appending to a
paged cache (moe_kv_append), attention of drafted tokens over that cache
(moe_tree_attention) and routing by given scores with a bias and expert groups
(moe_route_scores).

`run` computes a case in plain torch where `own` is false, and through the
library where it is true.  `exact` states the operators again in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ---------------------------------------------------------------
def listed():
    return [
        # one request's next token on its way into the cache: latency only
        dict(name="append 1 token", op="append", tokens=1, heads=32, kv_heads=4, head_dim=128, rot=128, page=16,
             interleaved=False, fused=True, dtype="bf16"),
        # the drafted tokens of a whole decode batch (the library's largest batch)
        dict(name="append 256 drafted", op="append", tokens=256, heads=64, kv_heads=4, head_dim=128, rot=128, page=16,
             interleaved=False, fused=True, dtype="bf16"),
        # a long prompt's keys and values
        dict(name="append 16000 of a prompt", op="append", tokens=16000, heads=32, kv_heads=4, head_dim=128, rot=128,
             page=64, interleaved=False, fused=True, dtype="bf16"),
        # fp32, half of each head rotated in adjacent pairs, separate projections, an odd count
        dict(name="append 1537 fp32 pairs", op="append", tokens=1537, heads=16, kv_heads=2, head_dim=64, rot=32, page=32,
             interleaved=True, fused=False, dtype="f32"),
        # a single user's next token after about a page of text: latency only
        dict(name="attend 1x1 at 1000", op="attend", requests=1, drafts=1, tree=False, ctx_min=1000, ctx_max=1000,
             heads=32, kv_heads=4, head_dim=128, page=16, dtype="bf16", lens=1),
        # an ordinary decode batch without drafts, contexts of all lengths
        dict(name="attend 64x1 to 8000", op="attend", requests=64, drafts=1, tree=False, ctx_min=0, ctx_max=8000,
             heads=32, kv_heads=4, head_dim=128, page=16, dtype="bf16", lens=2),
        # 16 requests with a tree of up to 16 drafted tokens each
        dict(name="attend 16x16 tree to 4000", op="attend", requests=16, drafts=16, tree=True, ctx_min=100, ctx_max=4000,
             heads=32, kv_heads=4, head_dim=128, page=16, dtype="bf16", lens=3),
        # one request, a 64-node tree over a long document
        dict(name="attend 1x64 tree at 131000", op="attend", requests=1, drafts=64, tree=True, ctx_min=131000,
             ctx_max=131000, heads=32, kv_heads=4, head_dim=128, page=64, dtype="bf16", lens=4),
        # fp32 with small heads, a chain of drafts (causal)
        dict(name="attend 4x7 fp32 to 2000", op="attend", requests=4, drafts=7, tree=False, ctx_min=1, ctx_max=2000,
             heads=8, kv_heads=2, head_dim=64, page=16, dtype="f32", lens=5),
        # the largest decode batch with long contexts
        dict(name="attend 256x1 to 16000", op="attend", requests=256, drafts=1, tree=False, ctx_min=500, ctx_max=16000,
             heads=64, kv_heads=4, head_dim=128, page=16, dtype="bf16", lens=6),
        # one token, softmax scores renormalised over the 8 kept, no groups
        dict(name="route 1 of 128", op="route", tokens=1, experts=128, k=8, score="softmax", bias=False, groups=1,
             topk_groups=1, group_top=1, renormalise=True, scale=1.0),
        # the largest batch, sigmoid scores with a balance bias, 4 of 8 groups
        dict(name="route 256 of 256 grouped", op="route", tokens=256, experts=256, k=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, renormalise=True, scale=2.5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "route"])
    if op == "append":
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 5, 8, 16])
        heads, D = kv * group, rng.choice([64, 80, 128, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        most = 16000 * 40 * 128 * 2 // ((heads + 2 * kv) * D * (2 if dtype == "bf16" else 4))
        return dict(op="append", tokens=_log_int(rng, 1, min(16000, most)), heads=heads, kv_heads=kv, head_dim=D,
                    rot=rng.choice([D, D, D // 2, D // 4]), page=rng.choice([8, 16, 32, 64, 128]),
                    interleaved=rng.random() < 0.4, fused=group > 1 and rng.random() < 0.7, dtype=dtype)
    if op == "attend":
        dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
        D = rng.choice([64, 128, 128, 128])
        kv = rng.choice([1, 2, 4, 4, 8])
        group = rng.choice([1, 2, 4, 5, 8, 8, 16])
        R = _log_int(rng, 1, 256)
        n = min(_log_int(rng, 1, 64), max(1, 512 // R))
        # keys of all requests times their heads: at most 5 million rows, and for the rows that attend to them a bound
        # on the products as well
        room = min(5_000_000 // (R * kv), int(1e11 / (R * n * kv * group * D * (8 if dtype == "f32" else 1))))
        top = _log_int(rng, 1, max(1, min(131000, room)))
        return dict(op="attend", requests=R, drafts=n, tree=n > 1 and rng.random() < 0.6,
                    ctx_min=rng.choice([0, top // 8, top]), ctx_max=top, heads=kv * group, kv_heads=kv, head_dim=D,
                    page=rng.choice([8, 16, 16, 32, 64, 128]), dtype=dtype, lens=rng.randrange(1 << 20))
    groups = rng.choice([1, 1, 2, 4, 8])
    N = groups * rng.choice([8, 12, 16, 20, 32, 40, 64])
    topk_groups = max(1, groups // 2)
    sig = groups > 1 or rng.random() < 0.5
    return dict(op="route", tokens=_log_int(rng, 1, 256), experts=N, k=rng.randint(1, min(16, topk_groups * (N // groups))),
                score="sigmoid" if sig else "softmax", bias=sig and rng.random() < 0.7, groups=groups,
                topk_groups=topk_groups, group_top=rng.choice([1, 2]) if sig else 1, renormalise=rng.random() < 0.7,
                scale=rng.choice([1.0, 2.5]))


# ---- lengths and trees (from the case alone, so that work() knows them) --------
def _lengths(case):
    """(context length, drafted tokens) of every request."""
    rng = random.Random(case["lens"])
    ctx = [rng.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["requests"])]
    n = [rng.randint((case["drafts"] + 1) // 2, case["drafts"]) for _ in range(case["requests"])]
    if case["requests"] == 1:
        n = [case["drafts"]]
    return ctx, n


def _trees(case, n):
    """Words of 32 bits: bit j of token i's row says that i sees drafted token j of its request.  Each token's parent
    is one of the few before it."""
    rng = random.Random(case["lens"] + 1)
    words = (max(n) + 31) // 32
    rows = []
    for nr in n:
        seen = []
        for i in range(nr):
            bits = 1 << i
            if i:
                bits |= seen[rng.randint(max(0, i - 6), i - 1)]
            seen.append(bits)
            rows.append([(bits >> (32 * w)) & 0xffffffff for w in range(words)])
    return torch.tensor(rows, dtype=torch.int64).to(torch.int32)


# ---- what a user's program has in hand ---------------------------------------
def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        s.update(_handles(case, s))
    return s


def _handles(case, s):
    """The descriptors and scratch of the library that a program makes once."""
    import aware_expert_routing_gb300 as moe
    if case["op"] == "route":
        params = moe.RouteParams(B=case["tokens"], d=2048, N=case["experts"], k=case["k"])
        select = moe.SelectParams(score=moe.SCORE_SIGMOID if case["score"] == "sigmoid" else moe.SCORE_SOFTMAX,
                                  n_group=case["groups"], topk_group=case["topk_groups"], group_top=case["group_top"],
                                  renormalise=case["renormalise"], scale=case["scale"])
        return {"params": params, "select": select, "routing": moe.Routing(params, "cuda", with_n_base=False),
                "workspace": moe.alloc_workspace(params, 0, "cuda")}
    cache = moe.KvCache(s["cache_k"], s["cache_v"], s["page_table"])
    return {"cache": cache, "workspace": moe.alloc_attention_workspace(s["q"].shape[0], case["heads"], cache, "cuda")}


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "append":
        T, H, K, D, dt = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
        if case["fused"]:      # slices of one projection's output
            qkv = _normal(g, (T, H + 2 * K, D), dt)
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        else:
            s["q"], s["k"], s["v"] = (_normal(g, (T, h, D), dt) for h in (H, K, K))
        # the rotation table of a context of 32768 positions: cos, then sin, of pos / 1e6^(2i / rot)
        half = case["rot"] // 2
        freq = 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(32768, device="cuda", dtype=torch.float64)[:, None] * freq
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
        start = int(torch.randint(0, 32768 - T, (1,), generator=g, device="cuda").item())
        s["positions"] = torch.arange(start, start + T, device="cuda", dtype=torch.int32)
        # pages handed out in the allocator's order, some pages of other requests between them
        pages = (T + case["page"] - 1) // case["page"]
        table = torch.randperm(pages + 8, generator=g, device="cuda")[:pages]
        at = torch.arange(T, device="cuda")
        s["slots"] = table[at // case["page"]] * case["page"] + at % case["page"]
        shape = (pages + 8, K, case["page"], D)
        s["cache_k"], s["cache_v"] = _normal(g, shape, dt), _normal(g, shape, dt)
        s["page_table"] = table[None].to(torch.int32)
        s["q_out"] = torch.empty(T, H, D, dtype=dt, device="cuda")
    elif case["op"] == "attend":
        H, K, D, dt, page = case["heads"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]], case["page"]
        ctx, n = _lengths(case)
        per = [(c + m + page - 1) // page for c, m in zip(ctx, n)]
        order = torch.randperm(sum(per) + 4, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(len(ctx), max(per), dtype=torch.int32, device="cuda")
        have = torch.arange(max(per), device="cuda")[None] < torch.tensor(per, device="cuda")[:, None]
        table[have] = order[:sum(per)]
        shape = (sum(per) + 4, K, page, D)
        s["cache_k"], s["cache_v"], s["page_table"] = _normal(g, shape, dt), _normal(g, shape, dt), table
        s["q"] = _normal(g, (sum(n), H, D), dt, 2.0)
        s["ctx_len"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["q_offsets"] = torch.tensor([0] + n, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        s["mask"] = _trees(case, n).cuda() if case["tree"] else None
        s["most"], s["longest"] = max(n), max(c + m for c, m in zip(ctx, n))
        s["out"] = torch.empty(sum(n), H, D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(sum(n), H, dtype=torch.float32, device="cuda")
    else:
        B, N = case["tokens"], case["experts"]
        # router scores of unlike experts, and the bias that balancing them has learnt
        s["scores"] = _normal(g, (B, N), torch.float32, 1.5) + _normal(g, (N,), torch.float32, 0.5)
        s["bias"] = _normal(g, (N,), torch.float32, 0.1) if case["bias"] else None
    return s


# ---- one pass ---------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "route": _plain_route}[op](s)
    import aware_expert_routing_gb300 as moe
    if op == "append":
        moe.moe_kv_append(s["q"], s["k"], s["v"], s["rope"], s["positions"], s["slots"], s["cache"], s["q_out"],
                          s["workspace"], interleaved=s["case"]["interleaved"])
        return {"q": s["q_out"], "k": s["cache_k"], "v": s["cache_v"]}
    if op == "attend":
        moe.moe_tree_attention(s["q"], s["q_offsets"], s["ctx_len"], s["mask"], s["cache"], s["out"], s["lse"],
                               s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    r = s["routing"]
    moe.moe_route_scores(s["scores"], s["bias"], s["params"], s["select"], r, s["workspace"])
    return {n: getattr(r, n) for n in ("expert_idx", "weights", "T", "active", "counts", "offsets", "perm")}


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    case, ck, cv = s["case"], s["cache_k"], s["cache_v"]
    rot, page = case["rot"], case["page"]
    at = s["rope"][s["positions"].long()][:, None]
    cos, sin = at[..., :rot // 2], at[..., rot // 2:]
    pg, row = s["slots"] // page, s["slots"] % page
    ck[pg, :, row] = _rotate(s["k"], cos, sin, rot, case["interleaved"]).to(ck.dtype)
    cv[pg, :, row] = s["v"]
    return {"q": _rotate(s["q"], cos, sin, rot, case["interleaved"]).to(s["q"].dtype), "k": ck, "v": cv}


def _plain_attend(s):
    q, ck, cv, off, ctx = s["q"], s["cache_k"], s["cache_v"], s["q_offsets"].long(), s["ctx_len"].long()
    R, n, L = ctx.numel(), s["most"], s["longest"]
    T, H, D = q.shape
    K, page = ck.shape[1], ck.shape[2]
    dev = q.device
    cnt = off[1:] - off[:-1]
    i = torch.arange(n, device=dev)
    tok = (off[:-1, None] + i).clamp(max=T - 1)                              # [R, n]
    j = torch.arange(L, device=dev)
    pg = s["page_table"][:, :(L + page - 1) // page].long()                     # [R, pages]
    keys = ck[pg].float().permute(0, 2, 1, 3, 4).reshape(R, K, -1, D)[:, :, :L]
    vals = cv[pg].float().permute(0, 2, 1, 3, 4).reshape(R, K, -1, D)[:, :, :L]
    d = j[None, :] - ctx[:, None]                                            # [R, L]: which drafted token, below 0: context
    if s["mask"] is None:
        draft = d[:, None, :] <= i[None, :, None]
    else:
        dd = d.clamp(0, n - 1)
        word = s["mask"][tok].gather(2, (dd // 32)[:, None, :].expand(R, n, L))
        draft = ((word >> (dd % 32)[:, None, :].to(torch.int32)) & 1).bool()
    seen = (d < 0)[:, None, :] | (draft & (d < cnt[:, None])[:, None, :])    # [R, n, L]
    qr = q[tok].float().reshape(R, n, K, H // K, D).permute(0, 2, 1, 3, 4).reshape(R, K, n * (H // K), D)
    x = (qr @ keys.transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = x.reshape(R, K, n, H // K, L).masked_fill(~seen[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    x = (x - m).exp()
    z = x.sum(-1, keepdim=True)
    o = x.reshape(R, K, n * (H // K), L) @ torch.where((d < cnt[:, None])[:, None, :, None], vals, torch.zeros_like(vals))
    o = o.reshape(R, K, n, H // K, D) / torch.where(z == 0, torch.ones_like(z), z)
    lse = (z.log() + m)[..., 0]
    live = i[None, :] < cnt[:, None]                                         # [R, n]
    out = o.permute(0, 2, 1, 3, 4).reshape(R, n, H, D)[live].to(q.dtype)
    return {"out": out, "lse": lse.permute(0, 2, 1, 3).reshape(R, n, H)[live]}


def _plain_route(s):
    case, x, bias = s["case"], s["scores"], s["bias"]
    B, N = x.shape
    G, k = case["groups"], case["k"]
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + (-x).exp())
    else:
        e = (x - x.amax(1, keepdim=True)).exp()
        p = e / e.sum(1, keepdim=True)
    # the softmax keeps the scores' order
    sel = p if bias is None else p + bias
    if case["score"] == "softmax" and bias is None and case["group_top"] == 1:
        sel = x
    if G > 1:
        grouped = sel.reshape(B, G, N // G)
        value = grouped.sort(dim=-1, descending=True).values[..., :case["group_top"]].sum(-1)
        kept = value.sort(dim=-1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        ok = torch.zeros(B, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        sel = grouped.masked_fill(~ok[..., None], float("-inf")).reshape(B, N)
    idx = sel.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, idx)
    if case["renormalise"]:
        z = w.sum(1, keepdim=True)
        w = w / torch.where(z == 0, torch.ones_like(z), z)
    return _grouping(idx, w * case["scale"], N)


def _grouping(idx, w, N):
    """The (token, slot) pairs grouped by expert, as the expert kernels read them."""
    flat = idx.reshape(-1)
    counts = (flat[None, :] == torch.arange(N, device=idx.device)[:, None]).sum(1)
    used = counts > 0
    order = torch.where(used, torch.arange(N, device=idx.device), N).sort().values
    return {"expert_idx": idx.to(torch.int32), "weights": w, "T": used.sum()[None].to(torch.int32),
            "active": torch.where(order < N, order, -1).to(torch.int32), "counts": counts.to(torch.int32),
            "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32),
            "perm": flat.sort(stable=True).indices.to(torch.int32)}


# ---- what a pass cannot do without -----------------------------------------------
def work(case):
    if case["op"] == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
        return {"bytes": T * (2 * (H + 2 * K) * D * e + 4 * case["rot"] + 12), "flops": 3 * T * (H + K) * case["rot"]}
    if case["op"] == "attend":
        e = 2 if case["dtype"] == "bf16" else 4
        ctx, n = _lengths(case)
        H, K, D, T = case["heads"], case["kv_heads"], case["head_dim"], sum(n)
        keys = sum(c + m for c, m in zip(ctx, n))
        return {"bytes": 2 * keys * K * D * e + 2 * T * H * D * e + 4 * T * H + 4 * keys // case["page"],
                "flops": 4 * D * H * sum(m * (c + m) for c, m in zip(ctx, n))}
    B, N, k = case["tokens"], case["experts"], case["k"]
    return {"bytes": 4 * (B * N + N + 3 * B * k + 3 * N + 2), "flops": B * N * (4 + k)}


# ---- the same in 64 bits ------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return _exact_route(case, s)


def _exact_append(case, s):
    """Each pair (a, b) as a complex number times cos + i sin."""
    rot, page, half = case["rot"], case["page"], case["rot"] // 2
    t = s["rope"].double().index_select(0, s["positions"].long())
    turn = torch.complex(t[:, :half], t[:, half:])[:, None, :]

    def turned(x):
        y = x.double().clone()
        if case["interleaved"]:
            at = (slice(0, rot, 2), slice(1, rot, 2))
        else:
            at = (slice(0, half), slice(half, rot))
        z = torch.complex(y[..., at[0]].contiguous(), y[..., at[1]].contiguous()) * turn
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
        return y

    k, v = (x.double().permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["head_dim"]).clone()
            for x in (s["cache_k"], s["cache_v"]))
    k.index_copy_(0, s["slots"], turned(s["k"]))
    v.index_copy_(0, s["slots"], s["v"].double())
    back = lambda x: x.reshape(-1, page, case["kv_heads"], case["head_dim"]).permute(0, 2, 1, 3).contiguous()  # noqa: E731
    return {"q": turned(s["q"]), "k": back(k), "v": back(v)}


def _exact_attend(case, s):
    """Request by request and key head by key head, over the keys that the request has."""
    ctx, n = _lengths(case)
    H, K, D, page = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    out = torch.zeros(sum(n), H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(n), H, dtype=torch.float64, device="cuda")
    t0 = 0
    for r, (c, m) in enumerate(zip(ctx, n)):
        L = c + m
        where = s["page_table"][r].long()[torch.arange(L, device="cuda") // page]
        row = torch.arange(L, device="cuda") % page
        see = torch.ones(m, L, dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            see[:, c:] = torch.tril(torch.ones(m, m, dtype=torch.bool, device="cuda"))
        else:
            words = s["mask"][t0:t0 + m].long() & 0xffffffff
            at = torch.arange(m, device="cuda")
            see[:, c:] = (words[:, at // 32] >> (at % 32)) & 1 != 0
        for h in range(K):
            key, val = s["cache_k"][where, h, row].double(), s["cache_v"][where, h, row].double()
            heads = slice(h * (H // K), (h + 1) * (H // K))
            x = torch.einsum("tgd,ld->tgl", s["q"][t0:t0 + m, heads].double(), key) / math.sqrt(D)
            x = x.masked_fill(~see[:, None, :], float("-inf"))
            lse[t0:t0 + m, heads] = torch.logsumexp(x, -1)
            out[t0:t0 + m, heads] = torch.einsum("tgl,ld->tgd", torch.softmax(x, -1).nan_to_num(0.0), val)
        t0 += m
    return {"out": out, "lse": lse}


def _exact_route(case, s):
    """Token by token; only the weights are computed numbers."""
    x = s["scores"].double().cpu()
    bias = None if s["bias"] is None else s["bias"].double().cpu()
    B, N = x.shape
    per, weights = N // case["groups"], []
    for b in range(B):
        p = torch.sigmoid(x[b]) if case["score"] == "sigmoid" else torch.softmax(x[b], 0)
        sel = (p if bias is None else p + bias).tolist()
        group = [sum(sorted(sel[i * per:(i + 1) * per], reverse=True)[:case["group_top"]]) for i in range(case["groups"])]
        kept = set(sorted(range(case["groups"]), key=lambda i: (-group[i], i))[:case["topk_groups"]])
        best = sorted((e for e in range(N) if e // per in kept), key=lambda e: (-sel[e], e))[:case["k"]]
        w = p[best]
        weights.append((w / w.sum() if case["renormalise"] else w) * case["scale"])
    return {"expert_idx": None, "weights": torch.stack(weights), "T": None, "active": None, "counts": None,
            "offsets": None, "perm": None}
