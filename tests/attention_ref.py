"""Plain 64-bit statements of the operators around the expert layer, with the
bounds that their fp32 (and bf16) forms have to keep.  Used by the tests of
moe_kv_append, moe_tree_attention and moe_route_scores."""
from __future__ import annotations

import math

import numpy as np
import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8    # unit roundoff of fp32 and bf16 (24 and 8 significant bits)


def rotate(x, table, positions, interleaved):
    """(rotated x, bound of the fp32 form's error) of x [T][H][D] in fp64."""
    rot = table.shape[1]
    x = x.double()
    y = x.clone()
    if rot == 0:
        return y, torch.zeros_like(x)
    c, s = (t[:, None] for t in table.double()[positions.long()].split(rot // 2, 1))
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    # two products and a sum, each rounded once
    e = torch.zeros_like(x)
    e[..., a] = e[..., b] = 2 * U32 * ((x[..., a] * c).abs() + (x[..., b] * s).abs()).maximum(
        (x[..., b] * c).abs() + (x[..., a] * s).abs())
    return y, e


def rope_frequencies(rot, base, scaling="plain", factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """(f_i, magnitude) in Python floats, from the published formulas."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "yarn":
        def index(beta):
            return rot * math.log(original_len / (beta * 2 * math.pi)) / (2 * math.log(base))
        low = max(math.floor(index(beta_fast)), 0)
        high = min(math.ceil(index(beta_slow)), rot - 1)
        if low == high:
            high += 0.001
        far = [min(max((i - low) / (high - low), 0.0), 1.0) for i in range(rot // 2)]
        return [x / factor * w + x * (1 - w) for x, w in zip(f, far)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def attend(q, k, v, table, q_offsets, ctx_len, mask, scale, bf16):
    """out, lse and the bounds of both, token by token, from the pages of the
    cache (all CPU tensors).  What a token does not see is not read."""
    q, k, v = q.double(), k.double(), v.double()
    T, H, D = q.shape
    G, page = H // k.shape[1], k.shape[2]
    out, lse = torch.zeros(T, H, D, dtype=torch.float64), torch.full((T, H), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(ctx_len)):
        t0, t1, ctx = int(q_offsets[r]), int(q_offsets[r + 1]), int(ctx_len[r])
        j = torch.arange(ctx + max(t1 - t0, 0))
        if j.numel() == 0:
            continue
        pg, row = table[r].long()[j // page], j % page
        kr, vr = k[pg, :, row].repeat_interleave(G, 1), v[pg, :, row].repeat_interleave(G, 1)   # [L][H][D]
        for t in range(t0, t1):
            if mask is None:
                see = j <= ctx + t - t0
            else:
                d = (j - ctx).clamp(min=0)
                words = mask[t].long() & 0xffffffff
                ok = d < 32 * len(words)
                see = (j < ctx) | (ok & (((words[(d // 32).clamp(max=len(words) - 1)] >> (d % 32)) & 1) != 0))
            if not see.any():
                continue
            x = torch.einsum("hd,lhd->lh", q[t], kr[see]) * scale
            p = torch.softmax(x, 0)
            out[t] = torch.einsum("lh,lhd->hd", p, vr[see])
            lse[t] = torch.logsumexp(x, 0)
            A = torch.einsum("lh,lhd->hd", p, vr[see].abs())
            # each score: D products and sums; each exponential: its argument and the function (2^-20); the sums: one
            # rounding a term (the tensor cores' may cut off, hence twice)
            es = (D + 2) * 2 * U32 * scale * torch.einsum("hd,lhd->lh", q[t].abs(), kr[see].abs()).amax(0)
            e = 2 * es + 2.0 ** -20 + x.shape[0] * 2 * U32
            tol_o[t] = A * e[:, None] + (U16 * 1.05 * (A + out[t].abs()) if bf16 else 2 * U32 * out[t].abs())
            tol_l[t] = es + 2.0 ** -20 + x.shape[0] * 2 * U32 + 4 * U32 * lse[t].abs()
    return out, lse, tol_o, tol_l


def select(scores, bias, k, sigmoid, n_group, topk_group, group_top, renorm, scale, B_valid=None):
    """idx [B][k] (-1: unused) and weights [B][k] of moe_route_scores."""
    x = np.asarray(scores, np.float64)
    B, N = x.shape
    gs = N // n_group
    idx, w = np.full((B, k), -1, np.int32), np.zeros((B, k))
    for b in range(B if B_valid is None else B_valid):
        ok = np.isfinite(x[b])
        with np.errstate(over="ignore", invalid="ignore"):
            if sigmoid:
                p = 1 / (1 + np.exp(-x[b]))
            else:
                e = np.where(ok, np.exp(x[b] - x[b][ok].max(initial=-np.inf)), 0)
                p = e / e.sum()
            val = p if bias is None else p + np.asarray(bias, np.float64)
        ok &= np.isfinite(val)
        groups = []
        for g in range(n_group):
            m = sorted((val[e] for e in range(g * gs, (g + 1) * gs) if ok[e]), reverse=True)[:group_top]
            if m:
                groups.append((-sum(m), g))
        kept = {g for _, g in sorted(groups)[:topk_group]}
        best = sorted((-val[e], e) for e in range(N) if ok[e] and e // gs in kept)[:k]
        ids = [e for _, e in best]
        idx[b, :len(ids)] = ids
        z = sum(p[e] for e in ids) if renorm else 1.0
        w[b, :len(ids)] = [(p[e] / z if z > 0 else 0.0) * scale for e in ids]
    return idx, w


def grouping(idx, N):
    """T, active, counts, offsets and perm of the chosen experts."""
    flat = idx.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(N)], np.int32)
    act = np.nonzero(counts)[0]
    active = np.full(N, -1, np.int32)
    active[:len(act)] = act
    perm = [q for e in act for q in range(flat.size) if flat[q] == e]
    return len(act), active, counts, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), np.array(perm, np.int32)
