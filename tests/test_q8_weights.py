"""How exact the weights and the queries of moe_tree_attention_q8 are with up to 64 rows a key head (tensor cores).

Weights: off by 2^-11 of themselves for their way through f16 and 2^-14 for their three e4m3 parts, and by 2^-28 of the
tile's largest.  Two groups of keys, each with one score and one value a component, and values of opposite signs: where they nearly cancel,
what the weights are off by is not hidden behind the rounding of the result.

Queries: two e4m3 numbers of a power of two that the rows of a unit share, off by 2^-21 of the largest of its components.
One row is 2^14 to 2^17 times the others, whose components, all alike, add up what they are off by."""
import pytest
import torch

import attention_ref as ref
import q8_ref as q8

moe = pytest.importorskip("aware_expert_routing_gb300")
DEV = "cuda:0"
PART = 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -20     # (and the exponential's own)


def parts_of(w, parts):
    """Weights up to 1 as the sum of so many e4m3 numbers, from f16."""
    left = (w * 256).to(torch.float16).double()
    got = torch.zeros_like(left)
    for p in range(parts):
        c = q8.decode(q8.encode(left))
        got += c * 32.0 ** -p
        left = (left - c) * 32
    return got / 256


class Case:
    def __init__(self, tokens, H, D, page, ctx=300):
        self.D, self.page = D, page
        L, g = ctx + tokens, torch.Generator().manual_seed(H + D)
        pages = (L + page - 1) // page
        self.scale = D ** -0.5
        self.table = torch.randperm(pages, generator=g).to(torch.int32)[None]
        j = torch.arange(pages * page)
        pg, row = self.table[0].long()[j // page], j % page
        mags = [x for x in q8.VALUES[:127].tolist() if x >= 16]
        b = torch.tensor([mags[d % len(mags)] for d in range(D)])
        k, v = (torch.zeros(pages, 1, page, D, dtype=torch.float64) for _ in range(2))
        k[pg, 0, row, 0] = torch.where(j % 2 == 0, 0.0, -64.0).double()
        v[pg, 0, row] = torch.where(j[:, None] % 2 == 0, torch.full((D,), 16.0).double(), -b[torch.randperm(D, generator=g)].double())
        self.k, self.v = q8.encode(k), q8.encode(v)
        self.ks, self.vs = torch.full((pages, 1, page // 8), 2.0 ** -6), torch.full((pages, 1, page // 8), 2.0 ** -3)
        self.q = torch.zeros(tokens, H, D, dtype=torch.bfloat16)
        # queries whose weight of the second group two parts would be worst at, beside a value that cancels it
        a = torch.linspace(0.01, 3.2 / self.scale, 20000).to(torch.bfloat16).unique()
        w = torch.exp(-a.double() * self.scale)
        near = (w[:, None] * b.double() - 16).abs().min(1).values
        hardness = (w - parts_of(w, 2)).abs() * 16 / w / (PART * 32 + ref.U16 * near)
        self.q[..., 0] = a[hardness.topk(tokens * H).indices].reshape(tokens, H)
        self.off, self.ctx = torch.tensor([0, tokens], dtype=torch.int32), torch.tensor([ctx], dtype=torch.int32)

    def want(self):
        """(out, its bound) in 64 bits."""
        k, v = q8.dequantised(self.k, self.ks), q8.dequantised(self.v, self.vs)
        out = ref.attend(self.q, k, v, self.table, self.off, self.ctx, None, self.scale, True)[0]
        most = ref.attend(self.q, k, v.abs(), self.table, self.off, self.ctx, None, self.scale, True)[0]
        # scores: one product of D components that is not zero, and three factors; sums of L terms in fp32
        L = int(self.ctx[0]) + self.q.shape[0]
        score = float(self.q.double().abs().max()) * self.scale
        e = most * (PART + 2 * (2 * ref.U32 * 5 * score + L * 2 * ref.U32))
        return out, e + ref.U16 * (out.abs() + e)

    def rounded_weights(self, parts):
        """The result with weights of so many parts, all else in 64 bits."""
        k, v = q8.dequantised(self.k, self.ks)[:, 0], q8.dequantised(self.v, self.vs)[:, 0]
        T, H, D = self.q.shape
        out = torch.zeros(T, H, D, dtype=torch.float64)
        for t in range(T):
            j = torch.arange(int(self.ctx[0]) + t + 1)
            pg, row = self.table[0].long()[j // self.page], j % self.page
            x = (self.q[t].double() @ k[pg, row].T) * self.scale
            w = torch.exp(x - x.amax(1, keepdim=True))
            out[t] = parts_of(w, parts) @ v[pg, row] / w.sum(1, keepdim=True)
        return out


CASES = [(1, 16, 128, 16), (2, 16, 128, 64), (4, 16, 128, 16), (1, 16, 64, 16), (3, 20, 64, 128)]


@pytest.mark.parametrize("tokens,H,D,page", CASES)
def test_the_bound_tells_two_parts_from_three(tokens, H, D, page):
    c = Case(tokens, H, D, page)
    out, tol = c.want()
    assert ((c.rounded_weights(3) - out).abs() <= tol).all()
    assert ((c.rounded_weights(2) - out).abs() > tol).any()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,H,D,page", CASES)
def test_weights_are_as_exact_as_stated(tokens, H, D, page):
    from aware_expert_routing_gb300 import build as b
    b.build()
    c = Case(tokens, H, D, page)
    cache = moe.KvCacheQ8(c.k.to(DEV).view(q8.F8), c.v.to(DEV).view(q8.F8), c.ks.to(DEV), c.vs.to(DEV), c.table.to(DEV))
    q = c.q.to(DEV)
    o = torch.empty_like(q)
    ws = moe.alloc_attention_workspace(tokens, H, cache, DEV)
    moe.moe_tree_attention_q8(q, c.off.to(DEV), c.ctx.to(DEV), None, cache, o, None, ws, scale=c.scale)
    assert moe.moe_device_status(ws) == 0
    out, tol = c.want()
    assert ((o.cpu().double() - out).abs() <= tol).all(), float(((o.cpu().double() - out).abs() / tol).max())


class Queries:
    def __init__(self, tokens, H, D):
        self.D, page, L, g = D, 16, 200 + tokens, torch.Generator().manual_seed(H + D)
        pages = (L + page - 1) // page
        self.table = torch.randperm(pages, generator=g).to(torch.int32)[None]
        k = torch.randint(-14, 15, (pages, 1, page, 1), generator=g).double().expand(-1, -1, -1, D).clone()
        k[..., 0] = 0
        self.k, self.ks = q8.encode(k), torch.full((pages, 1, page // 8), 2.0 ** -4)
        self.v, self.vs = q8.random_cache(pages, 1, page, D, 8, 5)
        self.scale = D ** -0.5
        # between the finest steps of the first number and of both
        size = 8192 * torch.exp2(-14 - 3 * torch.rand(tokens, H, generator=g))
        self.q = size[..., None].expand(-1, -1, D).to(torch.bfloat16).clone()
        self.q[0, 0] = 0
        self.q[0, 0, 0] = 8192.0
        self.off, self.ctx = torch.tensor([0, tokens], dtype=torch.int32), torch.tensor([200], dtype=torch.int32)

    def lse(self, q):
        """In 64 bits, with its bound."""
        k, v = q8.dequantised(self.k, self.ks), q8.dequantised(self.v, self.vs)
        _, e, _, tol = ref.attend(q, k, v, self.table, self.off, self.ctx, None, self.scale, True)
        return e, tol + 2.0 ** -21 * 8192 * float(k.abs().sum(-1).max()) * self.scale

    def rounded(self, parts):
        """The queries as the kernel takes them, or with the first number alone: the largest is 256 units."""
        x = self.q.double() / 32
        q0 = q8.decode(q8.encode(x))
        return 32 * (q0 if parts == 1 else q0 + q8.decode(q8.encode((x - q0) * 16)) / 16)


QUERIES = [(1, 16, 128), (2, 16, 64), (3, 10, 128)]


@pytest.mark.parametrize("tokens,H,D", QUERIES)
def test_the_bound_tells_one_number_from_two(tokens, H, D):
    c = Queries(tokens, H, D)
    e, tol = c.lse(c.q)
    assert ((c.lse(c.rounded(2))[0] - e).abs() <= tol).all()
    assert ((c.lse(c.rounded(1))[0] - e).abs() > tol).any()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,H,D", QUERIES)
def test_queries_are_as_exact_as_stated(tokens, H, D):
    from aware_expert_routing_gb300 import build as b
    b.build()
    c = Queries(tokens, H, D)
    cache = moe.KvCacheQ8(c.k.to(DEV).view(q8.F8), c.v.to(DEV).view(q8.F8), c.ks.to(DEV), c.vs.to(DEV), c.table.to(DEV))
    q = c.q.to(DEV)
    o, l = torch.empty_like(q), torch.empty(tokens, H, device=DEV)
    ws = moe.alloc_attention_workspace(tokens, H, cache, DEV)
    moe.moe_tree_attention_q8(q, c.off.to(DEV), c.ctx.to(DEV), None, cache, o, l, ws, scale=c.scale)
    assert moe.moe_device_status(ws) == 0
    e, tol = c.lse(c.q)
    assert ((l.cpu().double() - e).abs() <= tol).all(), float(((l.cpu().double() - e).abs() / tol).max())
