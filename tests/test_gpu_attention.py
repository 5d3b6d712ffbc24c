"""moe_tree_attention against a plain 64-bit statement."""
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


def trees(n, seed, words=None):
    """Mask words of random trees of n[r] tokens (tests' own walk)."""
    g = torch.Generator().manual_seed(seed)
    W = words or max(1, (max(n) + 31) // 32)
    rows = []
    for nr in n:
        par = [-1 if i == 0 else int(torch.randint(max(0, i - 5), i, (1,), generator=g)) for i in range(nr)]
        for i in range(nr):
            bits, at = 0, i
            while at >= 0:
                bits |= 1 << at
                at = par[at]
            rows.append([(bits >> (32 * w)) & 0xffffffff for w in range(W)])
    return torch.tensor(rows, dtype=torch.int64).reshape(len(rows), W).to(torch.int32)


class Case:
    def __init__(self, ctx, n, H, K, D, page, dtype, tree, seed, q_scale=2.0, extra_pages=2):
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.n = torch.tensor(ctx, dtype=torch.int32), n
        self.off = torch.tensor([0] + list(n)).cumsum(0).to(torch.int32)
        T = int(self.off[-1])
        per = [(c + m + page - 1) // page for c, m in zip(ctx, n)]
        total = sum(per) + extra_pages
        order = torch.randperm(total, generator=g).to(torch.int32)
        self.table = torch.zeros(len(ctx), max(max(per), 1), dtype=torch.int32)
        at = 0
        for r, p in enumerate(per):
            self.table[r, :p] = order[at:at + p]
            at += p
        self.k = torch.randn(total, K, page, D, generator=g).to(self.dt)
        self.v = (torch.randn(total, K, page, D, generator=g) + 0.25).to(self.dt)
        self.q = (torch.randn(T, H, D, generator=g) * q_scale).to(self.dt)
        self.mask = trees(n, seed + 1) if tree else None
        self.scale = D ** -0.5

    def run(self, q=None, ws=None, stream=None, lse=True):
        cache = moe.KvCache(self.k.to(DEV), self.v.to(DEV), self.table.to(DEV))
        q = self.q.to(DEV) if q is None else q
        T, H, D = q.shape
        out = torch.full((T, H, D), float("nan"), dtype=self.dt, device=DEV)
        l = torch.full((T, H), float("nan"), dtype=torch.float32, device=DEV) if lse else None
        if ws is None:
            ws = moe.alloc_attention_workspace(T, H, cache, DEV)
        mask = self.mask.to(DEV) if self.mask is not None else None
        moe.moe_tree_attention(q, self.off.to(DEV), self.ctx.to(DEV), mask, cache, out, l, ws, scale=self.scale,
                               stream=stream)
        return out, l, moe.moe_device_status(ws, stream)

    def check(self, out, l):
        o, e, to, te = ref.attend(self.q, self.k, self.v, self.table, self.off, self.ctx, self.mask, self.scale,
                                  self.dt == torch.bfloat16)
        out, l = out.cpu().double(), l.cpu().double()
        assert ((out - o).abs() <= to).all(), float(((out - o).abs() - to).max())
        dead = e == -math.inf
        assert (l[dead] == -math.inf).all() and (out[dead] == 0).all()
        assert ((l - e).abs()[~dead] <= te[~dead]).all(), float(((l - e).abs() - te)[~dead].max())


BF16 = [
    # ctx, drafted tokens, heads, key heads, D, page, tree
    ([0], [1], 1, 1, 128, 16, False), ([1], [1], 8, 1, 128, 16, False), ([127], [1], 8, 1, 128, 16, False),
    ([128], [1], 8, 2, 128, 16, False), ([1000], [1], 32, 4, 128, 16, False), ([5, 300, 0, 129], [1, 1, 1, 1], 16, 2, 128, 32, False),
    ([400, 17], [16, 9], 32, 4, 128, 16, True), ([250], [64], 16, 2, 128, 64, True), ([100], [40], 8, 8, 128, 16, True),
    ([60, 700, 0], [3, 0, 7], 10, 2, 128, 8, True), ([2100], [5], 64, 4, 128, 128, False), ([333], [33], 5, 1, 128, 256, True),
    ([90, 130], [130, 3], 4, 2, 128, 16, False), ([513, 3], [1, 20], 16, 1, 128, 1024, True), ([0, 0], [64, 1], 8, 2, 128, 16, True),
    ([200, 55], [4, 4], 8, 2, 64, 16, True), ([1500], [1], 16, 2, 64, 32, False), ([31], [70], 20, 4, 64, 8, True),
    # head sizes and pages that no tile is made for
    ([77, 140], [3, 2], 6, 3, 80, 16, True), ([200], [5], 4, 1, 256, 16, False), ([90], [2], 2, 2, 8, 16, True),
    ([150, 30], [6, 1], 8, 2, 128, 24, True), ([40], [3], 8, 2, 128, 1, False), ([300], [2], 8, 2, 128, 4, True),
    ([4000] + [10] * 30, [1] * 31, 8, 1, 128, 16, False),
]
F32 = [
    ([0], [1], 2, 1, 64, 16, False), ([300, 11], [7, 2], 8, 2, 64, 16, False), ([129], [20], 16, 2, 128, 16, True),
    ([1000], [1], 32, 4, 128, 16, False), ([50, 0, 260], [1, 64, 3], 10, 2, 40, 7, True), ([90], [9], 3, 3, 256, 32, True),
    ([2500], [3], 8, 1, 128, 64, False), ([70], [130], 4, 2, 64, 16, False),
]


@pytest.mark.parametrize("ctx,n,H,K,D,page,tree", BF16)
def test_bf16(ctx, n, H, K, D, page, tree):
    c = Case(ctx, n, H, K, D, page, "bf16", tree, 17 + len(ctx) + H)
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)


@pytest.mark.parametrize("ctx,n,H,K,D,page,tree", F32)
def test_f32(ctx, n, H, K, D, page, tree):
    c = Case(ctx, n, H, K, D, page, "f32", tree, 29 + len(ctx) + H)
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_that_leave_rows_empty(dtype):
    """No context and no bit: zeros and -inf.  No bit but a context: the context alone.  Words that do not reach
    every token: the rest is not seen."""
    c = Case([0, 20, 0, 200], [4, 3, 40, 40], 8, 2, 64, 16, dtype, True, 3)
    c.mask = c.mask.clone()
    c.mask[0] = 0
    c.mask[2] = 0
    c.mask[4:7] = 0
    c.mask[10:40, :] = 0
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)
    c.mask = c.mask[:, :1].contiguous()
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)


@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 16), ("bf16", 64, 64), ("bf16", 80, 16), ("f32", 64, 16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_unseen_positions_have_no_influence(dtype, D, page, bad):
    """Rows of a request's last page past its length, pages of nobody, and drafted tokens that no one sees hold
    anything."""
    c = Case([100, 0, 127], [5, 3, 1], 8, 2, D, page, dtype, True, 5)
    c.mask[:, 0] &= ~4              # the third drafted token is seen by nobody, itself included
    o, e, to, te = ref.attend(c.q, c.k, c.v, c.table, c.off, c.ctx, c.mask, c.scale, dtype == "bf16")
    seen = torch.zeros(c.k.shape[0], page, dtype=torch.bool)
    for r, (ctx, n) in enumerate(zip([100, 0, 127], [5, 3, 1])):
        for j in range(ctx + n):
            if j != ctx + 2:
                seen[c.table[r, j // page].long(), j % page] = True
    c.k.permute(0, 2, 1, 3)[~seen] = bad
    c.v.permute(0, 2, 1, 3)[~seen] = bad
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_siblings_nan_stays_with_those_who_see_it(dtype):
    """A drafted token whose key or value is NaN spoils the tokens that see it and no others."""
    for what in ("k", "v"):
        c = Case([50], [6], 8, 2, 128, 16, dtype, True, 6)
        c.mask[:, 0] = torch.tensor([1, 3, 5, 7, 17, 33], dtype=torch.int32)
        j = 52                                   # drafted token 2: seen by tokens 2 and 3
        x = getattr(c, what)
        x[c.table[0, j // 16].long(), :, j % 16, 5] = float("nan")
        out, l, flags = c.run()
        assert flags == 0
        spoilt = out.cpu().isnan().flatten(1).any(1)
        assert spoilt.tolist() == [False, False, True, True, False, False]
        x.nan_to_num_(0.0)
        o, e, to, te = ref.attend(c.q, c.k, c.v, c.table, c.off, c.ctx, c.mask, c.scale, dtype == "bf16")
        ok = ~spoilt
        assert ((out.cpu().double() - o).abs() <= to)[ok].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rising", "falling", "one far above", "very negative"])
def test_running_maximum(dtype, kind):
    """Scores that rise, fall or jump along the context: the running maximum's corrections."""
    c = Case([900], [2], 8, 2, 128, 16, dtype, False, 8, q_scale=0.0)
    c.q[..., 0] = 11.3
    j = torch.arange(902)
    s = {"rising": j * 0.11, "falling": -j * 0.11, "one far above": (j == 701) * 60.0, "very negative": -300.0 - j * 0.05}[kind]
    k = c.k.float()
    k[c.table[0].long()[j // 16], :, j % 16, 0] = s.float()[:, None]
    c.k = k.to(c.dt)
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)


def test_strided_queries_and_null_lse():
    c = Case([70, 3], [5, 2], 8, 2, 64, 16, "bf16", True, 11)
    want, l, _ = c.run()
    T = c.q.shape[0]
    wide = torch.zeros(T, 12, 64, dtype=torch.bfloat16, device=DEV)
    wide[:, 2:10] = c.q.to(DEV)
    got, _, _ = c.run(q=wide[:, 2:10], lse=False)
    assert torch.equal(got, want)
    first = c.q.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    got, l2, _ = c.run(q=first)
    assert torch.equal(got, want) and torch.equal(l, l2)
    c.check(got, l2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_again_on_another_stream_and_in_a_graph(dtype):
    c = Case([900, 40, 3000], [9, 1, 20], 16, 2, 128, 16, dtype, True, 12)
    want, l, flags = c.run()
    assert flags == 0
    ws = moe.alloc_attention_workspace(30, 16, moe.KvCache(c.k.to(DEV), c.v.to(DEV), c.table.to(DEV)), DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got, l2, flags = c.run(ws=ws, stream=s)
        assert flags == 0 and torch.equal(got, want) and torch.equal(l, l2)
    cache = moe.KvCache(c.k.to(DEV), c.v.to(DEV), c.table.to(DEV))
    q, off, ctx, mask = c.q.to(DEV), c.off.to(DEV), c.ctx.to(DEV), c.mask.to(DEV)
    out, l3 = torch.zeros_like(q), torch.zeros(30, 16, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_tree_attention(q, off, ctx, mask, cache, out, l3, ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(l3, l)
    # the lengths are read on the device: a captured call follows them
    ctx.copy_(torch.tensor([899, 0, 1234], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    c.ctx = ctx.cpu()
    c.check(out, l3)


@pytest.mark.parametrize("ctx,n", [([2000, 3500], [20, 30]), ([900, 40, 3000], [9, 1, 20]), ([1500], [3])])
def test_row_tiles_that_are_not_full_give_the_same_bits(ctx, n):
    """Rows of a tile past the unit's own hold what earlier calls left there; it must not show in the others."""
    c = Case(ctx, n, 16, 2, 128, 16, "bf16", True, 31)
    other = Case([700, 300], [50, 61], 16, 2, 128, 16, "bf16", True, 32, q_scale=30.0)
    want, l, flags = c.run()
    assert flags == 0
    c.check(want, l)
    for _ in range(20):
        other.run()
        got, l2, flags = c.run()
        assert flags == 0 and torch.equal(got, want) and torch.equal(l, l2)


def test_tokens_past_the_last_request_are_not_written():
    c = Case([30, 8], [2, 3], 8, 2, 64, 16, "bf16", False, 13)
    want, l, _ = c.run()
    q = torch.cat([c.q, c.q[:3]]).to(DEV)
    got, l2, flags = c.run(q=q)
    assert flags == 0
    assert torch.equal(got[:5], want) and got[5:].isnan().all() and l2[5:].isnan().all()


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("bf16", 12), ("f32", 16)])
def test_bad_tables_and_lengths_raise_the_flag_and_spare_the_others(dtype, page):
    for bad in ("page", "negative page", "length", "negative length"):
        c = Case([300, 100, 40], [2, 3, 1], 8, 2, 128, page, dtype, True, 14)
        want, l, flags = c.run()
        assert flags == 0
        if bad == "page":
            c.table[1, 2] = c.k.shape[0]
        elif bad == "negative page":
            c.table[1, 0] = -1
        elif bad == "length":
            c.ctx[1] = c.table.shape[1] * page - 2
        else:
            c.ctx[1] = -1
        got, l2, flags = c.run()
        assert flags == moe.FLAG_BAD_INDEX, bad
        for part in (slice(0, 2), slice(5, 6)):
            assert torch.equal(got[part], want[part]) and torch.equal(l2[part], l[part]), bad


def test_bad_offsets_raise_the_flag():
    c = Case([30, 8, 5], [2, 3, 1], 8, 2, 64, 16, "bf16", False, 15)
    want, _, _ = c.run()
    c.off = torch.tensor([0, 2, 5, 99], dtype=torch.int32)     # past T
    got, _, flags = c.run()
    assert flags == moe.FLAG_BAD_INDEX
    assert torch.equal(got[:5], want[:5])


def test_nothing_to_do():
    cache = moe.KvCache(torch.zeros(1, 1, 16, 64, device=DEV), torch.zeros(1, 1, 16, 64, device=DEV),
                        torch.zeros(2, 1, dtype=torch.int32, device=DEV))
    ws = moe.alloc_attention_workspace(0, 2, cache, DEV)
    q = torch.zeros(0, 2, 64, device=DEV)
    z = torch.zeros(3, dtype=torch.int32, device=DEV)
    moe.moe_tree_attention(q, z, z[:2], None, cache, torch.empty_like(q), None, ws)
    q = torch.zeros(2, 2, 64, device=DEV)
    out = torch.full_like(q, 7.0)
    ws = moe.alloc_attention_workspace(2, 2, cache, DEV)
    moe.moe_tree_attention(q, z, z[:2], None, cache, out, None, ws)    # every request has no token
    assert moe.moe_device_status(ws) == 0 and (out == 7).all()


def test_cache_past_2_31_elements():
    K, page, D = 4, 64, 128
    pages = (1 << 31) // (K * page * D) + 40
    ck, cv = (torch.empty(pages, K, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c = Case([150], [3], 16, K, D, page, "bf16", True, 16, extra_pages=0)
    far = torch.tensor([pages - 1, 5, pages - 3])
    for x, y in ((ck, c.k), (cv, c.v)):
        x[far.to(DEV)] = y[c.table[0].long()].to(DEV)
    table = far[None].to(torch.int32).to(DEV)
    cache = moe.KvCache(ck, cv, table)
    out, l = torch.empty(3, 16, D, dtype=torch.bfloat16, device=DEV), torch.empty(3, 16, device=DEV)
    ws = moe.alloc_attention_workspace(3, 16, cache, DEV)
    moe.moe_tree_attention(c.q.to(DEV), c.off.to(DEV), c.ctx.to(DEV), c.mask.to(DEV), cache, out, l, ws)
    assert moe.moe_device_status(ws) == 0
    c.check(out, l)


def test_long_context_many_splits():
    """One request's long context is worked on by many blocks whose sums are joined."""
    c = Case([20000], [3], 8, 1, 128, 64, "bf16", True, 18)
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)
    a = Case([9999], [1], 8, 1, 128, 64, "f32", False, 19)
    whole, lw, _ = a.run()
    a.check(whole, lw)


@pytest.mark.parametrize("R,most,n,H,K,D,page,dtype", [
    (90, 3500, 1, 32, 4, 128, 16, "bf16"), (40, 2500, 9, 32, 4, 128, 16, "bf16"), (25, 2000, 40, 16, 2, 128, 64, "bf16"),
    (200, 150, 2, 16, 4, 128, 16, "bf16"), (70, 3000, 2, 32, 4, 64, 32, "bf16"), (30, 1500, 33, 32, 4, 64, 8, "bf16"),
    (300, 60, 1, 8, 8, 128, 128, "bf16"), (60, 900, 3, 8, 2, 64, 16, "f32")])
def test_many_requests(R, most, n, H, K, D, page, dtype):
    """More units than blocks: a block goes through several units and parts of units, all with the same bits again."""
    g = torch.Generator().manual_seed(R)
    ctx = torch.randint(0, most + 1, (R,), generator=g).tolist()
    ns = torch.randint(0 if n > 1 else 1, n + 1, (R,), generator=g).tolist()
    c = Case(ctx, ns, H, K, D, page, dtype, n > 1, R + 1)
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)
    for _ in range(5):
        out2, l2, _ = c.run()
        assert torch.equal(out, out2) and torch.equal(l, l2)


# The same questions at other numbers of rows a key head: few rows share out a tile's keys, many share its copies.
@pytest.mark.parametrize("H", [4, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_unseen_positions_have_no_influence_at_any_number_of_rows(H, D, bad):
    ctx, n = [300, 0, 127], [5, 3, 1]
    c = Case(ctx, n, H, 2, D, 16, "bf16", True, 41)
    c.mask[:, 0] &= ~4
    seen = torch.zeros(c.k.shape[0], 16, dtype=torch.bool)
    for r in range(3):
        for j in range(ctx[r] + n[r]):
            if j != ctx[r] + 2:
                seen[c.table[r, j // 16].long(), j % 16] = True
    c.k.permute(0, 2, 1, 3)[~seen] = bad
    c.v.permute(0, 2, 1, 3)[~seen] = bad
    out, l, flags = c.run()
    assert flags == 0
    c.k.permute(0, 2, 1, 3)[~seen] = 0.0
    c.v.permute(0, 2, 1, 3)[~seen] = 0.0
    c.check(out, l)


@pytest.mark.parametrize("H", [4, 32, 64])
@pytest.mark.parametrize("what", ["k", "v"])
def test_a_siblings_nan_at_any_number_of_rows(H, what):
    c = Case([150], [6], H, 2, 128, 16, "bf16", True, 42)
    c.mask[:, 0] = torch.tensor([1, 3, 5, 7, 17, 33], dtype=torch.int32)
    x = getattr(c, what)
    x[c.table[0, 152 // 16].long(), :, 152 % 16, 5] = float("nan")
    out, l, flags = c.run()
    assert flags == 0
    spoilt = out.cpu().isnan().flatten(1).any(1)
    assert spoilt.tolist() == [False, False, True, True, False, False]
    x.nan_to_num_(0.0)
    o, e, to, te = ref.attend(c.q, c.k, c.v, c.table, c.off, c.ctx, c.mask, c.scale, True)
    assert ((out.cpu().double() - o).abs() <= to)[~spoilt].all()


@pytest.mark.parametrize("H", [4, 32, 64, 160])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["rising", "falling", "one far above", "very negative"])
def test_running_maximum_at_any_number_of_rows(H, D, kind):
    c = Case([900], [2], H, 2, D, 16, "bf16", False, 43, q_scale=0.0)
    c.q[..., 0] = 11.3 * (D / 128) ** 0.5
    j = torch.arange(902)
    s = {"rising": j * 0.11, "falling": -j * 0.11, "one far above": (j == 701) * 60.0, "very negative": -300.0 - j * 0.05}[kind]
    k = c.k.float()
    k[c.table[0].long()[j // 16], :, j % 16, 0] = s.float()[:, None]
    c.k = k.to(c.dt)
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("singles,many", [(29, 13), (19, 13), (3, 40), (1, 70)])
def test_many_tokens_of_one_request_among_single_ones(singles, many, D):
    """The units' height follows the mean: the request with many tokens has several units, or all fill a part of one."""
    g = torch.Generator().manual_seed(44)
    ctx = torch.randint(0, 700, (singles + 1,), generator=g).tolist()
    n = [1] * singles + [many]
    c = Case(ctx, n, 16, 2, D, 16, "bf16", True, 45)
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)
    again, l2, _ = c.run()
    assert torch.equal(again, out) and torch.equal(l2, l)


@pytest.mark.parametrize("ctx,n,H", [(500, 1, 2), (1000, 1, 2), (3000, 1, 32), (3000, 2, 40), (700, 3, 32)])
@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_lose_nothing_but_the_results_rounding(ctx, n, H, D):
    """With few rows a key head (up to 48 on average) a weight enters the product as two bf16 numbers, good to 2^-16 of
    it, against 2^-9 of the result's own rounding: the error is the rounding's, within a hundredth (2^-16 / 2^-9 = 1/128)."""
    for seed in range(5):
        c = Case([ctx], [n], H, 2, D, 16, "bf16", False, 50 + seed)
        out, _, flags = c.run()
        assert flags == 0
        o = ref.attend(c.q, c.k, c.v, c.table, c.off, c.ctx, c.mask, c.scale, True)[0]
        assert (out.cpu().double() - o).norm() <= 1.01 * (o.bfloat16().double() - o).norm()
