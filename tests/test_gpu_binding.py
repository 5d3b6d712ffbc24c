"""What the per-token calls make of unusual but valid (or invalid) tensors."""
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("aware_expert_routing_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from aware_expert_routing_gb300 import build as b
    b.build()
    moe.load()


def cache(dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(6, 2, 16, 64, generator=g, device=DEV).to(dtype) for _ in range(2))
    return moe.KvCache(k, v, torch.arange(6, dtype=torch.int32, device=DEV).reshape(2, 3))


def test_a_mask_without_words_is_refused():
    c = cache()
    q = torch.randn(3, 4, 64, device=DEV).to(torch.bfloat16)
    off, ctx = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 2, 3], [5, 9]))
    ws = moe.alloc_attention_workspace(3, 4, c, DEV)
    with pytest.raises(ValueError):
        moe.moe_tree_attention(q, off, ctx, torch.empty(3, 0, dtype=torch.int32, device=DEV), c, torch.empty_like(q), None, ws)
    # a call without tokens has a mask without words (tree_mask([]))
    none = q[:0].contiguous()
    moe.moe_tree_attention(none, torch.zeros_like(off), ctx, moe.tree_mask([]).to(DEV), c, torch.empty_like(none), None, ws)


def odd(shape, stride, values):
    """The values in a tensor with the given distances."""
    t = torch.zeros(4096, dtype=values.dtype, device=DEV).as_strided(shape, stride)
    t.copy_(values)
    return t


@pytest.mark.parametrize("T,H", [(1, 4), (1, 2), (3, 2)])
def test_the_distance_of_a_single_token_or_head_does_not_matter(T, H):
    """A dimension of size 1 may have any distance (slices of a wider row, expanded tensors)."""
    g = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn(T, h, 64, generator=g, device=DEV).to(torch.bfloat16) for h in (H, 2, 2))
    tok, head = (333 if T == 1 else 320), 64
    out = []
    for qq, kk, vv in ((q, k, v), (odd((T, H, 64), (tok, head, 1), q), odd((T, 2, 64), (tok, head, 1), k),
                                   odd((T, 2, 64), (tok, head, 1), v))):
        c = cache()
        ws = moe.alloc_attention_workspace(T, H, c, DEV)
        rope = moe.moe_rope_table(moe.RopeParams(rot=64), 32, DEV)
        pos = torch.arange(T, dtype=torch.int32, device=DEV)
        rot = torch.empty(T, H, 64, dtype=torch.bfloat16, device=DEV)
        moe.moe_kv_append(qq, kk, vv, rope, pos, 5 + pos.long(), c, rot, ws)
        o = torch.empty_like(rot)
        off, ctx = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, T, T], [5, 0]))
        moe.moe_tree_attention(qq, off, ctx, None, c, o, None, ws)
        assert moe.moe_device_status(ws) == 0
        out.append((rot, c.k, c.v, o))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    # one key head, its distance odd
    one = torch.randn(T, 1, 64, generator=g, device=DEV).to(torch.bfloat16)
    ck = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    w = odd((T, 1, 64), (320, 77, 1), one)
    moe.moe_kv_append(None, w, w, None, None, torch.arange(T, device=DEV), moe.KvCache(ck, ck.clone()), None, ws)
    assert moe.moe_device_status(ws) == 0 and torch.equal(ck[0, 0, :T], one[:, 0])


@pytest.mark.parametrize("kw", [dict(B=4), dict(N=32), dict(k=2)])
def test_a_routing_of_another_size_is_refused(kw):
    prm = moe.RouteParams(**{**dict(B=8, d=256, N=64, k=4), **kw})
    small = moe.Routing(prm, DEV)
    prm = moe.RouteParams(B=8, d=256, N=64, k=4)
    ws = moe.alloc_workspace(prm, 0, DEV)
    x = torch.randn(8, 64, device=DEV)
    with pytest.raises(ValueError):
        moe.moe_route_scores(x, None, prm, moe.SelectParams(), small, ws)
    good = moe.Routing(prm, DEV)
    moe.moe_route_scores(x, None, prm, moe.SelectParams(), good, ws)      # and one of this size serves, or a larger one
    want = good.expert_idx.clone()
    large = moe.Routing(moe.RouteParams(B=16, d=256, N=64, k=4), DEV)
    moe.moe_route_scores(x, None, prm, moe.SelectParams(), large, ws)
    assert torch.equal(large.expert_idx[:8], want)
    for name in ("counts", "weights"):
        bad = moe.Routing(prm, DEV)
        setattr(bad, name, getattr(bad, name).double())
        with pytest.raises(ValueError):
            moe.moe_route_scores(x, None, prm, moe.SelectParams(), bad, ws)
    bad = moe.Routing(prm, DEV)
    bad.perm = None
    with pytest.raises(ValueError):
        moe.moe_route_scores(x, None, prm, moe.SelectParams(), bad, ws)
