"""Edges of the grouped selection: padding tokens whose scores hold anything,
and which values rank a softmax when every group stays."""
import numpy as np
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


@pytest.mark.parametrize("B", [1, 11, 12, 40])
@pytest.mark.parametrize("groups", [1, 4])
def test_scores_of_padding_tokens_are_not_looked_at(B, groups):
    valid = B // 2
    prm = moe.RouteParams(B=B, B_valid=valid, d=256, N=64, k=4)
    sel = moe.SelectParams(score=moe.SCORE_SIGMOID, n_group=groups, topk_group=max(1, groups // 2), group_top=2)
    x = torch.randn(B, 64, generator=torch.Generator().manual_seed(B))
    x[valid:] = float("nan")
    r, ws = moe.Routing(prm, DEV), moe.alloc_workspace(prm, 0, DEV)
    moe.moe_route_scores(x.to(DEV), None, prm, sel, r, ws)
    assert moe.moe_device_status(ws) == 0
    idx, _ = ref.select(x.numpy(), None, 4, True, sel.n_group, sel.topk_group, 2, True, 1.0, valid)
    assert np.array_equal(r.expert_idx.cpu().numpy(), idx)


@pytest.mark.parametrize("B", [8, 24, 64])
def test_hidden_states_of_padding_tokens_are_not_looked_at(B):
    valid = B - 3
    prm = moe.RouteParams(B=B, B_valid=valid, d=256, N=64, k=4)
    sel = moe.SelectParams(score=moe.SCORE_SIGMOID, n_group=4, topk_group=2, group_top=2)
    g = torch.Generator().manual_seed(B)
    x = torch.randn(B, 256, generator=g).to(torch.bfloat16)
    x[valid:] = float("nan")
    w = (torch.randn(64, 256, generator=g) / 16).to(torch.bfloat16)
    r, ws = moe.Routing(prm, DEV, with_logits=True), moe.alloc_workspace(prm, 0, DEV)
    moe.moe_route_grouped(x.to(DEV), w.to(DEV), None, None, prm, sel, r, ws)
    assert moe.moe_device_status(ws) == 0
    assert (r.expert_idx[valid:] == -1).all() and (r.expert_idx[:valid] >= 0).all()
    assert (r.n_base.cpu() == torch.tensor([4] * valid + [0] * 3)).all()


@pytest.mark.parametrize("B", [2, 30])
@pytest.mark.parametrize("groups", [1, 4])
def test_a_softmax_with_sums_of_two_is_ranked_by_its_values(B, groups):
    """group_top 2: experts whose softmax underflows to the same value go by the lower id, also where every group
    stays; with group_top 1 the scores themselves rank them."""
    N, k = 8, 3
    x = torch.full((B, N), -400.0)
    x[:, 0], x[:, 5], x[:, 7] = 0.0, -150.0, -200.0
    prm = moe.RouteParams(B=B, d=256, N=N, k=k)
    ws = moe.alloc_workspace(prm, 0, DEV)
    for top, want in ((2, [0, 1, 2]), (1, [0, 5, 7])):
        r = moe.Routing(prm, DEV)
        moe.moe_route_scores(x.to(DEV), None, prm, moe.SelectParams(n_group=groups, topk_group=groups, group_top=top), r, ws)
        assert moe.moe_device_status(ws) == 0
        assert r.expert_idx.cpu().tolist() == [want] * B, top
        assert r.weights.cpu().tolist() == [[1.0, 0.0, 0.0]] * B
