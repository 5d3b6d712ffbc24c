"""moe_route_scores, moe_route_grouped and moe_decode_layer_grouped: the
selection by softmax or sigmoid scores with a bias and expert groups, against
a plain 64-bit statement, and the expert layer that follows it."""
import numpy as np
import pytest
import torch

import attention_ref as ref
import synth

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("aware_expert_routing_gb300")
import gpu_util as gu  # noqa: E402
import oracle  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from aware_expert_routing_gb300 import build as b
    b.build()
    moe.load()


def run(scores, bias, prm, sel, ws=None, stream=None):
    r = moe.Routing(prm, gu.DEV)
    if ws is None:
        ws = moe.alloc_workspace(prm, 0, gu.DEV)
    moe.moe_route_scores(scores, bias, prm, sel, r, ws, stream)
    return r, moe.moe_device_status(ws, stream)


def check(r, scores, bias, prm, sel, B_valid=None):
    """Whole numbers equal; weights: p to a few roundings of fp32, its sum over k of them, and the quotient."""
    idx, w = ref.select(scores, bias, prm.k, sel.score == moe.SCORE_SIGMOID, sel.n_group, sel.topk_group, sel.group_top,
                        sel.renormalise, sel.scale, B_valid)
    g = {n: getattr(r, n).cpu().numpy() for n in ("expert_idx", "weights", "T", "active", "counts", "offsets", "perm", "n_base")}
    assert np.array_equal(g["expert_idx"], idx)
    # relative: expf 2 ulp, the sums over N or k terms, the quotients; absolute: subnormal scores
    assert (np.abs(g["weights"] - w) <= (prm.N + prm.k + 16) * ref.U32 * np.abs(w) + 1e-37).all()
    T, active, counts, offsets, perm = ref.grouping(idx, prm.N)
    assert g["T"][0] == T and np.array_equal(g["active"], active) and np.array_equal(g["counts"], counts)
    assert np.array_equal(g["offsets"], offsets) and np.array_equal(g["perm"][:len(perm)], perm)
    assert np.array_equal(g["n_base"][:prm.B], (idx >= 0).sum(1))


def grid_scores(B, N, seed, step=0.125):
    """Scores on a grid: equal ones are frequent, unlike ones are far apart."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, N, generator=g) * 1.5 / step).round() * step


# B, N, k, sigmoid, bias, n_group, topk_group, group_top, renorm, scale
CASES = [
    (1, 1, 1, 0, 0, 1, 1, 1, 1, 1.0), (1, 128, 8, 0, 0, 1, 1, 1, 1, 1.0), (16, 128, 8, 0, 0, 1, 1, 1, 0, 2.0),
    (33, 64, 6, 0, 0, 8, 3, 1, 0, 16.0), (40, 160, 6, 0, 0, 8, 3, 1, 1, 1.0), (256, 256, 8, 1, 1, 8, 4, 2, 1, 2.5),
    (1, 256, 8, 1, 1, 8, 4, 2, 1, 2.5), (7, 60, 5, 1, 1, 4, 2, 2, 0, 1.0), (64, 48, 4, 1, 0, 1, 1, 1, 1, 1.0),
    (100, 384, 8, 1, 1, 1, 1, 1, 1, 2.827), (17, 1024, 32, 1, 1, 32, 9, 2, 1, 1.0), (5, 1024, 9, 0, 1, 16, 16, 2, 1, 1.0),
    (20, 33, 3, 1, 1, 11, 4, 2, 1, 1.0), (20, 32, 2, 1, 0, 32, 3, 1, 1, 1.0), (9, 14, 7, 1, 1, 2, 1, 2, 0, 0.5),
    (13, 96, 8, 0, 1, 1, 1, 1, 1, 1.0), (250, 72, 3, 1, 1, 3, 2, 1, 1, -1.5),
]


@pytest.mark.parametrize("B,N,k,sig,has_bias,G,tg,gt,renorm,scale", CASES)
def test_selection(B, N, k, sig, has_bias, G, tg, gt, renorm, scale):
    x = grid_scores(B, N, 100 + B + N)
    # biases on a grid too, with a part that no sum of scores hits
    bias = (torch.randn(N, generator=torch.Generator().manual_seed(N)) * 8).round() / 64 if has_bias else None
    prm = moe.RouteParams(B=B, d=256, N=N, k=k)
    sel = moe.SelectParams(score=sig, n_group=G, topk_group=tg, group_top=gt, renormalise=bool(renorm), scale=scale)
    r, flags = run(x.to(gu.DEV), bias.to(gu.DEV) if has_bias else None, prm, sel)
    assert flags == 0
    check(r, x.numpy(), None if bias is None else bias.numpy(), prm, sel)


def test_all_scores_equal_take_the_lowest_groups_and_experts():
    prm = moe.RouteParams(B=5, d=256, N=96, k=8)
    for sig in (0, 1):
        sel = moe.SelectParams(score=sig, n_group=8, topk_group=3, group_top=2 - (1 - sig))
        r, flags = run(torch.full((5, 96), 0.75, device=gu.DEV), None, prm, sel)
        assert flags == 0
        assert (r.expert_idx.cpu() == torch.arange(8, dtype=torch.int32)).all()
        assert (r.weights - 1 / 8).abs().max() <= 8 * ref.U32


def test_extreme_scores():
    """Scores at which exp overflows or a sigmoid is 0 or 1; a sum of chosen scores that is 0."""
    N = 64
    x = torch.zeros(4, N)
    x[0] = torch.linspace(-200, 200, N)
    x[1] = -1e30
    x[2] = torch.linspace(3e38, -3e38, N, dtype=torch.float64).float()
    x[3] = torch.linspace(-110, -90, N)
    prm = moe.RouteParams(B=4, d=256, N=N, k=4)
    sel = moe.SelectParams(score=moe.SCORE_SIGMOID, n_group=4, topk_group=2, group_top=2)
    r, flags = run(x.to(gu.DEV), None, prm, sel)
    assert flags == 0
    w = r.weights.cpu()
    assert w.isfinite().all() and (w[1] == 0).all()
    # row 0 has more than 4 scores whose sigmoid is 1 in fp32: the lowest ids of the best groups
    assert r.expert_idx.cpu()[1].tolist() == [0, 1, 2, 3] and r.expert_idx.cpu()[2].tolist() == [0, 1, 2, 3]
    sel = moe.SelectParams(score=moe.SCORE_SOFTMAX)
    r, flags = run(x.to(gu.DEV), None, prm, sel)
    assert flags == 0
    idx, w = ref.select(x.numpy(), None, 4, False, 1, 1, 1, True, 1.0)
    assert np.array_equal(r.expert_idx.cpu().numpy(), idx)
    assert np.abs(r.weights.cpu().numpy() - w).max() <= 1e-5


def test_non_finite_scores_and_biases_are_never_chosen():
    N = 64
    x = grid_scores(3, N, 5)
    x[0, 3], x[0, 7], x[1, :60] = float("nan"), float("inf"), -float("inf")
    bias = torch.zeros(N)
    bias[10], bias[11], bias[63] = -float("inf"), float("nan"), float("inf")
    prm = moe.RouteParams(B=3, d=256, N=N, k=6)
    for sig, G, tg in ((1, 1, 1), (1, 8, 3), (0, 1, 1)):
        sel = moe.SelectParams(score=sig, n_group=G, topk_group=tg, group_top=2 if sig and G > 1 else 1)
        r, flags = run(x.to(gu.DEV), bias.to(gu.DEV), prm, sel)
        assert flags == moe.FLAG_NONFINITE_SCORE
        check(r, x.numpy(), bias.numpy(), prm, sel)
    assert (r.expert_idx[1] >= 0).sum() == 3


def test_padding_and_empty_batches():
    x = grid_scores(40, 64, 6)
    sel = moe.SelectParams(score=moe.SCORE_SIGMOID, n_group=4, topk_group=2, group_top=2)
    for bv in (0, 1, 33, 40):
        prm = moe.RouteParams(B=40, B_valid=bv, d=256, N=64, k=4)
        r, flags = run(x.to(gu.DEV), None, prm, sel)
        assert flags == 0
        check(r, x.numpy(), None, prm, sel, bv)
    prm = moe.RouteParams(B=0, d=256, N=64, k=4)
    r, flags = run(torch.empty(0, 64, device=gu.DEV), None, prm, sel)
    assert flags == 0 and int(r.T.item()) == 0 and (r.counts == 0).all() and (r.active == -1).all()


def test_softmax_without_groups_is_the_plain_router():
    """Same experts and weights as moe_route's top-k on the same scores."""
    w = synth.Workload("t_sel", N=128, k=8, d=256, F=128, B=24, seed=3, zipf=True)
    D = gu.device_inputs(synth.make_layer(w, 0, 24), True)
    prm = gu.params_for(w, 24, 0)
    r0 = moe.Routing(prm, gu.DEV, with_logits=True)
    ws = moe.alloc_workspace(prm, w.F, gu.DEV)
    moe.moe_route(D["x"], D["w_router"], D["bias"], prm, r0, ws)
    r1, flags = run(r0.logits, None, prm, moe.SelectParams(), ws)
    assert flags == 0
    for n in ("expert_idx", "T", "active", "counts", "offsets", "perm"):
        assert torch.equal(getattr(r0, n), getattr(r1, n)), n
    assert (r0.weights - r1.weights).abs().max() <= 1e-6


@pytest.mark.parametrize("B,N,bf16", [(1, 64, True), (24, 128, True), (48, 128, True), (200, 256, True), (16, 64, False)])
def test_layer(B, N, bf16):
    """Router, grouped selection, experts and combine in one call, and the same from moe_route_scores and
    moe_expert_ffn; outputs against the oracle."""
    w = synth.Workload("t_sel_layer", N=N, k=6, d=256, F=128, B=B, seed=41, zipf=True, bf16=bf16)
    L = synth.make_layer(w, 0, B)
    D = gu.device_inputs(L, bf16)
    prm = gu.params_for(w, B, 0)
    sel = moe.SelectParams(score=moe.SCORE_SIGMOID, n_group=8, topk_group=4, group_top=2, scale=1.5)
    g = torch.Generator().manual_seed(2)
    bias = (torch.randn(N, generator=g) * 0.1).to(gu.DEV)
    r = moe.Routing(prm, gu.DEV, with_logits=True)
    ws = moe.alloc_workspace(prm, w.F, gu.DEV)
    out = torch.full((B, w.d), float("nan"), dtype=prm.torch_dtype, device=gu.DEV)
    args = (D["w_gate"], D["w_up"], D["w_down"], w.F)
    for _ in range(2):
        moe.moe_decode_layer_grouped(D["x"], D["w_router"], D["bias"], bias, *args, prm, sel, r, out, ws)
    assert moe.moe_device_status(ws) == 0
    check(r, r.logits.cpu().numpy(), bias.cpu().numpy(), prm, sel)
    o_ref = oracle.moe_experts(L["x"], L["w_gate"], L["w_up"], L["w_down"], r.expert_idx.cpu().numpy(),
                               r.weights.cpu().numpy().astype(np.float64))
    gu.check_output(out, o_ref, bf16)
    r2 = moe.Routing(prm, gu.DEV)
    out2 = torch.empty_like(out)
    moe.moe_route_scores(r.logits, bias, prm, sel, r2, ws)
    moe.moe_expert_ffn(D["x"], *args, prm, r2, out2, ws)
    assert moe.moe_device_status(ws) == 0
    assert torch.equal(out, out2)
    # an OEA layer on the same workspace afterwards is not disturbed
    if bf16:
        po = gu.params_for(w, B, 1, 3, 1.0)
        if moe.moe_workspace_bytes(po, w.F) <= ws.numel():
            ro, oo, _, flags = gu.run_layer(w, D, po, ws)
            assert flags == 0
            rf, of, _, _ = gu.run_layer(w, D, po)
            assert torch.equal(ro.expert_idx, rf.expert_idx) and torch.equal(oo, of)


def test_another_stream_and_a_graph():
    x = grid_scores(64, 128, 9).to(gu.DEV)
    prm = moe.RouteParams(B=64, d=256, N=128, k=8)
    sel = moe.SelectParams(score=moe.SCORE_SIGMOID, n_group=8, topk_group=4, group_top=2)
    want, _ = run(x, None, prm, sel)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, flags = run(x, None, prm, sel, stream=s)
    assert flags == 0 and torch.equal(got.expert_idx, want.expert_idx) and torch.equal(got.weights, want.weights)
    r, ws = moe.Routing(prm, gu.DEV), moe.alloc_workspace(prm, 0, gu.DEV)
    moe.moe_route_scores(x, None, prm, sel, r, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_route_scores(x, None, prm, sel, r, ws)
    r.weights.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.weights, want.weights) and torch.equal(r.perm, want.perm)
