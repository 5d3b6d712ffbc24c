"""moe_tree_attention_q8 when a wait runs out, in the forms of its tensor-core kernels for few rows and for one widened row
tile: the call gives up, says so and ends, and the next call on the same workspace is right."""
import pytest
import torch

import q8_ref as q8

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("aware_expert_routing_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from aware_expert_routing_gb300 import build as b
    b.build()
    moe.load()


# Four requests far apart in a table of 1024, all others without tokens.  A CTA whose stretch goes from one request to the
# next steps over some hundred others in between, which takes its softmax and its MMAs tens of microseconds, while its
# copies, which have gone ahead, wait with full rings for as long: far longer than the bound.  (A try of a barrier may
# suspend a thread for longer than a tile takes, so the waits within a unit need not give up.)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("group", [8, 16, 24, 40, 80])     # query heads a key head: units of 16, 32, and widened
def test_waits_that_run_out_are_flagged_in_every_form(group, page, D):
    R, K = 1024, 2
    real, ctx = [0, 300, 620, 1023], [160000, 277000, 201000, 254000]
    n = torch.zeros(R, dtype=torch.int32)
    n[real] = 1
    lens = torch.zeros(R, dtype=torch.int32)
    lens[real] = torch.tensor(ctx, dtype=torch.int32)
    per = [(c + page) // page for c in ctx]
    g = torch.Generator(device=DEV).manual_seed(3)
    P = sum(per)
    codes = [torch.randint(0, 0x70, (P, K, page, D), generator=g, device=DEV, dtype=torch.uint8).view(q8.F8) for _ in range(2)]
    scales = [torch.full((P, K, page // 8), 2.0 ** -6, device=DEV) for _ in range(2)]
    order = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(R, max(per), dtype=torch.int32, device=DEV)
    at = 0
    for r, p in zip(real, per):
        table[r, :p] = order[at:at + p]
        at += p
    cache = moe.KvCacheQ8(*codes, *scales, table)
    T, H = 4, group * K
    q = torch.randn(T, H, D, generator=g, device=DEV).to(torch.bfloat16)
    off = torch.cat([torch.zeros(1, dtype=torch.int32), n.cumsum(0).to(torch.int32)]).to(DEV)
    lens = lens.to(DEV)
    ws = moe.alloc_attention_workspace(T, H, cache, DEV)
    out, lse = torch.empty_like(q), torch.empty(T, H, device=DEV)

    def call():
        moe.moe_tree_attention_q8(q, off, lens, None, cache, out, lse, ws)
        return moe.moe_device_status(ws)

    assert call() == 0
    want, want_lse = out.clone(), lse.clone()
    assert bool(want.isfinite().all())
    for _ in range(3):
        moe.moe_set_wait_timeout_us(1)
        try:
            assert call() == moe.FLAG_WAIT_TIMEOUT
        finally:
            moe.moe_set_wait_timeout_us(0)
        assert call() == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
