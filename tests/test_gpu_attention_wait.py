"""moe_tree_attention when a wait runs out: with a bound of a microsecond it
gives up, says so and ends, and the next call on the same workspace is right."""
import pytest
import torch

from test_gpu_attention import Case, DEV, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from aware_expert_routing_gb300 import build as b
    b.build()
    moe.load()


# 320 or 272 rows a key head: units of 256 rows and of 64 or 16, in which the second row tile has nothing to do but to
# wait for the next unit, for as long as the first works through a context (118 key tiles of a microsecond or two)
@pytest.mark.parametrize("R,ctx,n,H,D", [(24, 15000, 40, 32, 128), (24, 15000, 40, 32, 64), (20, 20000, 34, 32, 128)])
def test_waits_that_run_out_are_flagged_and_the_workspace_recovers(R, ctx, n, H, D):
    K, page = 4, 16
    g = torch.Generator(device=DEV).manual_seed(3)
    pages = (ctx + n + page - 1) // page
    ck, cv = (torch.randn(R * pages, K, page, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    cache = moe.KvCache(ck, cv, torch.randperm(R * pages, generator=g, device=DEV).to(torch.int32).reshape(R, pages))
    q = torch.randn(R * n, H, D, generator=g, device=DEV).to(torch.bfloat16)
    off = torch.arange(R + 1, dtype=torch.int32, device=DEV) * n
    lens = torch.full((R,), ctx, dtype=torch.int32, device=DEV)
    ws = moe.alloc_attention_workspace(R * n, H, cache, DEV)
    out, lse = torch.empty_like(q), torch.empty(R * n, H, device=DEV)

    def call():
        moe.moe_tree_attention(q, off, lens, None, cache, out, lse, ws)
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



def test_a_small_call_after_one_that_gave_up():
    """The workspace serves another shape next; a call of units of few rows whose waits may run out or not."""
    K, page, D, H = 4, 16, 128, 32
    big = Case([9000] * 24, [40] * 24, H, K, D, page, "bf16", False, 71)
    small = Case([100, 7], [2, 3], H, K, D, page, "bf16", True, 72)
    few = Case([3000] * 8, [5] * 8, H, K, D, page, "bf16", True, 73)
    ws = moe.alloc_attention_workspace(960, H, moe.KvCache(big.k.to(DEV), big.v.to(DEV), big.table.to(DEV)), DEV)
    for c in (big, few):
        moe.moe_set_wait_timeout_us(1)
        try:
            flags = c.run(ws=ws)[2]
        finally:
            moe.moe_set_wait_timeout_us(0)
        assert flags == moe.FLAG_WAIT_TIMEOUT if c is big else flags in (0, moe.FLAG_WAIT_TIMEOUT)
        out, l, flags = small.run(ws=ws)
        assert flags == 0
        small.check(out, l)
