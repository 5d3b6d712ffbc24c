"""Appends into a cache in 8 bits at the edges of what they take."""
import math

import pytest
import torch

import test_gpu_append_norm as append

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("aware_expert_routing_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from aware_expert_routing_gb300 import build as b
    b.build()
    moe.load()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [1e-45, 1e-41, 1e-38, 1e-30, 1e30])
def test_rows_of_zeros_and_large_rows_at_any_eps(dtype, eps):
    """A row of zeros stays one whatever eps is; the codes of large rows (their sum of squares about 2^126) are those of the
    statement."""
    c = append.Case([(0, 24)], 2, 2, 64, 64, 16, layout="own", dtype=dtype, weights="shared", seed=6, eps=eps)
    c.k[3] = c.q[3] = 0
    c.k[16:] = c.q[16:] = 0
    c.k[5] = (c.k[5].float() * 2.0 ** 60).to(c.dt)
    c8 = append.Cache8(c, 8, 4)
    q, k, v, rope, pos, slots = c.on_gpu()
    q_out = torch.full_like(q, math.nan)
    ws = append.workspace()
    moe.moe_kv_append_q8(q, k, v, rope, pos, slots, c.norm, c8.gpu, q_out, ws)
    assert moe.moe_device_status(ws) == 0
    assert (q_out[3] == 0).all() and (q_out[16:] == 0).all()
    c8.check(c, c.slots, True, c.wk)


@pytest.mark.parametrize("T,block", [(9, 8), (9, 1), (300, 8), (300, 1), (1100, 8), (1100, 1)])
@pytest.mark.parametrize("skip", [-1, 1 << 40])
@pytest.mark.parametrize("position", [-1, 700])
def test_positions_of_skipped_tokens_are_checked_without_queries(T, block, skip, position):
    """The flag does not depend on whether queries are given, nor on the cache's kind."""
    c = append.Case([(4, T)], 2, 1, 64, 64, 16, layout="own", seed=3)
    at = T - 4                                  # (a slot past the cache raises the flag by itself: two calls differ)
    c.slots[at] = skip
    for bad in (False, True):
        if bad:
            c.positions[at] = position
        q, k, v, rope, pos, slots = c.on_gpu()
        plain = moe.KvCache(*(torch.zeros(c.P, 1, 16, 64, dtype=c.dt, device=DEV) for _ in range(2)))
        want = moe.FLAG_BAD_INDEX if bad or skip > 0 else 0
        q_out = torch.empty_like(q)
        for qs in ((None, None), (q, q_out)):
            c8 = append.Cache8(c, block, 2)
            ws = append.workspace()
            moe.moe_kv_append_q8(qs[0], k, v, rope, pos, slots, c.norm, c8.gpu, qs[1], ws)
            assert moe.moe_device_status(ws) == want
            moe.moe_kv_append_norm(qs[0], k, v, rope, pos, slots, c.norm, plain, qs[1], ws)
            assert moe.moe_device_status(ws) == want
            c8.check(c, c.slots, True, c.wk)


@pytest.mark.parametrize("T", [7, 64, 255, 256])
@pytest.mark.parametrize("block", [1, 4, 16])
@pytest.mark.parametrize("kind", ["singles", "drafts"])
def test_padded_decode_batches(T, block, kind):
    """Up to 256 tokens, some of them padding: between requests, inside blocks, at either end."""
    g = torch.Generator().manual_seed(T + block)
    if kind == "singles":
        spans = [(int(torch.randint(0, 16, (1,), generator=g)), 1) for _ in range(T)]
    else:
        spans, left = [], T
        while left:
            n = min(left, int(torch.randint(1, 12, (1,), generator=g)))
            spans.append((int(torch.randint(0, 16, (1,), generator=g)), n))
            left -= n
    c = append.Case(spans, 4, 2, 64, 64, 16, seed=T)
    c.slots[torch.rand(T, generator=g) < 0.35] = -1
    c.slots[0] = c.slots[T - 1] = -1
    c8 = append.Cache8(c, block, 12)
    q, k, v, rope, pos, slots = c.on_gpu()
    q_out = torch.full((T, 4, 64), math.nan, dtype=c.dt, device=DEV)
    ws = append.workspace()
    moe.moe_kv_append_q8(q, k, v, rope, pos, slots, c.norm, c8.gpu, q_out, ws)
    assert moe.moe_device_status(ws) == 0
    append.close(q_out, *c.want(c.q, c.wq), c.dt)
    c8.check(c, c.slots, True, c.wk)
