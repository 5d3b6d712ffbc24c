"""Descriptors of another device than the current one are refused: the kernels run on the current one."""
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


def test_descriptors_of_another_device_are_refused():
    """(Whose tensors only say so: no second device is there.)"""
    k, v, q = (torch.ones(2, h, 64, device=DEV).to(torch.bfloat16) for h in (2, 2, 4))
    slots = torch.arange(2, device=DEV)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    off, ctx = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 2], [0]))
    plain = moe.KvCache(*(torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)), table)
    q8 = moe.alloc_kv_cache_q8(1, 2, 16, 64, 8, DEV, table)
    norm = moe.HeadNorm(torch.ones(64, dtype=torch.bfloat16, device=DEV), None)
    ws = moe.alloc_attention_workspace(2, 4, plain, DEV)
    ws8 = moe.alloc_attention_workspace(2, 4, q8, DEV)
    out = torch.empty_like(q)
    calls = [(plain, lambda: moe.moe_kv_append(None, k, v, None, None, slots, plain, None, ws)),
             (plain, lambda: moe.moe_kv_append_norm(None, k, v, None, None, slots, norm, plain, None, ws)),
             (norm, lambda: moe.moe_kv_append_norm(None, k, v, None, None, slots, norm, plain, None, ws)),
             (plain, lambda: moe.moe_tree_attention(q, off, ctx, None, plain, out, None, ws)),
             (q8, lambda: moe.moe_kv_append_q8(None, k, v, None, None, slots, norm, q8, None, ws8)),
             (norm, lambda: moe.moe_kv_append_q8(None, k, v, None, None, slots, norm, q8, None, ws8)),
             (q8, lambda: moe.moe_kv_read_q8(slots, q8, k.clone(), None, ws8)),
             (q8, lambda: moe.moe_tree_attention_q8(q, off, ctx, None, q8, out, None, ws8))]
    for x, call in calls:
        assert x._c.device == 0
        call()
        x._c.device = 1
        with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
            call()
        x._c.device = 0
    assert moe.moe_device_status(ws) == 0 and moe.moe_device_status(ws8) == 0
