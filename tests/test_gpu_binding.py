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
