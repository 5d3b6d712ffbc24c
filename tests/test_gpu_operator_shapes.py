"""Sizes at which moe_kv_append and moe_tree_attention take kernels that the
other tests' sizes do not reach."""
import pytest
import torch

import attention_ref as ref
from test_gpu_append import DEV, check, make
from test_gpu_attention import Case, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from aware_expert_routing_gb300 import build as b
    b.build()
    moe.load()


# from 4000 tokens on the append has small blocks: both pair layouts, both types, rotated in part or not at all
@pytest.mark.parametrize("T,H,K,D,rot,page,inter,layout,dtype", [
    (4000, 4, 2, 64, 64, 16, 0, "fused", "bf16"), (4133, 3, 1, 128, 64, 32, 0, "own", "bf16"),
    (4100, 4, 2, 64, 32, 16, 1, "fused", "bf16"), (4001, 2, 2, 80, 80, 8, 1, "heads first", "bf16"),
    (4050, 2, 1, 64, 0, 16, 0, "own", "bf16"), (4003, 2, 1, 256, 256, 16, 0, "fused", "bf16"),
    (4010, 4, 1, 64, 32, 16, 0, "fused", "f32"), (4002, 2, 1, 128, 128, 16, 1, "own", "f32"),
    (4000, 2, 1, 40, 20, 5, 0, "own", "bf16")])
def test_append_of_many_tokens(T, H, K, D, rot, page, inter, layout, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, rope, positions, slots, ck, cv = make(T, H, K, D, rot, page, layout, dt, 2000 + T)
    slots[T // 3] = -1
    want_v, before_k = cv.cpu().clone(), ck.cpu().clone()
    q_out = torch.full((T, H, D), float("nan"), dtype=dt, device=DEV)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    moe.moe_kv_append(q, k, v, rope, positions.to(DEV) if rot else None, slots.to(DEV), moe.KvCache(ck, cv), q_out, ws,
                      interleaved=bool(inter))
    assert moe.moe_device_status(ws) == 0
    table = rope.cpu() if rot else torch.zeros(1, 0)
    pos = positions if rot else torch.zeros(T, dtype=torch.int32)
    yq, eq = ref.rotate(q.cpu(), table, pos, inter)
    yk, ek = ref.rotate(k.cpu(), table, pos, inter)
    check(q_out, yq, eq, dt)
    live = slots >= 0
    pg, row = slots[live] // page, slots[live] % page
    check(ck[pg.to(DEV), :, row.to(DEV)], yk[live], ek[live], dt)
    want_v[pg, :, row] = v.cpu()[live]
    assert torch.equal(cv.cpu(), want_v)
    touched = torch.zeros(ck.shape[0], page, dtype=torch.bool)
    touched[pg, row] = True
    assert torch.equal(ck.cpu().permute(0, 2, 1, 3)[~touched], before_k.permute(0, 2, 1, 3)[~touched])


# CUDA cores: heads of 129 to 192 components, and every height of a unit (4, 8, 16, 32, 64 rows) at every width; the
# contexts are long enough that units are cut
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [136, 192, 256, 80, 48])
@pytest.mark.parametrize("ctx,n,H,K,tree", [([700, 3], [1, 1], 2, 1, False), ([1500], [3], 4, 2, True),
                                            ([900, 40, 0], [4, 2, 7], 8, 2, True), ([600], [8], 4, 1, False),
                                            ([410, 5], [20, 9], 4, 1, True), ([300], [70], 2, 1, True),
                                            ([0, 90], [130, 3], 2, 2, False)])
def test_attention_on_cuda_cores(dtype, D, ctx, n, H, K, tree):
    c = Case(ctx, n, H, K, D, 16, dtype, tree, 61 + D + H)
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)
    again, l2, _ = c.run()
    assert torch.equal(again, out) and torch.equal(l2, l)
