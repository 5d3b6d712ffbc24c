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
