"""The block of examples/drafted_block.py against the same step in plain
64-bit arithmetic, up to the routing, and its expert half against the oracle."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("aware_expert_routing_gb300")
import oracle  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from aware_expert_routing_gb300 import build as b
    b.build()
    spec = importlib.util.spec_from_file_location("drafted_block", os.path.join(ROOT, "examples", "drafted_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_example_runs(example, capsys):
    example.main()
    assert "a step takes" in capsys.readouterr().out


def test_block_step(example):
    b = example.Block(d=256, heads=8, kv_heads=2, head_dim=64, experts=64, k=4, d_ff=128, pages=64, requests=3, max_len=256,
                      max_tokens=16)
    parents = [[-1, 0, 0, 1], [-1], [-1, 0, 1, 1, 0]]
    off, depth, request, mask = example.drafted(parents)
    T = int(off[-1])
    ctx = torch.tensor([70, 33, 0], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    b.cache.k.normal_(generator=g)
    b.cache.v.normal_(generator=g)
    x = torch.randn(T, 256, generator=g, device="cuda").to(torch.bfloat16)
    y = b.step(x, ctx, off, depth, request, mask)
    assert moe.moe_device_status(b.scratch) == 0 and moe.moe_device_status(b.ws) == 0
    # the attention's result, from the rows that the step wrote and the rest of the cache
    qkv = (x @ b.w_qkv.T).view(T, -1, 64).cpu()
    pos = (ctx[request.long()] + depth).cpu()
    q, _ = ref.rotate(qkv[:, :8], b.rope.cpu(), pos, 0)
    o, _, tol, _ = ref.attend(q.to(torch.bfloat16), b.cache.k.cpu(), b.cache.v.cpu(), b.table.cpu(), off.cpu(), ctx.cpu(),
                              mask.cpu(), 64 ** -0.5, True)
    h = x.double().cpu() + o.reshape(T, -1) @ b.w_out.double().cpu().T
    # hidden states are rounded to bf16 twice on the way (product, sum), and the attention's to bf16 once
    slack = 4 * ref.U16 * (h.abs() + (o.abs().reshape(T, -1) @ b.w_out.double().cpu().abs().T)) + \
        tol.reshape(T, -1) @ b.w_out.double().cpu().abs().T
    r = b.routing
    idx, w = r.expert_idx.cpu().numpy(), r.weights.cpu().numpy()
    assert (idx >= 0).all() and abs(w.sum(1) - 2.5).max() < 1e-5
    # y - experts(h) = h: the expert half is checked with the chosen experts on the 64-bit hidden states
    e = oracle.moe_experts(h.numpy().astype(np.float32), *(t.float().cpu().numpy() for t in (b.w_gate, b.w_up, b.w_down)), idx,
                           w.astype(np.float64))
    err = (y.double().cpu() - h - torch.from_numpy(e)).abs()
    scale = float(np.abs(e).max()) + float(h.abs().max())
    assert (err <= slack + 2e-2 * scale).all()
