"""moe_rope_table, moe_kv_append, moe_tree_attention and the grouped routing
without a GPU: bad arguments are refused on the host before anything is
launched, and the host-side helpers."""
import ctypes
import math

import pytest
import torch

import attention_ref as ref

import aware_expert_routing_gb300 as moe
from aware_expert_routing_gb300 import build as moe_build

FAKE = 4096    # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def cache(**kw):
    base = dict(k=FAKE, v=FAKE, page_table=FAKE, n_pages=10, page_size=16, kv_heads=4, head_dim=128, n_requests=2,
                max_pages=4, dtype=0)
    base.update(kw)
    return moe._KvCache(**base)


BAD_CACHE = [dict(dtype=2), dict(head_dim=0), dict(head_dim=12), dict(head_dim=264), dict(page_size=0),
             dict(page_size=65537), dict(kv_heads=0), dict(n_pages=-1), dict(k=None), dict(v=FAKE + 8)]


def append(lib, c=None, q=FAKE, k=FAKE, v=FAKE, rope=FAKE, pos=FAKE, slots=FAKE, q_out=FAKE, ws=FAKE, ws_bytes=512, **kw):
    base = dict(T=3, heads=8, rot=128, n_pos=100, interleaved=0, q_tok=2048, q_head=128, k_tok=2048, k_head=128,
                v_tok=2048, v_head=128, out_tok=1024, out_head=128)
    base.update(kw)
    c = cache(page_table=None, n_requests=0, max_pages=0) if c is None else c
    return lib.moe_kv_append(q, k, v, rope, pos, slots, ctypes.byref(moe._Append(**base)), ctypes.byref(c), q_out, ws,
                             ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(heads=0), dict(heads=1025), dict(rot=3), dict(rot=130), dict(rot=-2), dict(n_pos=0),
    dict(interleaved=2), dict(q_tok=2049), dict(k_head=4), dict(v_tok=-2048), dict(out_head=1), dict(q=None),
    dict(q_out=None), dict(k=None), dict(v=None), dict(rope=None), dict(pos=None), dict(slots=None), dict(q=FAKE + 2),
    dict(v=FAKE + 8), dict(pos=FAKE + 2), dict(slots=FAKE + 4), dict(rope=FAKE + 4)])
def test_append_refuses(lib, kw):
    assert append(lib, **kw) == moe.MOE_ERR_ARG
    assert lib.moe_last_error()


@pytest.mark.parametrize("kw", BAD_CACHE)
def test_append_refuses_a_bad_cache(lib, kw):
    assert append(lib, cache(**kw)) == moe.MOE_ERR_ARG
    assert lib.moe_kv_append(*([FAKE] * 6), None, ctypes.byref(cache()), FAKE, FAKE, 512, None) == moe.MOE_ERR_ARG
    prm = moe._Append()
    assert lib.moe_kv_append(*([FAKE] * 6), ctypes.byref(prm), None, FAKE, FAKE, 512, None) == moe.MOE_ERR_ARG


def test_append_workspace(lib):
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=511)):
        assert append(lib, **kw) == moe.MOE_ERR_WORKSPACE
    assert append(lib, T=0, k=None, slots=None) == moe.MOE_OK      # nothing to do, nothing launched


def attend(lib, c=None, q=FAKE, off=FAKE, ctx=FAKE, mask=FAKE, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40, **kw):
    base = dict(T=5, heads=8, mask_words=1, scale=0.1, q_tok=1024, q_head=128)
    base.update(kw)
    c = cache() if c is None else c
    return lib.moe_tree_attention(q, off, ctx, mask, ctypes.byref(moe._Attention(**base)), ctypes.byref(c), out, lse, ws,
                                  ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(heads=0), dict(heads=6), dict(heads=1028), dict(mask_words=0), dict(mask_words=-1), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(q=None), dict(off=None), dict(ctx=None),
    dict(out=None), dict(q=FAKE + 8), dict(out=FAKE + 2), dict(off=FAKE + 1), dict(ctx=FAKE + 2), dict(mask=FAKE + 2),
    dict(lse=FAKE + 1), dict(q_tok=1023), dict(q_head=-128)])
def test_attention_refuses(lib, kw):
    assert attend(lib, **kw) == moe.MOE_ERR_ARG
    assert lib.moe_last_error()


@pytest.mark.parametrize("kw", BAD_CACHE + [dict(n_requests=1025), dict(n_requests=-1), dict(max_pages=-1),
                                            dict(max_pages=1 << 30), dict(page_table=None), dict(page_table=FAKE + 2)])
def test_attention_refuses_a_bad_cache(lib, kw):
    assert attend(lib, cache(**kw)) == moe.MOE_ERR_ARG
    assert lib.moe_attention_workspace_bytes(5, 8, ctypes.byref(cache(**kw))) == 0


def test_attention_workspace(lib):
    need = lib.moe_attention_workspace_bytes(5, 8, ctypes.byref(cache()))
    assert need >= moe.ATTENTION_WORKSPACE_MIN
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=need - 1)):
        assert attend(lib, **kw) == moe.MOE_ERR_WORKSPACE
    assert lib.moe_attention_workspace_bytes(-1, 8, ctypes.byref(cache())) == 0
    assert lib.moe_attention_workspace_bytes(5, 6, ctypes.byref(cache())) == 0
    assert lib.moe_attention_workspace_bytes(5, 8, None) == 0
    assert attend(lib, T=0, q=None, off=None) == moe.MOE_OK
    assert attend(lib, cache(n_requests=0, page_table=None), q=None) == moe.MOE_OK


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=7), dict(rot=258), dict(scaling=4), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
    dict(scaling=1, factor=0.5), dict(scaling=2, factor=math.inf), dict(scaling=2, rot=2, factor=2.0),
    dict(scaling=3, factor=2.0, original_len=0.0), dict(scaling=3, factor=2.0, original_len=10.0, beta_fast=1.0),
    dict(scaling=3, factor=2.0, original_len=10.0, beta_slow=0.0), dict(magnitude=math.nan)])
def test_rope_table_refuses(lib, kw):
    prm = moe.RopeParams(**{"rot": 64, **kw}).c()
    assert lib.moe_rope_table(ctypes.byref(prm), 10, FAKE, None) == moe.MOE_ERR_ARG
    ok = moe.RopeParams(rot=64).c()
    assert lib.moe_rope_table(ctypes.byref(ok), -1, FAKE, None) == moe.MOE_ERR_ARG
    assert lib.moe_rope_table(ctypes.byref(ok), 10, None, None) == moe.MOE_ERR_ARG
    assert lib.moe_rope_table(ctypes.byref(ok), 10, FAKE + 4, None) == moe.MOE_ERR_ARG
    assert lib.moe_rope_table(None, 10, FAKE, None) == moe.MOE_ERR_ARG
    assert lib.moe_rope_table(ctypes.byref(ok), 0, None, None) == moe.MOE_OK


@pytest.mark.parametrize("sel", [
    dict(score=2), dict(n_group=0), dict(n_group=7), dict(n_group=64), dict(n_group=8, topk_group=0),
    dict(n_group=8, topk_group=9), dict(group_top=0), dict(group_top=3), dict(n_group=16, topk_group=1),
    dict(renormalise=2), dict(scale=math.inf), dict(scale=math.nan)])
def test_selection_refuses(lib, sel):
    prm = moe.RouteParams(B=4, d=256, N=128, k=10).c()
    r = moe._Routing(*([FAKE] * 7 + [None, None]))
    s = moe._Select(**{**dict(score=1, n_group=1, topk_group=1, group_top=1, renormalise=1, scale=1.0), **sel})
    a = (ctypes.byref(prm), ctypes.byref(s), ctypes.byref(r))
    assert lib.moe_route_scores(FAKE, None, *a, FAKE, 1 << 30, None) == moe.MOE_ERR_ARG
    assert lib.moe_route_grouped(FAKE, FAKE, None, None, *a, FAKE, 1 << 30, None) == moe.MOE_ERR_ARG
    assert lib.moe_decode_layer_grouped(FAKE, FAKE, None, None, FAKE, FAKE, FAKE, 128, *a, FAKE, FAKE, 1 << 30,
                                        None) == moe.MOE_ERR_ARG


def test_selection_refuses_pointers_modes_and_workspaces(lib):
    r = moe._Routing(*([FAKE] * 7 + [None, None]))
    s = moe.SelectParams(score=1, n_group=8, topk_group=4, group_top=2).c()
    prm = moe.RouteParams(B=4, d=256, N=128, k=8)

    def call(scores=FAKE, bias=None, p=prm, sel=s, ws=FAKE, n=1 << 30):
        return lib.moe_route_scores(scores, bias, ctypes.byref(p.c()) if p else None, ctypes.byref(sel) if sel else None,
                                    ctypes.byref(r), ws, n, None)

    for kw in (dict(scores=None), dict(scores=FAKE + 2), dict(bias=FAKE + 1), dict(p=None), dict(sel=None),
               dict(p=moe.RouteParams(B=4, d=256, N=128, k=8, mode=moe.MODE_OEA, k0=3)),
               dict(p=moe.RouteParams(B=257, d=256, N=128, k=8))):
        assert call(**kw) == moe.MOE_ERR_ARG, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 64), dict(n=100)):
        assert call(**kw) == moe.MOE_ERR_WORKSPACE, kw
    assert lib.moe_route_grouped(FAKE, None, None, None, ctypes.byref(prm.c()), ctypes.byref(s), ctypes.byref(r), FAKE,
                                 1 << 30, None) == moe.MOE_ERR_ARG


def test_python_calls_refuse_tensors_of_the_wrong_kind(lib):
    cpu = torch.zeros(2, 4, 16, 64)
    with pytest.raises(ValueError):
        moe.KvCache(cpu, cpu)
    with pytest.raises(ValueError):
        moe.KvCache(cpu.half(), cpu.half())
    with pytest.raises(ValueError):
        moe.moe_route_scores(torch.zeros(4, 128), None, moe.RouteParams(B=4, d=256, N=128, k=8), moe.SelectParams(), None,
                             None)
    with pytest.raises(ValueError):
        moe.moe_rope_table(moe.RopeParams(rot=64), 4, "cpu")


def test_tree_mask():
    # 0 - 1 - 3
    #   \ 2   4 (a second root)
    m = moe.tree_mask([-1, 0, 0, 1, -1])
    assert m.tolist() == [[0b1], [0b11], [0b101], [0b1011], [0b10000]]
    chain = moe.tree_mask(range(-1, 69))
    assert chain.shape == (70, 3) and chain.dtype == torch.int32
    bits = [sum(bin(w & 0xffffffff).count("1") for w in row) for row in chain.tolist()]
    assert bits == list(range(1, 71))
    assert moe.tree_mask([]).shape == (0, 0)
    for bad in ([0], [-2], [-1, 1], [-1, 5]):
        with pytest.raises(ValueError):
            moe.tree_mask(bad)


def test_reference_attention_is_a_softmax_and_a_derivative():
    """The 64-bit statement itself: lse's derivative by the scores is the weight of each value (by differences), and a
    causal mask given as words equals none."""
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(3, 1, 4, 8, generator=g, dtype=torch.float64) for _ in range(2))
    q = torch.randn(3, 2, 8, generator=g, dtype=torch.float64)
    table, off, ctx = torch.tensor([[2, 0, 1]], dtype=torch.int32), torch.tensor([0, 3]), torch.tensor([5])
    o, l, _, _ = ref.attend(q, k, v, table, off, ctx, None, 0.3, False)
    o2, l2, _, _ = ref.attend(q, k, v, table, off, ctx, moe.tree_mask([-1, 0, 1]), 0.3, False)
    assert torch.equal(o, o2) and torch.equal(l, l2)
    # d lse / d q = scale * sum_j p_j k_j: the output with k in the values' place
    grad, _, _, _ = ref.attend(q, k, k, table, off, ctx, None, 0.3, False)
    h = 1e-6
    for c in range(8):
        dq = torch.zeros_like(q)
        dq[..., c] = h
        up = ref.attend(q + dq, k, v, table, off, ctx, None, 0.3, False)[1]
        down = ref.attend(q - dq, k, v, table, off, ctx, None, 0.3, False)[1]
        assert ((up - down) / (2 * h) - 0.3 * grad[..., c]).abs().max() < 1e-8
