"""moe_rope_table and moe_kv_append against plain 64-bit statements."""
import math

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("aware_expert_routing_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from aware_expert_routing_gb300 import build as b
    b.build()
    moe.load()


def normal(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("kw", [
    dict(rot=64, base=10000.0), dict(rot=2, base=500.0), dict(rot=128, base=1e6, scaling="linear", factor=4.0),
    dict(rot=96, base=10000.0, scaling="ntk", factor=8.0),
    dict(rot=128, base=10000.0, scaling="yarn", factor=16.0, original_len=4096.0),
    dict(rot=64, base=1e6, scaling="yarn", factor=40.0, original_len=32768.0, beta_fast=32.0, beta_slow=1.0),
    dict(rot=8, base=10000.0, scaling="yarn", factor=2.0, original_len=64.0, beta_fast=4.0, beta_slow=3.9)])
def test_rope_table(kw):
    f, mag = ref.rope_frequencies(**kw)
    n = 5001
    mode = dict(plain=moe.ROPE_PLAIN, linear=moe.ROPE_LINEAR, ntk=moe.ROPE_NTK, yarn=moe.ROPE_YARN)
    prm = moe.RopeParams(**{**kw, "scaling": mode[kw.get("scaling", "plain")]})
    got = moe.moe_rope_table(prm, n, DEV).cpu().double()
    a = torch.arange(n, dtype=torch.float64)[:, None] * torch.tensor(f, dtype=torch.float64)
    want = torch.cat([a.cos(), a.sin()], 1) * mag
    # one rounding to fp32, and the angle's own: 5000 turns of 2^-52 relative
    assert (got - want).abs().max() <= ref.U32 * mag + 1e-10


def test_rope_table_long_positions_and_magnitude():
    got = moe.moe_rope_table(moe.RopeParams(rot=4, base=100.0, magnitude=0.5), 1_048_576, DEV)[-1].cpu().double()
    want = [0.5 * g(1_048_575 * f) for g in (math.cos, math.sin) for f in (1.0, 0.1)]
    assert (got - torch.tensor(want, dtype=torch.float64)).abs().max() <= ref.U32
    assert moe.moe_rope_table(moe.RopeParams(rot=8), 0, DEV).shape == (0, 8)


# T, heads, kv_heads, D, rot, page, interleaved, layout of q/k/v, dtype
CASES = [
    (1, 8, 1, 128, 128, 16, 0, "fused", "bf16"), (1, 1, 1, 8, 0, 1, 0, "own", "bf16"),
    (7, 4, 2, 64, 64, 16, 1, "fused", "bf16"), (33, 6, 3, 80, 20, 5, 0, "own", "bf16"),
    (33, 6, 3, 80, 40, 8, 1, "heads first", "bf16"), (130, 16, 4, 128, 64, 32, 0, "fused", "bf16"),
    (64, 5, 5, 256, 256, 64, 1, "own", "bf16"), (19, 10, 2, 72, 18, 7, 0, "fused", "bf16"),
    (3, 2, 1, 96, 2, 16, 1, "fused", "bf16"), (300, 32, 8, 128, 128, 128, 0, "heads first", "bf16"),
    (1, 8, 2, 128, 128, 16, 1, "fused", "f32"), (21, 4, 4, 64, 32, 16, 0, "own", "f32"),
    (40, 5, 1, 40, 36, 3, 1, "heads first", "f32"), (129, 16, 2, 256, 64, 16, 0, "fused", "f32"),
    (2000, 4, 2, 64, 64, 16, 0, "fused", "bf16"),
]


def make(T, H, K, D, rot, page, layout, dt, seed, n_pos=700):
    if layout == "fused":
        qkv = normal((T, H + 2 * K, D), dt, seed).to(DEV)
        q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    elif layout == "own":
        q, k, v = (normal((T, h, D), dt, seed + i).to(DEV) for i, h in enumerate((H, K, K)))
    else:
        q, k, v = (normal((h, T, D), dt, seed + i).to(DEV).transpose(0, 1) for i, h in enumerate((H, K, K)))
    g = torch.Generator().manual_seed(seed + 9)
    pages = (T + page - 1) // page + 3
    slots = torch.randperm(pages * page, generator=g)[:T]
    positions = torch.randint(0, n_pos, (T,), generator=g).to(torch.int32)
    rope = moe.moe_rope_table(moe.RopeParams(rot=rot), n_pos, DEV) if rot else None
    ck, cv = (normal((pages, K, page, D), dt, seed + 20 + i).to(DEV) for i in range(2))
    return q, k, v, rope, positions, slots, ck, cv


def check(got, want, err, dt):
    tol = err + (ref.U16 * (want.abs() + err) if dt == torch.bfloat16 else ref.U32 * want.abs())
    assert ((got.cpu().double() - want).abs() <= tol + 1e-40).all()


@pytest.mark.parametrize("T,H,K,D,rot,page,inter,layout,dtype", CASES)
def test_append(T, H, K, D, rot, page, inter, layout, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, rope, positions, slots, ck, cv = make(T, H, K, D, rot, page, layout, dt, 1000 + T)
    slots[T // 2] = -1                       # one token is padding
    want_k, want_v = ck.cpu().clone(), cv.cpu().clone()
    before_k = want_k.clone()
    q_out = torch.full((T, H, D), float("nan"), dtype=dt, device=DEV)
    cache = moe.KvCache(ck, cv)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    moe.moe_kv_append(q, k, v, rope, positions.to(DEV) if rot else None, slots.to(DEV), cache, q_out, ws,
                      interleaved=bool(inter))
    assert moe.moe_device_status(ws) == 0
    table = rope.cpu() if rot else torch.zeros(1, 0)
    pos = positions if rot else torch.zeros(T, dtype=torch.int32)
    yq, eq = ref.rotate(q.cpu(), table, pos, inter)
    yk, ek = ref.rotate(k.cpu(), table, pos, inter)
    check(q_out, yq, eq, dt)
    assert torch.equal(q_out[..., rot:].cpu(), q[..., rot:].cpu())
    live = slots >= 0
    pg, row = slots[live] // page, slots[live] % page
    check(ck[pg.to(DEV), :, row.to(DEV)], yk[live], ek[live], dt)
    # every other row of the cache is as it was, values are copied bit for bit
    want_v[pg, :, row] = v.cpu()[live]
    assert torch.equal(cv.cpu(), want_v)
    touched = torch.zeros(ck.shape[0], page, dtype=torch.bool)
    touched[pg, row] = True
    assert torch.equal(ck.cpu().permute(0, 2, 1, 3)[~touched], before_k.permute(0, 2, 1, 3)[~touched])


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_in_place_and_without_queries(inter):
    T, H, K, D, page = 37, 4, 2, 64, 16
    q, k, v, rope, positions, slots, ck, cv = make(T, H, K, D, 64, page, "fused", torch.bfloat16, 5)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    q_out = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    args = (rope, positions.to(DEV), slots.to(DEV))
    moe.moe_kv_append(q, k, v, *args, moe.KvCache(ck, cv), q_out, ws, interleaved=inter)
    k1, v1 = torch.zeros_like(ck), torch.zeros_like(cv)
    moe.moe_kv_append(None, k, v, *args, moe.KvCache(k1, v1), None, ws, interleaved=inter)
    moe.moe_kv_append(q, k, v, *args, moe.KvCache(ck, cv), q, ws, interleaved=inter)   # q rotated in place
    assert torch.equal(q, q_out)
    pg, row = (slots // page).to(DEV), (slots % page).to(DEV)
    assert torch.equal(k1[pg, :, row], ck[pg, :, row]) and torch.equal(v1[pg, :, row], v)


def test_relative_positions():
    """A rotated query's product with a rotated key depends on the distance."""
    D = 64
    q, k = normal((1, 1, D), torch.float32, 1).to(DEV), normal((1, 1, D), torch.float32, 2).to(DEV)
    rope = moe.moe_rope_table(moe.RopeParams(rot=D), 4096, DEV)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    T = 3
    at = torch.tensor([5, 1005, 4000], dtype=torch.int32, device=DEV)
    dots = []
    for shift in (0, 90):
        ck, cv, qo = (torch.zeros(1, 1, T, D, device=DEV), torch.zeros(1, 1, T, D, device=DEV),
                      torch.empty(T, 1, D, device=DEV))
        slots = torch.arange(T, device=DEV)
        qs, ks = q.expand(T, 1, D).contiguous(), k.expand(T, 1, D).contiguous()
        moe.moe_kv_append(qs, ks, ks, rope, at + shift, slots, moe.KvCache(ck, cv), qo, ws)
        dots.append(qo if shift else ck[0, 0, :, None])
    d = (dots[0].double() * dots[1].double()).sum(-1)
    # table entries 2^-24 off, products of norms about 64
    assert (d - d[0]).abs().max() <= 8 * ref.U32 * float(q.norm() * k.norm())


def test_bad_slots_and_positions_raise_the_flag_and_write_nothing_else():
    T, H, K, D, page = 6, 2, 1, 64, 4
    q, k, v, rope, positions, slots, ck, cv = make(T, H, K, D, 64, page, "own", torch.bfloat16, 8, n_pos=50)
    n = ck.shape[0] * page
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    q_out = torch.empty_like(q)
    for bad in (n, n + 5, 1 << 40):
        s = slots.clone()
        s[2] = bad
        k1, v1 = torch.zeros_like(ck), torch.zeros_like(cv)
        moe.moe_kv_append(q, k, v, rope, positions.to(DEV), s.to(DEV), moe.KvCache(k1, v1), q_out, ws)
        assert moe.moe_device_status(ws) == moe.FLAG_BAD_INDEX
        assert moe.moe_device_status(ws) == 0
        assert int((v1.permute(0, 2, 1, 3).abs().sum((-1, -2)) != 0).sum()) == T - 1
    for bad in (-1, 50, 1 << 30):
        p = positions.clone()
        p[1] = bad
        near = positions.clone()
        near[1] = 0 if bad < 0 else 49
        moe.moe_kv_append(q, k, v, rope, p.to(DEV), slots.to(DEV), moe.KvCache(ck, cv), q_out, ws)
        assert moe.moe_device_status(ws) == moe.FLAG_BAD_INDEX
        want = torch.empty_like(q)
        moe.moe_kv_append(q, k, v, rope, near.to(DEV), slots.to(DEV), moe.KvCache(ck, cv), want, ws)
        assert torch.equal(q_out, want) and moe.moe_device_status(ws) == 0


def test_cache_past_2_31_elements():
    """Pages whose offsets in the cache pass 32 bits."""
    K, page, D = 4, 64, 128
    pages = (1 << 31) // (K * page * D) + 40
    ck = torch.empty(pages, K, page, D, dtype=torch.bfloat16, device=DEV)
    cv = torch.empty_like(ck)
    ck[-2:] = 0
    cv[-2:] = 0
    T = 3
    q, k, v, rope, positions, _, _, _ = make(T, 8, K, D, D, page, "fused", torch.bfloat16, 3)
    slots = torch.tensor([(pages - 1) * page + 63, (pages - 2) * page, (pages - 1) * page], device=DEV)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    q_out = torch.empty(T, 8, D, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv_append(q, k, v, rope, positions.to(DEV), slots, moe.KvCache(ck, cv), q_out, ws)
    assert moe.moe_device_status(ws) == 0
    assert torch.equal(cv[-1, :, 63], v[0]) and torch.equal(cv[-2, :, 0], v[1]) and torch.equal(cv[-1, :, 0], v[2])
    yk, ek = ref.rotate(k.cpu(), rope.cpu(), positions, 0)
    check(ck[-1, :, 63], yk[0], ek[0], torch.bfloat16)
    assert int((cv[-2:] != 0).any(-1).sum()) == T * K


def test_on_another_stream_and_in_a_graph():
    T, H, K, D, page = 50, 8, 2, 128, 16
    q, k, v, rope, positions, slots, ck, cv = make(T, H, K, D, D, page, "fused", torch.bfloat16, 77)
    positions, slots = positions.to(DEV), slots.to(DEV)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    want, got, again = (torch.zeros(T, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    moe.moe_kv_append(q, k, v, rope, positions, slots, moe.KvCache(ck, cv), want, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    moe.moe_kv_append(q, k, v, rope, positions, slots, moe.KvCache(ck, cv), got, ws, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_kv_append(q, k, v, rope, positions, slots, moe.KvCache(ck, cv), again, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, want)
