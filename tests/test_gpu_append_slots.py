"""Append by slots (GPU): norm, rotation and write of rows whose positions and slots are given, against
the fp64 oracle; the tolerance is test_gpu_qk_rows.py's."""
import math

import pytest
import torch

from margins import check
from oracle import rows as R
from test_gpu_qk_rows import DEV, ROPES, excess, f64, gen, packed, weight

pytestmark = pytest.mark.gpu


def rope_of(g, d, which):
    layout, offset, share, scaling = ROPES[which]
    rot = max(2, int(d * share) // 2 * 2)
    offset = min(offset, d - rot)
    kw = dict(scaling)
    kind = kw.pop("scaling", "none")
    rope = g.rope_init(rot, 1e5, layout=layout, rot_offset=offset, scaling=kind, **kw)
    freqs = R.frequencies(rot, 1e5, kind, kw.get("factor", 1.0), kw.get("original_max", 0.0), kw.get("low", 1.0), kw.get("high", 4.0))
    return rope, layout, offset, freqs, 0.1 * math.log(kw["factor"]) + 1 if kind == "index" else 1.0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,H,Hkv,d,dv,bs,which,norm", [
    (1, 1, 1, 64, 64, 16, 0, True),
    (37, 8, 2, 128, 128, 16, 1, True),
    (130, 14, 2, 64, 64, 12, 2, False),
    (11, 6, 3, 96, 48, 8, 3, True),
    (9, 4, 4, 32, 32, 128, 4, True),
    (23, 0, 2, 256, 256, 64, 5, False),
    (700, 1, 1, 64, 64, 16, None, True),
    (21000, 1, 1, 64, 64, 16, 0, True),   # several tokens a warp
])
def test_append_slots(gpu_lib, dt, N, H, Hkv, d, dv, bs, which, norm):
    g, r = gpu_lib, gen(N + d)
    nb = N // bs + 3
    if H:
        q, k = packed([H, Hkv], (N,), d, dt, r)
    else:
        q, (k,) = None, packed([Hkv], (N,), d, dt, r)
    v = torch.randn(N, Hkv, dv, generator=r).to(dt).to(DEV)
    slots = torch.randperm(nb * bs, generator=r)[:N].to(DEV)
    slots[1::7] = -1  # rows without a slot (a single row has one)
    pos = torch.randint(0, 200000, (N,), generator=r).to(torch.int32).to(DEV)
    wq, wk = (weight(d, dt, r), weight(d, dt, r)) if norm else (None, None)
    rope, layout, offset, freqs, mag = rope_of(g, d, which) if which is not None else (None, "half", 0, [], 1.0)
    kp, vp = torch.randn(nb, Hkv, bs, d, generator=r).to(dt).to(DEV), torch.randn(nb, Hkv, bs, dv, generator=r).to(dt).to(DEV)
    kp0, vp0 = kp.clone(), vp.clone()
    q_out = None if q is None else torch.full((N, H, d), 7.0, dtype=dt, device=DEV)
    g.kv_append_slots(q, k, v, q_out, kp, vp, slots, pos if rope is not None else None, rope, wq if H else None, wk, 1e-5)
    assert g.attn_get_device_error() == g.OK
    real = (slots >= 0).cpu().numpy()
    at = pos.cpu().numpy()
    blk, row = slots.clamp(min=0) // bs, slots.clamp(min=0) % bs
    want, size = R.rotate(R.norm(f64(k), f64(wk), 1e-5), at, freqs, layout, offset, mag)
    check(excess(kp[blk, :, row][slots >= 0], want[real], size[real], dt, at[real]), 1.0)
    assert torch.equal(vp[blk, :, row][slots >= 0], v[slots >= 0])
    if H:
        want, size = R.rotate(R.norm(f64(q), f64(wq), 1e-5), at, freqs, layout, offset, mag)
        check(excess(q_out[slots >= 0], want[real], size[real], dt, at[real]), 1.0)
        assert (q_out[slots < 0] == 7.0).all()
    kept = torch.ones(nb * bs, dtype=torch.bool, device=DEV)
    kept[slots[slots >= 0]] = False  # the other slots are as they were
    for pool, was in ((kp, kp0), (vp, vp0)):
        flat, flat0 = pool.transpose(1, 2).reshape(nb * bs, -1), was.transpose(1, 2).reshape(nb * bs, -1)
        assert torch.equal(flat[kept], flat0[kept])


def test_the_slots_of_a_plain_append(gpu_lib):
    """With the slots and positions behind each sequence's rows the call is kv_append_paged_rows, bit for bit."""
    g, r = gpu_lib, gen(5)
    B, H, Hkv, d, bs, mbps = 5, 8, 2, 128, 16, 20
    lens, rows = torch.tensor([0, 17, 100, 5, 250]), torch.tensor([30, 1, 0, 44, 9])
    starts = torch.cat([torch.zeros(1, dtype=torch.long), rows.cumsum(0)])
    N = int(starts[-1])
    tables = torch.randperm(B * mbps, generator=r).view(B, mbps)
    b = torch.repeat_interleave(torch.arange(B), rows)
    pos = lens[b] + torch.arange(N) - starts[b]
    slots = tables[b, pos // bs] * bs + pos % bs
    i32 = lambda x: x.to(torch.int32).to(DEV)  # noqa: E731
    q, k, v = packed([H, Hkv, Hkv], (N,), d, torch.bfloat16, r)
    w = weight(d, torch.bfloat16, r)
    rope = g.rope_init(d, 1e6, layout="half")
    pools = [torch.zeros(B * mbps, Hkv, bs, d, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    outs = [torch.zeros(N, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    g.kv_append_paged_rows(q, k, v, outs[0], pools[0], pools[1], i32(tables), i32(starts), i32(lens),
                           torch.empty(B, dtype=torch.int32, device=DEV), rope=rope, q_weight=w, k_weight=w)
    g.kv_append_slots(q, k, v, outs[1], pools[2], pools[3], slots.to(DEV), i32(pos), rope=rope, q_weight=w, k_weight=w)
    assert torch.equal(outs[0], outs[1]) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert g.attn_get_device_error() == g.OK


@pytest.mark.parametrize("N", [3, 21000])
def test_slots_past_the_pool_and_queries_in_place(gpu_lib, N):
    g, r = gpu_lib, gen(6)
    q, k, v = packed([1, 1, 1], (N,), 64, torch.bfloat16, r)
    nb = N // 16 + 2
    kp, vp = torch.zeros(nb, 1, 16, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(nb, 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(N, device=DEV)
    slots[1] = nb * 16
    slots[2] = 1 << 40
    before = q.clone()
    pos = torch.zeros(N, dtype=torch.int32, device=DEV)
    pos[0] = 9
    g.kv_append_slots(q, k, v, q, kp, vp, slots, pos, g.rope_init(64, 1e4))
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    assert torch.equal(q[1:], before[1:]) and not torch.equal(q[0], before[0])  # (position 0 turns by nothing)
    assert not kp[0, 0, 1:3].any() and torch.equal(vp[0, 0, 0], v[0, 0])
