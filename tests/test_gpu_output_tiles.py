"""Cross attention whose warpgroups write one output tile after another (GPU): units of several
row tiles a slot, so that the output buffer is reused and its barriers pass many phases."""
import math

import pytest
import torch

from dense_bound import excess
from margins import check
from oracle import rows as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inputs(B, S, L, H, Hkv, dk, dv):
    g = torch.Generator(device=DEV).manual_seed(B + S)
    t = [torch.randn(s, generator=g, device=DEV).bfloat16()
         for s in ((B, S, H, dk), (B, Hkv, L, dk), (B, Hkv, L, dv))]
    lens = torch.randint(0, L + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    return *t, lens


def run(g, q, k, v, lens):
    B, S, H, dk = q.shape
    _, Hkv, L, dv = v.shape
    out = torch.full((B, S, H, dv), float("nan"), dtype=q.dtype, device=DEV)
    g.attn_cross(q, k, v, out, 1 / math.sqrt(dk), lens, g.cross_workspace(B, S, H, Hkv, dk, dv, L))
    return out


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)], ids=str)
def test_many_tiles_a_slot(gpu_lib, dims):
    dk, dv = dims
    B, S, L, H, Hkv = 60, 301, 90, 16, 8  # 60 x 8 x 5 row tiles of 64 rows on at most 304 slots
    q, k, v, lens = inputs(B, S, L, H, Hkv, dk, dv)
    out = run(gpu_lib, q, k, v, lens)
    assert gpu_lib.attn_get_device_error() == gpu_lib.OK
    worst = 0.0
    f = lambda t: t.double().cpu().numpy()
    for b in range(0, B, 7):
        n = int(lens[b])
        o = R.attend(f(q[b]), f(k[b, :, :n]), f(v[b, :, :n]), 1 / math.sqrt(dk))
        worst = max(worst, excess(out[b], o, True, True, dk, n))
    check(worst, 1.0)
    for _ in range(3):
        assert torch.equal(run(gpu_lib, q, k, v, lens), out)


def test_withheld_tile_with_many_tiles_a_slot(gpu_lib):
    """Every slot gives up in its first tile, none waits for the others' outputs."""
    g = gpu_lib
    q, k, v, lens = inputs(60, 301, 90, 16, 8, 128, 128)
    lens.clamp_(min=1)
    want = run(g, q, k, v, lens)
    assert g.attn_get_device_error() == g.OK
    g.gqa_debug_withhold_first_tile(1)
    try:
        run(g, q, k, v, lens)
        assert g.attn_get_device_error() == g.ERR_DEVICE_TIMEOUT
    finally:
        g.gqa_debug_withhold_first_tile(0)
    assert torch.equal(run(g, q, k, v, lens), want)
    assert g.attn_get_device_error() == g.OK
