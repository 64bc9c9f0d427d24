"""attn_cross_workspace_bytes bounds what every smaller batch and every shorter encoder length
needs (CPU: the sizes; GPU: calls of many sizes with the workspace of the largest)."""
import random

import pytest
import torch

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    from causal_gqa_attention_row_gb300 import build
    build.build()
    import causal_gqa_attention_row_gb300 as g
    g.load()
    return g


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 2, 16, 40, 300])
def test_never_falls_with_the_batch_or_the_length(g, dt, S):
    rng = random.Random(S)
    f = g.attn_cross_workspace_bytes
    assert f(8, 16, 4096, 8, 8, 64, 64) <= f(64, 16, 4096, 8, 8, 64, 64)
    for _ in range(3000):
        B, L = rng.randint(1, 300), int(2 ** rng.uniform(0, 17))
        Hkv, d = rng.choice([1, 2, 8, 16, 128]), rng.choice([16, 64, 128])
        H = Hkv * rng.choice([1, 1, 2, 7, 16, 130])
        most = f(B, S, L, H, Hkv, d, d, dt)
        assert f(rng.randint(1, B), S, rng.randint(1, L), H, Hkv, d, d, dt) <= most


def test_the_call_asks_for_no_more(g):
    """(a misaligned workspace of that size is refused as misaligned, one byte less of what the
    call itself needs as too small; both before any launch)"""
    P, INV, WS = 16, 1, 4

    def call(B, S, L, H, Hkv, d, dt, ws, size):
        return g.load().attn_cross(P, P, P, P, P, B, S, L, H, Hkv, d, d, 0.1, dt, ws, size, None)

    for B, S, L, H, Hkv, d, dt in ((8, 16, 4096, 8, 8, 64, 1), (2, 40, 700, 8, 2, 64, 1), (1, 1, 5000, 8, 2, 128, 0),
                                   (64, 1, 1500, 16, 16, 64, 1), (3, 1, 300, 4, 4, 128, 1)):
        size = g.attn_cross_workspace_bytes(B, S, L, H, Hkv, d, d, BF16 if dt else F32)
        assert call(B, S, L, H, Hkv, d, dt, P + 8, size) == INV
        assert call(B, S, L, H, Hkv, d, dt, None, size) == WS


@pytest.mark.gpu
@pytest.mark.parametrize("S,H,Hkv,dt", [(16, 8, 8, BF16), (3, 14, 2, BF16), (1, 4, 4, BF16), (1, 4, 2, F32)],
                         ids=["bf16 16", "bf16 group", "bf16 one row", "f32 one row"])
def test_one_workspace_for_a_shrinking_batch(gpu_lib, S, H, Hkv, dt):
    g = gpu_lib
    B, L, d = 64, 4096, 64
    gen = torch.Generator(device="cuda").manual_seed(S)
    q, k, v = (torch.randn(s, generator=gen, device="cuda").to(dt) for s in ((B, S, H, d), (B, Hkv, L, d), (B, Hkv, L, d)))
    ws = g.cross_workspace(B, S, H, Hkv, d, d, L, dt)
    for b, n in ((64, 4096), (33, 4096), (8, 4096), (1, 4096), (8, 700), (1, 300), (2, 100)):
        args = q[:b].contiguous(), k[:b, :, :n].contiguous(), v[:b, :, :n].contiguous()
        out, want = torch.empty_like(args[0]), torch.empty_like(args[0])
        g.attn_cross(*args, out, 0.125, workspace=ws)
        g.attn_cross(*args, want, 0.125, workspace=g.cross_workspace(b, S, H, Hkv, d, d, n, dt))
        assert g.attn_get_device_error() == g.OK
        assert torch.equal(out, want)
