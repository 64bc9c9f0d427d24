"""Host-side refusals and workspaces of attn_decode_shared_prefix and attn_cross (CPU): each
call fails a check before any launch."""
import ctypes

import pytest
import torch

INV, UNSUP, WS = 1, 2, 4
P = 16  # a non-null, 16-byte aligned stand-in: never dereferenced
N = None


@pytest.fixture(scope="module")
def g():
    from causal_gqa_attention_row_gb300 import build
    build.build()
    import causal_gqa_attention_row_gb300 as g
    g.load()
    return g


def shared(g, q=P, k=P, v=P, tab=P, lens=P, starts=P, sb=P, out=P, B=4, n=1, mbps=8, nb=50, bs=16, H=8, Hkv=2, dk=128,
           dv=128, scale=0.1, dt=1, ws=P, size=1 << 40, arms=N):
    a = N if arms is N else ctypes.byref(g.GqaArms(*arms))
    return g.load().attn_decode_shared_prefix(q, k, v, tab, lens, starts, sb, out, B, n, mbps, nb, bs, H, Hkv, dk, dv,
                                              scale, dt, ws, size, a, N)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=5), INV), (dict(B=-1), INV), (dict(n=-1), INV), (dict(mbps=0), INV), (dict(nb=0), INV), (dict(bs=0), INV),
    (dict(H=7), INV), (dict(dk=100), INV), (dict(dv=0), INV), (dict(mbps=1 << 20, bs=1 << 20), INV),
    (dict(q=N), INV), (dict(k=N), INV), (dict(v=N), INV), (dict(tab=N), INV), (dict(lens=N), INV), (dict(out=N), INV),
    (dict(starts=N), INV), (dict(sb=N), INV), (dict(q=18), INV), (dict(out=24), INV),
    (dict(ws=N), WS), (dict(size=100), WS), (dict(ws=24), INV),
    (dict(arms=(0, float("nan"), N, N)), INV), (dict(arms=(0, 0.0, 18, N)), INV),
    (dict(dk=40, dv=40), UNSUP),
])
def test_shared_prefix_refusals(g, kw, want):
    assert shared(g, **kw) == want


def test_shared_prefix_workspace(g):
    f = g.attn_decode_shared_prefix_workspace_bytes
    assert shared(g, B=0, q=N, ws=N) == 0
    assert f(0, 8, 2, 128, 1000, 1) == 0 and f(4, 8, 3, 128, 1000, 1) == 0
    # a sequence's own rows always leave partial results; prefixes only where two can share
    assert f(1, 8, 2, 128, 1000, 1) < f(2, 8, 2, 128, 1000, 1)
    assert f(4, 8, 2, 128, 1000, 1) < f(4, 8, 2, 128, 8000, 1)  # a partial result per key range
    # groups beyond the pairs of sequences add their records only
    assert f(4, 8, 2, 128, 1000, 50) - f(4, 8, 2, 128, 1000, 2) < 4096
    need = f(4, 8, 2, 128, 8 * 16, 1)
    assert shared(g, size=need - 1) == WS


def cross(g, q=P, k=P, v=P, lens=P, out=P, B=2, S=40, L=700, H=8, Hkv=2, dk=64, dv=64, scale=0.1, dt=1, ws=P,
          size=1 << 40):
    return g.load().attn_cross(q, k, v, lens, out, B, S, L, H, Hkv, dk, dv, scale, dt, ws, size, N)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=-1), INV), (dict(B=-1), INV), (dict(S=-1), INV), (dict(L=0), INV), (dict(L=2 ** 31 - 1), INV),
    (dict(H=7), INV), (dict(dk=60), INV), (dict(dv=264), INV), (dict(B=1 << 20, S=1 << 20), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(q=N), INV), (dict(k=N), INV), (dict(v=N), INV), (dict(out=N), INV), (dict(k=20), INV), (dict(out=40), INV),
    (dict(ws=N), WS), (dict(size=64), WS), (dict(ws=40), INV), (dict(dk=24, dv=24), UNSUP),
])
def test_cross_refusals(g, kw, want):
    assert cross(g, **kw) == want


def test_cross_empty_and_workspace(g):
    assert cross(g, B=0, q=N) == 0 and cross(g, S=0, q=N) == 0
    f = g.attn_cross_workspace_bytes
    assert f(0, 1, 10, 2, 1, 64, 64) == 0
    assert f(64, 1024, 100, 8, 8, 64, 64) == 0                     # enough row tiles: keys whole
    n = f(2, 40, 700, 8, 2, 64, 64)
    assert n > 0 and n % (128 * 66 * 4) == 0                       # a partial result per unit
    assert f(2, 40, 700, 8, 2, 64, 64, torch.float32) == 0         # fp32 rows read their keys whole
    assert f(1, 1, 5000, 8, 2, 128, 128, torch.float32) > 0        # one row: its keys are split


def test_binding_checks(g):
    x = torch.zeros(2, 3, 4, 64)
    with pytest.raises(ValueError):
        g.attn_cross(x, x, x, x[:, :2], 0.1)    # out of another shape
    t = torch.zeros(2, 8, dtype=torch.int32)
    pool = torch.zeros(5, 2, 16, 64)
    with pytest.raises(ValueError):
        g.attn_decode_shared_prefix(x[:, 0], pool, pool, t, t[:, 0], t[0, :1], t[0, :1], x[:, 0], 0.1, None)
