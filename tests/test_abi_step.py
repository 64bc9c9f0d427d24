"""Host-side refusals of the calls of a step that verifies drafted tokens (CPU): each fails a check
before any launch."""
import ctypes
import random

import pytest
import torch

INV, UNSUP = 1, 2
P = 16  # a non-null, aligned stand-in: never dereferenced
N = None


@pytest.fixture(scope="module")
def g():
    from causal_gqa_attention_row_gb300 import build
    build.build()
    import causal_gqa_attention_row_gb300 as g
    g.load()
    return g


def plan(g, lens=P, new=P, tab=P, bin=P, bout=4096, keep=N, flist=P, fin=P, fout=4096, starts=P, pos=P, slots=P, par=N,
         mask=N, words=0, n=64, B=4, mbps=8, nb=50, bs=16):
    return g.load().kv_plan_rows(lens, new, tab, bin, bout, keep, flist, fin, fout, starts, pos, slots, par, mask, words, n, B,
                                 mbps, nb, bs, N)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INV), (dict(B=-1), INV), (dict(mbps=0), INV), (dict(nb=0), INV), (dict(bs=0), INV),
    (dict(mbps=1 << 20, bs=1 << 20), INV), (dict(B=16384, mbps=1 << 18), INV), (dict(B=16385), UNSUP),
    (dict(lens=N), INV), (dict(new=N), INV), (dict(tab=N), INV), (dict(bin=N), INV), (dict(bout=N), INV),
    (dict(flist=N), INV), (dict(fin=N), INV), (dict(fout=N), INV), (dict(starts=N), INV), (dict(pos=N), INV),
    (dict(slots=N), INV), (dict(slots=20), INV), (dict(par=P), INV), (dict(mask=P, words=1), INV),
    (dict(par=P, mask=P), INV), (dict(par=P, mask=20, words=1), INV), (dict(words=1), INV),
    (dict(bin=16, bout=20), INV), (dict(bin=20, bout=16), INV), (dict(fin=20, fout=16), INV),
])
def test_plan_refusals(g, kw, want):
    assert plan(g, **kw) == want


def test_plan_of_nothing(g):
    assert plan(g, B=0, lens=N) == 0


def append(g, q=True, k=True, v=True, qo=True, kp=P, vp=P, slots=P, pos=P, n=5, nb=50, bs=16, H=8, Hkv=2, dk=128, dv=128,
           wq=N, wk=N, eps=1e-6, rope=True, dt=1, at=P, stride=128):
    def view(on):
        return ctypes.byref(g.GqaHeads(at, 0, 8 * stride, stride)) if on else N
    r = ctypes.byref(g.GqaRope(1, 0, 64, 1.0, P)) if rope else N
    return g.load().kv_append_slots(view(q), view(k), view(v), view(qo), kp, vp, slots, pos, n, nb, bs, H, Hkv, dk, dv, wq, wk,
                                    eps, r, dt, N)


@pytest.mark.parametrize("kw", [
    dict(dt=7), dict(n=-1), dict(nb=0), dict(bs=0), dict(H=-1), dict(Hkv=0), dict(dk=100), dict(dv=264), dict(q=False),
    dict(qo=False), dict(H=0), dict(k=False), dict(v=False), dict(kp=N), dict(vp=N), dict(kp=24), dict(slots=N),
    dict(slots=12), dict(pos=N), dict(wq=24), dict(eps=float("nan")), dict(eps=-1.0), dict(at=18), dict(stride=100), dict(dk=32),
])
def test_append_refusals(g, kw):
    assert append(g, **kw) == INV


def test_append_of_nothing(g):
    assert append(g, n=0, slots=N) == 0


def commit(g, k=(P, P), v=(P, P), layers=2, tab=P, lin=P, starts=P, path=P, npath=P, lout=4096, B=3, most=4, mbps=8, nb=50,
           bs=16, Hkv=2, dk=64, dv=64, dt=1):
    def array(x):
        return N if x is N else (ctypes.c_void_p * len(x))(*x)
    return g.load().kv_commit_rows(array(k), array(v), layers, tab, lin, starts, path, npath, lout, B, most, mbps, nb, bs, Hkv, dk,
                                   dv, dt, N)


@pytest.mark.parametrize("kw", [
    dict(dt=3), dict(layers=0), dict(B=-1), dict(most=-1), dict(mbps=0), dict(nb=0), dict(bs=0), dict(Hkv=0), dict(dk=12),
    dict(dv=1032), dict(mbps=1 << 20, bs=1 << 20), dict(k=N), dict(k=(P, N)), dict(k=(P, 24)), dict(v=(P, N)), dict(tab=N),
    dict(lin=N), dict(starts=N), dict(path=N), dict(npath=N), dict(lout=N), dict(lin=16, lout=20),
])
def test_commit_refusals(g, kw):
    assert commit(g, **kw) == INV


def test_commit_of_nothing(g):
    assert commit(g, B=0, k=N) == 0


def test_binding_checks(g):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool = torch.zeros(5, 2, 16, 64)
    with pytest.raises(ValueError):  # a mask without parents
        g.kv_plan_rows(i(2), i(2), i(2, 8), i(2), i(2), i(9), i(1), i(2), i(3), i(6), torch.zeros(6, dtype=torch.int64), 16,
                       tree_mask=torch.zeros(6, 1, dtype=torch.int64))
    with pytest.raises(ValueError):  # free_out of one entry
        g.kv_plan_rows(i(2), i(2), i(2, 8), i(2), i(2), i(9), i(1), i(1), i(3), i(6), torch.zeros(6, dtype=torch.int64), 16)
    with pytest.raises(ValueError):  # slots of another number
        g.kv_append_slots(None, torch.zeros(3, 2, 64), torch.zeros(3, 2, 64), None, pool, pool, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):  # layers without values
        g.kv_commit_rows([pool, pool], [pool], i(2, 8), i(2), i(3), i(2, 4), i(2), i(2))
    with pytest.raises(ValueError):  # pools of two shapes
        g.kv_commit_rows([pool, pool[:4]], None, i(2, 8), i(2), i(3), i(2, 4), i(2), i(2))


def tree(g, q=P, k=P, v=P, tab=P, off=P, starts=P, mask=P, out=P, n=20, B=4, most=8, words=1, mbps=8, nb=50, bs=16, H=8, Hkv=2,
         dk=128, dv=128, scale=0.1, dt=1, ws=P, size=1 << 40, arms=N):
    a = N if arms is N else ctypes.byref(g.GqaArms(*arms))
    return g.load().attn_tree_paged(q, k, v, tab, off, starts, mask, out, n, B, most, words, mbps, nb, bs, H, Hkv, dk, dv, scale,
                                    dt, ws, size, a, N)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=5), INV), (dict(n=-1), INV), (dict(B=-1), INV), (dict(most=0), INV), (dict(words=-1), INV), (dict(mbps=0), INV),
    (dict(nb=0), INV), (dict(bs=0), INV), (dict(H=7), INV), (dict(dk=100), INV), (dict(dv=0), INV), (dict(mbps=1 << 20, bs=1 << 20), INV),
    (dict(n=1 << 30), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(mask=N), INV), (dict(words=0), INV),
    (dict(most=65), INV), (dict(q=N), INV), (dict(k=N), INV), (dict(v=N), INV), (dict(tab=N), INV), (dict(starts=N), INV),
    (dict(out=N), INV), (dict(q=24), INV), (dict(out=40), INV), (dict(mask=20), INV), (dict(ws=N), 4), (dict(size=1000), 4), (dict(ws=24), INV),
    (dict(arms=(0, float("nan"), N, N)), INV), (dict(arms=(0, 0.0, 18, N)), INV), (dict(dk=40, dv=40), UNSUP),
    (dict(n=4000, B=1000, mbps=1 << 25), INV),
])
def test_tree_refusals(g, kw, want):
    assert tree(g, **kw) == want


def test_tree_of_nothing_and_its_workspace(g):
    assert tree(g, B=0, q=N, ws=N) == 0 and tree(g, n=0, q=N, ws=N) == 0
    f = g.attn_tree_paged_workspace_bytes
    assert f(0, 4, 8, 128, 8, 2, 128, 128) == 0 and f(20, 4, 8, 128, 8, 3, 128, 128) == 0
    need = f(20, 4, 8, 128, 8, 2, 128, 128, torch.float32)
    assert tree(g, dt=0, size=need - 1) == 4
    # a workspace does for everything smaller

    r = random.Random(1)
    for _ in range(300):
        H, Hkv = r.choice([(8, 2), (14, 2), (4, 4), (130, 1), (64, 1)])
        d, dt = r.choice([(64, torch.bfloat16), (128, torch.bfloat16), (32, torch.bfloat16), (64, torch.float32), (256, torch.float32)])
        big = (r.randint(1, 5000), r.randint(1, 3000), r.randint(1, 300), r.randint(1, 9000))
        small = tuple(r.randint(1, x) for x in big)
        assert f(*small, H, Hkv, d, d, dt) <= f(*big, H, Hkv, d, d, dt), (small, big, H, Hkv, d, dt)


def test_tree_binding_checks(g):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool, q = torch.zeros(5, 2, 16, 64), torch.zeros(6, 4, 64)
    mask = torch.zeros(6, 1, dtype=torch.int64)
    for kw in (dict(mask=mask[:5]), dict(mask=mask[:, 0]), dict(out=q[:5]), dict(starts=i(2)), dict(off=i(3))):
        a = dict(dict(mask=mask, out=q, starts=i(3), off=i(2)), **kw)
        with pytest.raises(ValueError):
            g.attn_tree_paged(q, pool, pool, i(2, 8), a["off"], a["starts"], a["mask"], a["out"], 0.1, 4, None)
