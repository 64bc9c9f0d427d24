"""Host-side refusals of the calls of a step that verifies drafted tokens (CPU): each fails a check
before any launch."""
import ctypes

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
