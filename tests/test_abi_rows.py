"""Host-side refusals of the q/k row calls (CPU): each call fails a check before any launch."""
import ctypes

import pytest
import torch

INV = 1
P = 16  # a non-null, 16-byte aligned stand-in: never dereferenced
N = None


@pytest.fixture(scope="module")
def g():
    from causal_gqa_attention_row_gb300 import build
    build.build()
    import causal_gqa_attention_row_gb300 as g
    g.load()
    return g


def norm_rope(g, q=(P, 64, 64, 8), k=(32, 64, 64, 8), qo=(48, 64, 64, 8), ko=(64, 64, 64, 8), wq=N, wk=N, eps=1e-6,
              pos=P, B=2, T=3, H=4, Hkv=2, d=64, rope=(0, 0, 64, 1.0, 8), dt=1):
    v = [N if x is N else ctypes.byref(g.GqaHeads(*x)) for x in (q, k, qo, ko)]
    r = N if rope is N else ctypes.byref(g.GqaRope(*rope))
    return g.load().attn_qk_norm_rope(*v, wq, wk, eps, pos, B, T, H, Hkv, d, r, dt, N)


@pytest.mark.parametrize("kw", [
    dict(dt=7), dict(B=-1), dict(T=-1), dict(H=-1), dict(d=60), dict(d=264), dict(B=1 << 20, T=1 << 20),
    dict(q=N), dict(qo=N), dict(k=N), dict(ko=N), dict(H=0), dict(Hkv=0),
    dict(q=(0, 64, 64, 8)), dict(q=(18, 64, 64, 8)), dict(q=(P, 60, 64, 8)), dict(k=(32, 64, 4, 8)),
    dict(ko=(64, 64, 64, 4)), dict(qo=(P, 64, 64, 16)),            # in place with other strides
    dict(wq=24), dict(wk=8), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(pos=N),
    dict(rope=(2, 0, 64, 1.0, 8)), dict(rope=(-1, 0, 64, 1.0, 8)), dict(rope=(0, 0, 63, 1.0, 8)),
    dict(rope=(0, 0, 0, 1.0, 8)), dict(rope=(0, -1, 64, 1.0, 8)), dict(rope=(0, 1, 64, 1.0, 8)),
    dict(rope=(0, 0, 64, float("nan"), 8)), dict(rope=(0, 0, 64, 1.0, 0)), dict(rope=(0, 0, 64, 1.0, 4)),
    dict(rope=(0, 2 ** 31 - 1, 64, 1.0, 8)),
])
def test_norm_rope_refusals(g, kw):
    assert norm_rope(g, **kw) == INV


def test_norm_rope_empty(g):
    assert norm_rope(g, B=0) == 0 and norm_rope(g, T=0) == 0
    assert norm_rope(g, q=N, k=N, qo=N, ko=N, H=0, Hkv=0) == 0


def append(g, q=(P, 0, 64, 64), k=(32, 0, 64, 64), v=(48, 0, 64, 64), qo=(64, 0, 64, 64), kp=P, vp=P, tab=P, starts=P,
           lin=64, lout=128, n=5, B=2, mbps=4, nb=9, bs=16, H=4, Hkv=2, dk=64, dv=64, wq=N, wk=N, eps=1e-6, rope=N,
           dt=1):
    x = [N if y is N else ctypes.byref(g.GqaHeads(*y)) for y in (q, k, v, qo)]
    r = N if rope is N else ctypes.byref(g.GqaRope(*rope))
    return g.load().kv_append_paged_rows(*x, kp, vp, tab, starts, lin, lout, n, B, mbps, nb, bs, H, Hkv, dk, dv, wq, wk,
                                         eps, r, dt, N)


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(n=-1), dict(B=-1), dict(mbps=0), dict(nb=0), dict(bs=0), dict(mbps=1 << 20, bs=1 << 20),
    dict(H=-1), dict(Hkv=0), dict(dk=12), dict(dv=0), dict(dk=512), dict(q=N), dict(qo=N), dict(H=0),
    dict(k=N), dict(v=N), dict(kp=N), dict(vp=N), dict(tab=N), dict(starts=N), dict(lin=N), dict(lout=N),
    dict(kp=24), dict(vp=8), dict(k=(34, 0, 64, 64)), dict(v=(48, 0, 63, 64)), dict(q=(P, 0, 64, 4)),
    dict(qo=(P, 0, 64, 128)), dict(lout=68), dict(wq=4), dict(eps=-0.5), dict(rope=(1, 32, 64, 1.0, 8)),
])
def test_append_refusals(g, kw):
    assert append(g, **kw) == INV


def test_append_empty(g):
    assert append(g, B=0) == 0


def test_binding_checks(g):
    """Shapes and layouts that the binding turns down, with tensors that live on the CPU."""
    x = torch.zeros(2, 3, 4, 64)
    with pytest.raises(ValueError):
        g._view(x.transpose(-1, -2), 4)      # last axis not dense
    with pytest.raises(ValueError):
        g._view(x, 3)
    with pytest.raises(ValueError):
        g._writes_once(x[:, :, :1].expand(2, 3, 4, 64))
    with pytest.raises(ValueError):
        g.attn_qk_norm_rope(None, None, None, None, None)
    with pytest.raises(ValueError):
        g.attn_qk_norm_rope(x, None, None, None, None)
    with pytest.raises(ValueError):
        g.rope_frequencies(8, 1e4, divisors=[1.0])
    assert g._view(None, 4) is None
    for y in (x, x.transpose(1, 2)):
        h = g.GqaHeads.from_buffer_copy(g._view(y, 4))
        assert (h.data, h.batch_stride, h.token_stride, h.head_stride) == (y.data_ptr(), *y.stride()[:3])
    h = g.GqaHeads.from_buffer_copy(g._view(x[0], 3))
    assert (h.data, h.batch_stride, h.token_stride, h.head_stride) == (x.data_ptr(), 0, 256, 64)


def test_an_axis_of_one_element_has_no_stride(g):
    # B = T = Hkv = 1: any strides go; refused for another reason (no positions), not for them
    odd = dict(q=(P, 3, 5, 64), qo=(48, 7, 1, 64), k=(32, 1, 1, 1), ko=(64, 9, 9, 9), B=1, T=1, Hkv=1)
    assert norm_rope(g, **odd, pos=N) == INV
    assert norm_rope(g, **{**odd, "q": (P, 3, 5, 60)}, pos=P) == INV      # the heads' own stride counts
