"""Scores of -infinity (GPU): an infinite element of a key whose factor in the query is of the
other sign. Such a key weighs zero, wherever it stands among the others (alone in what a group
of lanes has seen so far, first, in whole tiles); a row with no other key gets zeros. The
result is the oracle's on the keys that remain, within dense_bound.py's tolerance."""
import math

import numpy as np
import pytest
import torch

from dense_bound import excess
from margins import check
from oracle import rows as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32

# which keys score -infinity: j -> bool
HIDDEN = {
    "first": lambda j: j == 0,
    "last": lambda j: j == j.max(),
    "all but the last": lambda j: j < j.max(),
    "a pair of rows": lambda j: (j % 16 == 5) & (j < 32),
    "every eighth": lambda j: j % 8 == 3,
    "the first tile": lambda j: j < 128,
    "all": lambda j: j >= 0,
}


def case(B, S, L, H, Hkv, d, dt, hidden, seed=3):
    g = torch.Generator().manual_seed(seed + L)
    q = torch.randn(B, S, H, d, generator=g) * 1.5
    q[..., 3] = q[..., 3].abs() + 0.5
    k, v = torch.randn(B, Hkv, L, d, generator=g), torch.randn(B, Hkv, L, d, generator=g)
    out = HIDDEN[hidden](torch.arange(L))
    k[:, :, out, 3] = -float("inf")
    return [t.to(dt).to(DEV) for t in (q, k, v)] + [out.numpy()]


def verify(q, k, v, hidden, scale, out, tc, seen=lambda i: None):
    """seen(i): how many keys row i sees (None: all)."""
    f = lambda t: t.double().cpu().numpy()
    worst = 0.0
    for b in range(q.shape[0]):
        for i in range(q.shape[1]):
            keep = np.flatnonzero(~hidden[:seen(i)])
            o = R.attend(f(q[b, i:i + 1]), f(k[b])[:, keep], f(v[b])[:, keep], scale)
            worst = max(worst, excess(out[b, i:i + 1], o, q.dtype == BF16, tc, q.shape[-1], len(hidden)))
    check(worst, 1.0)


def cross(g, q, k, v, scale):
    B, S, H, d = q.shape
    out = torch.full_like(q, float("nan"))
    ws = g.cross_workspace(B, S, H, k.shape[1], d, d, k.shape[2], q.dtype)
    g.attn_cross(q, k, v, out, scale, workspace=ws)
    assert g.attn_get_device_error() == g.OK
    return out


@pytest.mark.parametrize("hidden", HIDDEN)
@pytest.mark.parametrize("dt,d", [(F32, 16), (F32, 64), (F32, 128), (BF16, 32), (BF16, 64), (BF16, 128), (BF16, 256)],
                         ids=lambda x: str(x).replace("torch.", ""))
def test_cross_one_row(gpu_lib, dt, d, hidden):
    scale = 1 / math.sqrt(d)
    for L in (*range(1, 18), 33, 70, 300, 700):  # 700: the row's keys are split
        q, k, v, out_of = case(2, 1, L, 2, 2, d, dt, hidden)
        verify(q, k, v, out_of, scale, cross(gpu_lib, q, k, v, scale), False)


@pytest.mark.parametrize("hidden", HIDDEN)
@pytest.mark.parametrize("dt,S,G,d", [(F32, 5, 2, 64), (F32, 3, 1, 128), (BF16, 3, 2, 32), (BF16, 20, 2, 64),
                                      (BF16, 5, 4, 128)], ids=lambda x: str(x).replace("torch.", ""))
def test_cross_several_rows(gpu_lib, dt, S, G, d, hidden):
    scale = 1 / math.sqrt(d)
    for L in (1, 2, 9, 16, 130, 300):
        q, k, v, out_of = case(2, S, L, 2 * G, 2, d, dt, hidden)
        verify(q, k, v, out_of, scale, cross(gpu_lib, q, k, v, scale), dt == BF16 and d in (64, 128))


@pytest.mark.parametrize("hidden", HIDDEN)
@pytest.mark.parametrize("dt,d", [(F32, 64), (BF16, 64), (BF16, 128)], ids=lambda x: str(x).replace("torch.", ""))
def test_decode_and_prefill(gpu_lib, dt, d, hidden):
    """The causal calls on the same kernel: one row against a contiguous and a paged cache, and
    fp32 rows each of which sees one key more."""
    g = gpu_lib
    scale = 1 / math.sqrt(d)
    for L in (1, 2, 8, 16, 17, 33, 300):
        q, k, v, out_of = case(2, 1, L, 4, 2, d, dt, hidden)
        lens = torch.full((2,), L, dtype=torch.int32, device=DEV)
        out = torch.full((2, 4, d), float("nan"), dtype=dt, device=DEV)
        g.attn_decode_contig(q[:, 0].contiguous(), k, v, lens, out, scale)
        verify(q, k, v, out_of, scale, out[:, None], False)
        n = (L + 15) // 16
        pools = []
        for x in (k, v):
            pool = torch.full((2 * n, 2, 16, d), float("nan"), dtype=dt, device=DEV)
            for b in range(2):
                for j in range(L):
                    pool[b * n + j // 16, :, j % 16] = x[b, :, j]
            pools.append(pool)
        tables = torch.arange(2 * n, dtype=torch.int32, device=DEV).view(2, n)
        paged = torch.full_like(out, float("nan"))
        g.attn_decode_paged(q[:, 0].contiguous(), *pools, tables, lens, paged, scale)
        assert torch.equal(paged, out)
    if dt == F32:
        for L in (1, 5, 17, 40):
            q, k, v, out_of = case(1, L, L, 4, 2, d, dt, hidden)
            out = torch.full_like(q, float("nan"))
            g.attn_prefill_causal(q, k, v, out, scale)
            verify(q, k, v, out_of, scale, out, False, seen=lambda i: i + 1)
    assert g.attn_get_device_error() == g.OK
