"""Cross attention (GPU) against the fp64 oracle; the tolerance is dense_bound.py's."""
import math

import numpy as np
import pytest
import torch

from dense_bound import excess
from margins import check
from oracle import rows as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TC_ROWS = 2  # rows of a KV head from which bf16 calls run on the tensor cores, as the header says


def case(B, S, L, H, Hkv, dk, dv, dt, seed=1, std=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, S, H, dk, generator=g) * std).to(dt).to(DEV)
    k = torch.randn(B, Hkv, L, dk, generator=g).to(dt).to(DEV)
    v = torch.randn(B, Hkv, L, dv, generator=g).to(dt).to(DEV)
    return q, k, v


def f64(t):
    return t.double().cpu().numpy()


def run(g, q, k, v, scale, lens=None, ws="own", fill=None):
    B, S, H, dk = q.shape
    _, Hkv, L, dv = v.shape
    out = torch.full((B, S, H, dv), float("nan"), dtype=q.dtype, device=DEV)
    if ws == "own":
        ws = g.cross_workspace(B, S, H, Hkv, dk, dv, L, q.dtype)
        if ws is not None:
            ws.fill_(255 if fill is None else fill)  # NaN in every float: contents are not relied on
    g.attn_cross(q, k, v, out, scale, kv_lens=lens, workspace=ws)
    return out


def verify(g, q, k, v, scale, lens, out, tc):
    L = k.shape[2]
    n = [L] * q.shape[0] if lens is None else lens.tolist()
    worst = 0.0
    for b, m in enumerate(n):
        o = R.attend(f64(q[b]), f64(k[b, :, :m]), f64(v[b, :, :m]), scale)
        worst = max(worst, excess(out[b], o, q.dtype == torch.bfloat16, tc, q.shape[-1], m))
    check(worst, 1.0)


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)], ids=str)
@pytest.mark.parametrize("shape", [
    # B, S, L, H, Hkv, lens
    (1, 16, 1, 1, 1, None),             # one key
    (2, 16, 128, 2, 2, [128, 127]),     # one tile, and one key less
    (2, 33, 129, 8, 2, [129, 1]),       # a second tile of one key
    (3, 5, 700, 14, 2, [700, 0, 257]),  # group of 7 (126 of 128 rows), an empty sequence, split keys
    (1, 300, 520, 3, 1, [500]),         # several row tiles, a ragged last one
    (2, 40, 1025, 12, 3, None),
    (1, 2, 300, 130, 1, [299]),         # more heads than a tile has rows (chunks of 65)
    (1, 1, 2000, 16, 1, [1999]),        # one row of a large group
])
def test_tensor_cores(gpu_lib, dims, shape):
    g = gpu_lib
    B, S, L, H, Hkv, lens = shape
    dk, dv = dims
    q, k, v = case(B, S, L, H, Hkv, dk, dv, torch.bfloat16, seed=S + L, std=1.5)
    t = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    if lens is not None:
        for b, n in enumerate(lens):  # rows behind the length may hold anything
            k[b, :, n:] = float("nan")
            v[b, :, n:] = float("inf")
            v[b, :, n + 1:] = float("nan")
    scale = 1 / math.sqrt(dk)
    out = run(g, q, k, v, scale, t)
    assert g.attn_get_device_error() == g.OK
    verify(g, q, k, v, scale, t, out, True)
    assert torch.equal(out, run(g, q, k, v, scale, t, fill=0))  # the same bits again


@pytest.mark.parametrize("shape", [
    # dtype, B, S, L, H, Hkv, d, lens
    (torch.float32, 2, 7, 50, 4, 2, 16, [50, 0]),
    (torch.float32, 1, 33, 200, 8, 2, 64, None),
    (torch.float32, 3, 1, 5000, 4, 2, 128, [5000, 2049, 0]),
    (torch.bfloat16, 5, 1, 700, 4, 4, 64, [700, 0, 1, 256, 513]),
    (torch.bfloat16, 2, 2, 900, 8, 8, 128, [900, 31]),
    (torch.bfloat16, 2, 6, 60, 2, 1, 32, [60, 33]),
    (torch.bfloat16, 1, 1, 4100, 2, 1, 256, None),
])
def test_few_rows_and_other_types(gpu_lib, shape):
    g = gpu_lib
    dt, B, S, L, H, Hkv, d, lens = shape
    q, k, v = case(B, S, L, H, Hkv, d, d, dt, seed=L, std=1.5)
    t = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    if lens is not None:
        for b, n in enumerate(lens):
            k[b, :, n:] = float("nan")
            v[b, :, n:] = float("nan")
    scale = 1 / math.sqrt(d)
    out = run(g, q, k, v, scale, t)
    assert g.attn_get_device_error() == g.OK
    tc = dt == torch.bfloat16 and d in (64, 128) and S * H // Hkv >= TC_ROWS
    verify(g, q, k, v, scale, t, out, tc)
    assert torch.equal(out, run(g, q, k, v, scale, t, fill=0))


@pytest.mark.parametrize("dt,S", [(torch.bfloat16, 40), (torch.bfloat16, 1), (torch.float32, 9)])
def test_peaked_and_flat_scores(gpu_lib, dt, S):
    """Scores of hundreds (one key takes all), equal scores, and growing ones (the
    reference max moves in every tile)."""
    g = gpu_lib
    q, k, v = case(2, S, 900, 4, 2, 64, 64, dt, seed=4)
    k[0] *= 20
    k[1, 0] = k[1, 0, :1]
    k[1, 1] = k[1, 1, :1] * torch.linspace(-30, 30, 900, device=DEV)[:, None]
    out = run(g, q, k, v, 0.125)
    verify(g, q, k, v, 0.125, None, out, dt == torch.bfloat16 and S * 2 >= TC_ROWS)


@pytest.mark.parametrize("dt,S", [(torch.bfloat16, 40), (torch.bfloat16, 1), (torch.float32, 9)])
def test_nan_and_infinity_reach_their_rows(gpu_lib, dt, S):
    g = gpu_lib
    q, k, v = case(3, S, 300, 4, 2, 64, 64, dt)
    q[0, 0, 1, 5] = float("nan")        # one row, one head
    k[1, 1, 7, 3] = float("inf")        # every row of heads 2 and 3 of sequence 1
    v[2, 0, 299, 10] = float("nan")     # column 10 of heads 0 and 1 of sequence 2
    out = run(g, q, k, v, 0.125)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 0, 1] = True
    want[1, :, 2:] = True
    want[2, :, :2, 10] = True
    # a score of -infinity weighs zero: only rows whose own factor is positive are NaN
    neg = (q[1, :, 2:, 3] < 0)
    want[1, :, 2:][neg] = False
    assert torch.equal(bad, want)


def test_bad_lengths_give_zeros_and_an_error(gpu_lib):
    g = gpu_lib
    for dt, S in ((torch.bfloat16, 20), (torch.bfloat16, 1), (torch.float32, 5)):
        q, k, v = case(3, S, 200, 4, 2, 64, 64, dt)
        lens = torch.tensor([-1, 201, 200], dtype=torch.int32, device=DEV)
        out = run(g, q, k, v, 0.125, lens)
        assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
        assert (out[:2] == 0).all()
        verify(g, q[2:], k[2:], v[2:], 0.125, None, out[2:], dt == torch.bfloat16 and S * 2 >= TC_ROWS)


def test_one_row_is_the_decode(gpu_lib):
    """seq_q = 1: attn_decode_contig's operation over the same rows. Two heads a group run on
    the tensor cores, where each p_j is rounded to bf16, by 2^-8 of itself at most: that moves
    sum p_j v_j / sum p_j by 2^-8 sum p_j |v_j| / sum p_j, which the decode of |v| gives. Both
    stores round too."""
    g = gpu_lib
    q, k, v = case(4, 1, 1500, 4, 2, 128, 128, torch.bfloat16)
    lens = torch.tensor([1, 700, 1499, 1500], dtype=torch.int32, device=DEV)
    out = run(g, q, k, v, 0.1, lens)
    want = torch.empty(4, 4, 128, dtype=torch.bfloat16, device=DEV)
    g.attn_decode_contig(q[:, 0].contiguous(), k, v, lens, want, 0.1)
    size = torch.empty_like(want)
    g.attn_decode_contig(q[:, 0].contiguous(), k, v.abs(), lens, size, 0.1)
    allowed = 2.0 ** -7 * want.float().abs() + 2.0 ** -8 * (1 + 2.0 ** -7) ** 2 * size.float() + 1e-6
    assert bool(((out[:, 0].float() - want.float()).abs() <= allowed).all())


def test_graph_and_stream(gpu_lib):
    g = gpu_lib
    B, S, L, H, Hkv, d = 2, 20, 700, 8, 2, 64
    q, k, v = case(B, S, L, H, Hkv, d, d, torch.bfloat16)
    lens = torch.tensor([700, 333], dtype=torch.int32, device=DEV)
    ws = g.cross_workspace(B, S, H, Hkv, d, d, L)
    assert ws is not None
    out = torch.empty(B, S, H, d, dtype=torch.bfloat16, device=DEV)
    g.attn_cross(q, k, v, out, 0.125, kv_lens=lens, workspace=ws)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.attn_cross(q, k, v, out, 0.125, kv_lens=lens, workspace=ws)
    out.zero_()
    graph.replay()
    assert torch.equal(out, want)
    lens.fill_(10)
    graph.replay()
    verify(g, q, k, v, 0.125, lens, out, True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    lens2 = torch.tensor([700, 333], dtype=torch.int32, device=DEV)
    out2, ws2 = torch.empty_like(out), torch.empty_like(ws)
    torch.cuda.synchronize()
    g.attn_cross(q, k, v, out2, 0.125, kv_lens=lens2, workspace=ws2, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out2, want)


def test_workspace_refusals(gpu_lib):
    g = gpu_lib
    q, k, v = case(1, 20, 700, 8, 2, 64, 64, torch.bfloat16)
    with pytest.raises(g.GqaError) as e:
        run(g, q, k, v, 0.125, ws=None)
    assert e.value.status == g.ERR_WORKSPACE


def test_withheld_tile_is_reported(gpu_lib):
    """The bounded waits: a K tile that never comes ends in an error, and the next call is right."""
    g = gpu_lib
    q, k, v = case(1, 20, 700, 8, 2, 64, 64, torch.bfloat16)
    want = run(g, q, k, v, 0.125)
    torch.cuda.synchronize()
    g.gqa_debug_withhold_first_tile(1)
    try:
        run(g, q, k, v, 0.125)
        assert g.attn_get_device_error() == g.ERR_DEVICE_TIMEOUT
    finally:
        g.gqa_debug_withhold_first_tile(0)
    assert torch.equal(run(g, q, k, v, 0.125), want)
    assert g.attn_get_device_error() == g.OK
