"""Attention of drafted rows (GPU) over tables with entries that are no blocks, and over keys that score -infinity; the
tolerance is dense_bound.py's."""
import pytest
import torch

from dense_bound import excess
from margins import check
from oracle import step as S
from test_gpu_tree import BF16, DEV, F32, PATHS, case, rows_of, run, verify

pytestmark = pytest.mark.gpu
WIDE = (192, 128)
KINDS = [(dt, (d, d)) for dt, d in PATHS] + [(BF16, WIDE), (F32, WIDE)]


@pytest.mark.parametrize("dt,dims", KINDS, ids=str)
def test_drafted_rows_without_blocks(gpu_lib, dt, dims):
    """Entries below 0 behind the history are no error: the sequence's outputs mean nothing, the others are as ever. In
    front of it, or past the pool, they are."""
    g = gpu_lib
    c = case([40, 20, 70], [60, 100, 32], 4, 2, *dims, dt=dt, seed=3)
    want = run(g, c, 0.1)
    verify(c, 0.1, want, tc=dt == BF16)
    good = c["tables"].clone()
    end = int(c["starts"][1]), int(c["starts"][2])
    for entry, first, error in ((-1, 7, False), (-(1 << 31), 7, False), (-1, 6, True), (-1, 2, True), (c["k"].shape[0], 7, True)):
        c["tables"] = good.clone()
        c["tables"][0, 4:] = -1  # (60 rows of history lie in four blocks)
        c["tables"][1, first] = entry  # (100 in seven, of which the last has four of them)
        out = run(g, c, 0.1)
        assert g.attn_get_device_error() == (g.ERR_DEVICE_BOUNDS if error else g.OK)
        assert torch.equal(out[end[1]:], want[end[1]:])


@pytest.mark.parametrize("dt,dims", KINDS, ids=str)
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_values_of_keys_that_score_minus_infinity(gpu_lib, dt, dims, what):
    """Such a key weighs zero. What its value holds may reach a row that sees it, in that column alone; the other rows
    and columns are as without it."""
    g = gpu_lib
    rows, hist = [30, 12], [100, 290]
    for b, j in ((0, 7), (0, 104), (1, 200), (1, 295)):
        c = case(rows, hist, 4, 2, *dims, dt=dt, seed=5)
        c["q"][:, :, 0] = 1.0
        at = int(c["tables"][b, j // 16]), slice(None), j % 16
        c["k"][at][:, 0] = -float("inf")
        c["v"][at][:, 3] = what
        out = run(g, c, 0.1).double()
        assert g.attn_get_device_error() == g.OK
        c["v"][at][:, 3] = 0.0
        worst = 0.0
        for x, n in enumerate(rows):
            s = slice(int(c["starts"][x]), int(c["starts"][x + 1]))
            o = S.attend(c["q"][s].double().cpu().numpy(), rows_of(c, c["k"], x), rows_of(c, c["v"], x), hist[x], c["seen"][s], 0.1)
            sees = [i for i in range(n) if x == b and (j < hist[x] or j - hist[x] in c["seen"][s.start + i])]
            got = out[s].clone()
            for i in sees:
                col = got[i, :, 3]
                got[i, :, 3] = torch.where(torch.isfinite(col), col, torch.tensor(o[0][i, :, 3], device=DEV))
            worst = max(worst, excess(got, o, dt == BF16, dt == BF16, dims[0], hist[x] + n))
        check(worst, 1.0)


@pytest.mark.parametrize("dt,dims", KINDS, ids=str)
@pytest.mark.parametrize("many", [False, True])
def test_a_sequence_without_numbers(gpu_lib, dt, dims, many):
    """Queries, keys and values of a sequence's drafted rows, or its queries and drafted values, are NaN: its rows are
    NaN throughout, the others to the bit as they were. many: more row tiles than the GPU takes at a time."""
    g = gpu_lib
    rows, hist = ([30, 12, 9], [100, 290, 40]) if not many else ([5, 12, 9] * 70, [20, 60, 0] * 70)
    c = case(rows, hist, 4, 2, *dims, dt=dt, seed=8)
    want = run(g, c, 0.1)
    verify(c, 0.1, want, tc=dt == BF16)
    s, at = slice(int(c["starts"][1]), int(c["starts"][2])), hist[1] + torch.arange(rows[1], device=DEV)
    where = c["tables"][1].long()[at // c["bs"]], slice(None), at % c["bs"]
    c["q"][s] = float("nan")
    c["v"][where] = float("nan")
    for of in ("v", "k"):
        c[of][where] = float("nan")
        out = run(g, c, 0.1)
        assert g.attn_get_device_error() == g.OK
        assert torch.isnan(out[s]).all()
        assert torch.equal(out[:s.start], want[:s.start]) and torch.equal(out[s.stop:], want[s.stop:])
