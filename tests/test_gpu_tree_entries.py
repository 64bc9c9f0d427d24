"""Attention of drafted rows (GPU) over tables with entries that are no blocks."""
import pytest
import torch

from test_gpu_tree import BF16, F32, PATHS, case, run, verify

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
