"""Attention of drafted rows (GPU) with heads of 192 and 128 columns, which have their own kernels: the arms, masks, values
that rows do not see, a wait that runs out. The tolerance is dense_bound.py's."""
import numpy as np
import pytest
import torch

from dense_bound import excess
from margins import check
from oracle import step as S
from test_gpu_tree import ARMS, BF16, DEV, F32, case, rows_of, run, verify, verify_arms

pytestmark = pytest.mark.gpu
WIDE = (192, 128)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("arms", ARMS, ids=lambda a: "-".join(a) + str(a.get("window", "")))
def test_arms(gpu_lib, dt, arms):
    g = gpu_lib
    H = 6
    a = dict(arms)
    if "sinks" in a:
        a["sinks"] = torch.linspace(-2, 5, H, device=DEV)
    if "alibi_slopes" in a:
        a["alibi_slopes"] = torch.tensor([2.0 ** -(h + 1) for h in range(H)], device=DEV)
    for seen in (None, "chain"):
        c = case([20, 1, 66, 9], [150, 30, 513, 0], H, 2, *WIDE, dt=dt, seed=11, seen=seen)
        if "window" in a:
            for b, h in enumerate(c["hist"]):
                c["tables"][b, :max(0, h - a["window"] + 1) // c["bs"]] = -1
        out = run(g, c, 0.09, **a)
        assert g.attn_get_device_error() == g.OK
        verify_arms(c, 0.09, out, dt == BF16, a)
        assert torch.equal(out, run(g, c, 0.09, fill=0, **a))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_masks(gpu_lib, dt):
    g, r = gpu_lib, np.random.default_rng(3)
    rows, hist = [70, 5, 8], [50, 0, 300]
    seen = [set(np.nonzero(r.random(n) < 0.3)[0].tolist()) for n in rows for _ in range(n)]
    seen[0] = seen[70] = seen[76] = set()
    c = case(rows, hist, 4, 2, *WIDE, dt=dt, seen=seen, words=3)
    for window in (0, 1, 4, 40):
        out = run(g, c, 0.1, window=window)
        verify(c, 0.1, out, tc=dt == BF16, window=window)
        assert (out[70] == 0).all()  # no history, no bit
    assert g.attn_get_device_error() == g.OK


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("window", [0, 20])
def test_values_that_rows_do_not_see(gpu_lib, dt, window):
    """Written by a unit and joined, with an infinity or NaN in a drafted row of every seventh sequence."""
    g, r = gpu_lib, np.random.default_rng(192)
    rows, hist = r.integers(1, 13, 200).tolist(), r.integers(0, 60, 200).tolist()
    c = case(rows, hist, 8, 4, *WIDE, dt=dt, seed=7)
    bad = {b: int(r.integers(0, rows[b])) for b in range(0, 200, 7)}
    for b, j in bad.items():
        at = hist[b] + j
        c["v"][int(c["tables"][b, at // 16]), 2, at % 16, 3] = (float("nan"), float("inf"), -float("inf"))[b % 3]
    out = run(g, c, 0.1, window=window).double()
    assert g.attn_get_device_error() == g.OK
    worst = 0.0
    for b, n in enumerate(rows):
        s = slice(int(c["starts"][b]), int(c["starts"][b + 1]))
        o = S.attend(c["q"][s].double().cpu().numpy(), rows_of(c, c["k"], b), rows_of(c, c["v"], b), hist[b], c["seen"][s], 0.1, window=window)
        assert (np.isfinite(o[0]) == torch.isfinite(out[s]).cpu().numpy()).all()
        free = [i for i in range(n) if b not in bad or bad[b] not in c["seen"][s.start + i]]
        if free:
            worst = max(worst, excess(out[s][free], tuple(x[free] for x in o), dt == BF16, dt == BF16, 192, hist[b] + n))
    check(worst, 1.0)


def test_a_wait_that_runs_out(gpu_lib):
    """The test hook: the first K tile never comes; the call returns, says so, and the next one is right."""
    g = gpu_lib
    c = case([90, 7], [100, 400], 8, 2, *WIDE)
    want = run(g, c, 0.1)
    verify(c, 0.1, want)
    g.gqa_debug_withhold_first_tile(True)
    try:
        run(g, c, 0.1)
        assert g.attn_get_device_error() == g.ERR_DEVICE_TIMEOUT
    finally:
        g.gqa_debug_withhold_first_tile(False)
    assert torch.equal(run(g, c, 0.1), want)
    assert g.attn_get_device_error() == g.OK
