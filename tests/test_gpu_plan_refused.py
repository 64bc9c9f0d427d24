"""The index arrays of a step that cannot serve a sequence (GPU): every output of every sequence against the plain plan;
whole numbers, equal."""
import numpy as np
import pytest

from oracle import step as S
from test_gpu_plan_rows import run

pytestmark = pytest.mark.gpu


def small(**kw):
    """Seven sequences: 0, 4 and 5 take a block or more, 1, 2 and 3 give some back, 6 has what it needs."""
    c = dict(lens=np.array([30, 100, 40, 0, 64, 10, 33]), new=np.array([5, 0, 3, 0, 20, 40, 2]), held=np.array([2, 9, 9, 6, 4, 1, 3]),
             bs=16, nb=60, free=3, keep=None)
    perm = np.random.default_rng(9).permutation(c["nb"])
    c["tables"] = np.full((7, 12), -1)
    at = 0
    for b, n in enumerate(c["held"]):
        c["tables"][b, :n] = perm[at:at + n]
        at += n
    c["free_list"] = np.full(c["nb"], -7)
    c["free_list"][:c["free"]] = perm[at:at + c["free"]]
    c["N"] = int(c["new"].sum()) + 3
    return dict(c, **kw)


def verify(c, got, bad, parents=None, words=1):
    """parents: with those out of range as -1."""
    want = S.plan(c["lens"], c["new"], c["tables"], c["held"], c["free_list"], c["free"], c["bs"], c["nb"], c["N"], c["keep"], bad)
    tables, held, flist, left, missing, starts, pos, slots = want
    if parents is not None:
        seen = S.ancestors(parents, starts)
        pos[:len(seen)] = np.repeat(c["lens"], np.maximum(c["new"], 0)) + np.array([len(s) - 1 for s in seen], np.int64)
        mask = np.zeros((c["N"], words), np.int64)
        mask[:len(seen)] = S.words([{j for j in s if j < 64 * words} for s in seen], words)
        np.testing.assert_array_equal(got[7], mask)
    for x, y in zip(got, (tables, held, flist, [left, missing], starts, pos, slots)):
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("same", [False, True])
def test_a_sequence_that_cannot_be_served_has_no_entries_behind_its_own(gpu_lib, same):
    """What it wanted and did not get is -1 in its row of the table, not a block of before that others hold by now."""
    g, c = gpu_lib, small(free=0)
    c["new"][0] = 150  # takes ten blocks, of fourteen that come back
    c["new"][4] = 100  # wants seven
    c["N"] = int(c["new"].sum())
    for b in range(7):  # (stale entries)
        c["tables"][b, c["held"][b]:] = np.arange(12 - c["held"][b]) + 5
    got, _ = run(g, c, same=same)
    assert g.attn_get_device_error() == g.OK
    assert got[3][1] > 0 and (got[0][4, 4:11] == -1).all() and got[0][4, 11] != -1
    verify(c, got, [])
