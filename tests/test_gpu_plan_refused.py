"""The index arrays of a step that cannot serve a sequence, or whose numbers are out of range (GPU): the sequence that
has them keeps its blocks and its rows have no slot; every output of every sequence against the plain plan; whole
numbers, equal."""
import numpy as np
import pytest
import torch

from oracle import step as S
from test_gpu_plan_rows import case, run

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


def flagged(g):
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    assert g.attn_get_device_error() == g.OK


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("entry", [-1, 60, 1 << 30])
@pytest.mark.parametrize("at", [3, 5, 8])
def test_an_entry_given_back_that_is_no_block(gpu_lib, at, entry, same):
    """(a request behind a window, say, whose first entries are gone)"""
    g, c = gpu_lib, small()
    c["tables"][2, at] = entry
    got, _ = run(g, c, same=same)
    flagged(g)
    verify(c, got, [2])


@pytest.mark.parametrize("same", [False, True])
def test_a_finished_request_with_entries_that_are_gone(gpu_lib, same):
    g, c = gpu_lib, small()
    c["tables"][3, :4] = -1
    c["tables"][1, 8] = c["nb"]
    got, _ = run(g, c, same=same)
    flagged(g)
    verify(c, got, [1, 3])


@pytest.mark.parametrize("B,finished", [(257, 0.3), (1500, 0.6), (4000, 0.2), (3000, 0.8)])
def test_many_sequences_with_such_entries(gpu_lib, B, finished):
    """More rounds than one of lengths and of entries, more sequences that give back many than are noted, blocks wanting."""
    g = gpu_lib
    c = case(B, 500, 20, 16, seed=B, finished=finished, room=0.8, pad=5)
    r = np.random.default_rng(1)
    need = -(-(c["lens"] + c["new"]) // c["bs"])
    giving = np.flatnonzero(need < c["held"])
    bad = sorted(r.choice(giving, 9, replace=False).tolist()) + [int(giving[-1])]
    for b in bad:
        c["tables"][b, r.integers(need[b], c["held"][b])] = r.choice([-1, c["nb"], -(1 << 31)])
    got, _ = run(g, c)
    flagged(g)
    verify(c, got, sorted(set(bad)))


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("less", [1, 2, 21, 63])
def test_more_rows_than_there_is_room_for(gpu_lib, less, same):
    """The sequence that does not fit, and those behind it that have rows."""
    g, c = gpu_lib, small()
    total = int(c["new"].sum())
    c["N"] = total - less
    end = np.cumsum(c["new"])
    got, _ = run(g, c, same=same)
    flagged(g)
    verify(c, got, [b for b in range(7) if c["new"][b] and end[b] > c["N"]])


@pytest.mark.parametrize("same", [False, True])
def test_more_rows_than_a_mask_can_name(gpu_lib, same):
    g, c = gpu_lib, small()
    c["new"][2] = 70
    c["N"] = int(c["new"].sum()) + 1
    par = np.full(c["N"], -1)
    at = 0
    r = np.random.default_rng(2)
    for n in c["new"]:
        par[at + 1:at + n] = [r.integers(0, i) for i in range(1, n)]
        at += n
    got, _ = run(g, c, par, 1, same=same)
    flagged(g)
    verify(c, got, [2], par)


def test_a_parent_that_does_not_precede_its_row(gpu_lib):
    """It counts as hanging on the history, and those below it go by that."""
    g, c = gpu_lib, small()
    par = np.full(c["N"], -1)
    start = int(c["new"][:5].sum())
    par[start + 1:start + 40] = np.arange(39)
    for up in (7, 9, 39, -2, 1 << 30):
        given, meant = par.copy(), par.copy()
        given[start + 7], meant[start + 7] = up, -1
        got, _ = run(g, c, given, 1)
        flagged(g)
        verify(c, got, [], meant)


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("what", ["length", "rows", "many", "capacity", "held", "keep"])
def test_the_others_are_as_ever(gpu_lib, what, same):
    g, c = gpu_lib, small()
    c["keep"] = np.array([0, 8, 0, 2, 0, 1, 0])
    if what == "length":
        c["lens"][2] = -1
    elif what == "rows":
        c["new"][2] = -3
    elif what == "many":  # more than N by itself: no row behind it is in range
        c["new"][2] = 1 << 30
    elif what == "capacity":
        c["lens"][2] = 12 * 16 - 2
    elif what == "held":
        c["held"][2] = 13
    else:
        c["keep"][2] = 10
    got, _ = run(g, c, same=same)
    flagged(g)
    verify(c, got, [2, 4, 5, 6] if what == "many" else [2])


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


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("what", ["list", "rows"])
def test_rows_whose_block_is_none(gpu_lib, what, same):
    """A place of the list that holds no block, or an entry in use where rows would lie: just those rows have no slot."""
    g, c = gpu_lib, small(held=np.array([2, 7, 3, 0, 4, 1, 3]), free=6)
    c["free_list"][:6] = [x for x in range(c["nb"]) if x not in c["tables"]][:6]
    nb = c["nb"]
    if what == "list":
        c["free_list"][4] = nb  # sequence 4 takes it for the first of its two
    else:
        c["tables"][6, 2] = nb
    got, _ = run(g, c, same=same)
    flagged(g)
    tables, held, flist, left, missing, starts, pos, slots = S.plan(c["lens"], c["new"], c["tables"], c["held"], c["free_list"],
                                                                    c["free"], c["bs"], nb, c["N"])
    assert (slots >= nb * c["bs"]).sum() == (16 if what == "list" else 2)
    slots[slots >= nb * c["bs"]] = -1
    if what == "list":
        assert tables[4, 4] == nb
        tables[4, 4] = -1
    for x, y in zip(got, (tables, held, flist, [left, missing], starts, pos, slots)):
        np.testing.assert_array_equal(x, y)


def test_refused_and_captured(gpu_lib):
    """The same in a graph, replayed on other numbers: good ones, then bad ones again."""
    g, c = gpu_lib, small()
    first, (args, kw) = run(g, c)
    verify(c, first, [])
    assert g.attn_get_device_error() == g.OK
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.kv_plan_rows(*args, **kw)
    outs = (args[2], args[4], args[5], args[7], args[8], args[9], args[10])
    for bad in ([2], [], [2]):
        c = small()
        if bad:
            c["tables"][2, 4] = -1
        args[2].copy_(torch.tensor(c["tables"]))
        args[5].copy_(torch.tensor(c["free_list"]))
        graph.replay()
        torch.cuda.synchronize()
        verify(c, [x.cpu().numpy() for x in outs] + [None], bad)
        assert g.attn_get_device_error() == (g.ERR_DEVICE_BOUNDS if bad else g.OK)
