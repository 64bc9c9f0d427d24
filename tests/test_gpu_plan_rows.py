"""The index arrays of a step (GPU) against a plain plan in Python; whole numbers, equal."""
import numpy as np
import pytest
import torch

from oracle import step as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def case(B, hist, rows, bs, seed, spare=3, room=1.0, finished=0.1, keep=False, pad=0):
    """Lengths up to hist, up to `rows` new rows; held blocks with some to spare; a list of `room` of the blocks wanted."""
    r = np.random.default_rng(seed)
    lens, new = r.integers(0, hist + 1, B), r.integers(0, rows + 1, B)
    held = -(-(lens + r.integers(0, 3 * bs, B) * (r.random(B) < 0.4)) // bs)
    over = r.random(B) < finished
    lens[over] = new[over] = 0
    need = -(-(lens + new) // bs)
    mbps = int(max(need.max(), held.max())) + spare
    nb = B * mbps + 5
    perm = r.permutation(nb)
    tables = np.full((B, mbps), -1)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = min(nb - at, int(np.maximum(need - held, 0).sum() * room))
    free_list = np.full(nb, -7)
    free_list[:free] = perm[at:at + free]
    c = dict(lens=lens, new=new, held=held, tables=tables, free_list=free_list, free=free, bs=bs, nb=nb, N=int(new.sum()) + pad)
    c["keep"] = np.minimum(held, r.integers(0, 4, B)) if keep else None
    return c


def trees(c, seed, roots=1):
    r = np.random.default_rng(seed)
    par = np.full(c["N"], -1)
    at = 0
    for n in c["new"]:
        for i in range(n):
            par[at + i] = -1 if i < roots else r.integers(max(0, i - 9), i)
        at += n
    return par


def run(g, c, parents=None, words=1, same=False, stream=None):
    tables, flist = i32(c["tables"]), i32(c["free_list"])
    held = i32(c["held"])
    free = i32([c["free"], 99])
    bout, fout = (held, free) if same else (torch.full_like(held, -9), torch.full_like(free, -9))
    N = c["N"]
    starts, pos = i32(np.full(len(c["lens"]) + 1, -9)), i32(np.full(N, -9))
    slots = torch.full((N,), -9, dtype=torch.int64, device=DEV)
    mask = None if parents is None else torch.full((N, words), -9, dtype=torch.int64, device=DEV)
    args = (i32(c["lens"]), i32(c["new"]), tables, held, bout, flist, free[:1] if not same else free, fout, starts, pos, slots, c["bs"])
    kw = dict(keep_blocks=None if c["keep"] is None else i32(c["keep"]), parents=None if parents is None else i32(parents),
              tree_mask=mask)
    torch.cuda.synchronize()
    g.kv_plan_rows(*args, stream=stream, **kw)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (tables, bout, flist, fout, starts, pos, slots)] + [None if mask is None else mask.cpu().numpy()], (args, kw)


def verify(c, got, parents=None, words=1):
    tables, held, flist, left, missing, starts, pos, slots = S.plan(c["lens"], c["new"], c["tables"], c["held"], c["free_list"],
                                                                    c["free"], c["bs"], c["nb"], c["N"], c["keep"])
    if parents is not None:
        seen = S.ancestors(parents, starts)
        base = np.repeat(c["lens"], c["new"])
        pos[:len(seen)] = base + np.array([len(s) - 1 for s in seen], np.int64)
        want = np.zeros((c["N"], words), np.int64)
        want[:len(seen)] = S.words(seen, words)
        np.testing.assert_array_equal(got[7], want)
    for x, y in zip(got, (tables, held, flist, [left, missing], starts, pos, slots)):
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("B,hist,rows,bs,kw", [
    (1, 0, 1, 16, dict(finished=0.0)),
    (1, 5000, 3000, 16, dict(finished=0.0)),                # one sequence, its rows in slices
    (3, 20, 1, 1, dict()),                                  # blocks of one row
    (7, 100, 40, 12, dict(pad=9)),                          # an odd block size, padding
    (64, 900, 70, 16, dict(keep=True, room=1.1)),
    (64, 900, 70, 16, dict(room=0.5)),                      # too few blocks
    (64, 900, 700, 128, dict(room=0.0, finished=0.6)),      # only what is given back
    (700, 300, 9, 8, dict(room=0.9, finished=0.3)),         # more sequences than CTAs
    (1500, 60, 3, 16, dict(finished=0.3, keep=True)),       # more than one round of the scan
    (300, 50, 0, 16, dict(finished=0.5)),                   # no rows: blocks only go back
])
def test_plan(gpu_lib, B, hist, rows, bs, kw, same):
    g = gpu_lib
    c = case(B, hist, rows, bs, seed=B + rows, **kw)
    got, _ = run(g, c, same=same)
    assert g.attn_get_device_error() == g.OK
    verify(c, got)


@pytest.mark.parametrize("B,rows,words,roots,pad", [(1, 1, 1, 1, 0), (5, 64, 1, 1, 3), (40, 30, 1, 4, 0), (3, 200, 4, 1, 7), (9, 65, 3, 65, 0)])
def test_trees(gpu_lib, B, rows, words, roots, pad):
    g = gpu_lib
    c = case(B, 333, rows, 16, seed=rows, finished=0.0, pad=pad)
    c["new"][0] = rows
    c = dict(c, N=int(c["new"].sum()) + pad)
    need = -(-(c["lens"] + c["new"]) // 16)
    c["free"] = min(c["nb"], int(np.maximum(need - c["held"], 0).sum()))
    if need.max() > c["tables"].shape[1]:
        c["tables"] = np.pad(c["tables"], ((0, 0), (0, int(need.max()) - c["tables"].shape[1])), constant_values=-1)
    used = {int(e) for b in range(B) for e in c["tables"][b, :c["held"][b]]}
    rest = [e for e in range(c["nb"]) if e not in used]
    c["free"] = min(c["free"], len(rest))
    c["free_list"][:c["free"]] = rest[:c["free"]]
    par = trees(c, 5, roots)
    got, _ = run(g, c, par, words)
    assert g.attn_get_device_error() == g.OK
    verify(c, got, par, words)


def test_a_step_without_rows(gpu_lib):
    """Blocks go back, trees of no rows and all."""
    g = gpu_lib
    c = case(20, 300, 0, 16, seed=2, finished=0.5)
    got, _ = run(g, c, np.zeros(0), 1)
    assert g.attn_get_device_error() == g.OK
    verify(c, got)


def test_chain_of_one_tree(gpu_lib):
    """Every row on the one before: the longest walk, every bit below a row's own."""
    g = gpu_lib
    c = case(2, 10, 0, 16, seed=1, finished=0.0)
    c["new"] = np.array([0, 300])
    c["N"] = 300
    need = -(-(c["lens"] + c["new"]) // 16)
    c["tables"] = np.pad(c["tables"], ((0, 0), (0, 30)), constant_values=-1)
    used = {int(e) for b in range(2) for e in c["tables"][b, :c["held"][b]]}
    c["nb"] += 40
    rest = [e for e in range(c["nb"]) if e not in used]
    c["free"] = int(np.maximum(need - c["held"], 0).sum())
    c["free_list"] = np.array(rest[:c["free"]] + [-7] * (c["nb"] - c["free"]))
    par = np.arange(300) - 1
    got, _ = run(g, c, par, 5)
    assert g.attn_get_device_error() == g.OK
    verify(c, got, par, 5)


def test_the_same_call_again_and_a_captured_one(gpu_lib):
    g = gpu_lib
    c = case(33, 700, 50, 16, seed=3, room=0.8, finished=0.4)
    par = trees(c, 2)
    first, (args, kw) = run(g, c, par)
    verify(c, first, par)
    outs = (args[2], args[4], args[5], args[7], args[8], args[9], args[10])
    g.kv_plan_rows(*args, **kw)
    for x, y in zip(outs, first):
        np.testing.assert_array_equal(x.cpu().numpy(), y)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        g.kv_plan_rows(*args, **kw)
    for x in outs[3:]:
        x.fill_(-5)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(outs, first):
        np.testing.assert_array_equal(x.cpu().numpy(), y)
    assert g.attn_get_device_error() == g.OK


def test_steps_in_a_row_lose_no_block(gpu_lib):
    """Twenty steps in place: requests come, grow, shrink and go; every block is in one table or on the list."""
    g = gpu_lib
    r = np.random.default_rng(8)
    B, bs, mbps, nb = 24, 16, 40, 300
    tables = i32(np.full((B, mbps), -1))
    flist, free, held = i32(r.permutation(nb)), i32([nb, 0]), i32(np.zeros(B))
    lens = np.zeros(B, np.int64)
    for _ in range(20):
        new = r.integers(0, 40, B)
        new[lens + new > mbps * bs] = 0
        N = int(new.sum())
        pos, slots, starts = i32(np.zeros(N)), torch.zeros(N, dtype=torch.int64, device=DEV), i32(np.zeros(B + 1))
        g.kv_plan_rows(i32(lens), i32(new), tables, held, held, flist, free, free, starts, pos, slots, bs)
        assert g.attn_get_device_error() == g.OK
        t, h, n = tables.cpu().numpy(), held.cpu().numpy(), int(free[0])
        all_blocks = [int(e) for b in range(B) for e in t[b, :h[b]]] + flist.cpu().numpy()[:n].tolist()
        assert sorted(all_blocks) == list(range(nb))
        real = slots[slots >= 0]
        assert real.unique().numel() == real.numel()
        served = np.array([(slots[starts[b]:starts[b + 1]] >= 0).all().item() for b in range(B)])
        lens = np.where(served, lens + r.integers(0, new + 1), lens)  # some of the rows are kept
        lens[r.random(B) < 0.15] = 0


@pytest.mark.parametrize("what", ["length", "rows", "capacity", "held", "keep", "count", "parent", "words", "entry", "N"])
def test_numbers_out_of_range(gpu_lib, what):
    """Flagged; the sequence that has them keeps its blocks, and the others are served."""
    g = gpu_lib
    c = case(6, 200, 20, 16, seed=4, finished=0.0, keep=True, pad=2)
    par, words, b = None, 1, 2
    c["new"][b] = 5
    if what in ("parent", "words"):
        c["new"][b] = 70 if what == "words" else 5
        c["N"] = int(c["new"].sum())
        par = trees(c, 1)
        if what == "parent":
            par[int(c["new"][:b].sum()) + 3] = 3
    c["N"] = int(c["new"].sum())
    if what == "length":
        c["lens"][b] = -1
    elif what == "rows":
        c["new"][b] = -3
        c["N"] = int(np.maximum(c["new"], 0).sum())
    elif what == "capacity":
        c["lens"][b] = c["tables"].shape[1] * 16 - 4
    elif what == "held":
        c["held"][b] = c["tables"].shape[1] + 1
    elif what == "keep":
        c["keep"][b] = c["held"][b] + 1
    elif what == "count":
        c["free"] = c["nb"] + 1
    elif what == "entry":
        c["lens"][b], c["held"][b] = 40, 3
        c["tables"][b, 2] = c["nb"]
    elif what == "N":
        c["N"] -= 1
    got, _ = run(g, c, par, words)
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    assert g.attn_get_device_error() == g.OK
    starts = np.concatenate([[0], np.cumsum(np.maximum(c["new"], 0))])
    np.testing.assert_array_equal(got[4], starts)
    if what in ("length", "capacity", "held", "keep"):
        assert got[1][b] == c["held"][b]
        assert (got[6][starts[b]:starts[b + 1]] == -1).all()
    if what in ("length", "capacity", "keep", "entry"):
        other = [x for x in range(6) if x != b]
        assert all((got[6][starts[x]:starts[x + 1]] >= 0).all() for x in other[:1])
