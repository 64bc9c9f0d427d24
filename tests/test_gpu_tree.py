"""Attention of drafted rows (GPU) against the fp64 oracle; the tolerance is dense_bound.py's."""
import math

import numpy as np
import pytest
import torch

from dense_bound import excess
from margins import check
from oracle import step as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def some_trees(rows, seed, near=9):
    """For each packed row the drafted rows that it sees: trees that hang on a row of the last `near`, or on the history."""
    r = np.random.default_rng(seed)
    par = []
    for n in rows:
        par += [-1 if i == 0 or r.random() < 0.1 else int(r.integers(max(0, i - near), i)) for i in range(n)]
    return S.ancestors(par, np.concatenate([[0], np.cumsum(rows)]))


def case(rows, hist, H, Hkv, dk, dv, bs=16, dt=BF16, seed=1, seen=None, lead=0, pad=0, spare=1, words=None, std=1.5):
    """Sequences of rows[b] drafted rows behind hist[b]; `lead` rows before the first sequence and `pad` behind the last
    are no sequence's. Unused slots of the pool hold NaN."""
    g = torch.Generator().manual_seed(seed)
    B, N = len(rows), lead + sum(rows) + pad
    lens = [h + n for h, n in zip(hist, rows)]
    need = [-(-x // bs) for x in lens]
    mbps, nb = max(need) + spare, sum(need) + 2
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.full((B, mbps), -1, dtype=torch.int32)
    k = torch.full((nb, Hkv, bs, dk), float("nan"))
    v = torch.full((nb, Hkv, bs, dv), float("nan"))
    at = 0
    for b in range(B):
        tables[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        for j in range(0, lens[b], bs):
            e, n = int(tables[b, j // bs]), min(bs, lens[b] - j)
            k[e, :, :n] = torch.randn(Hkv, n, dk, generator=g)
            v[e, :, :n] = torch.randn(Hkv, n, dv, generator=g)
    seen = some_trees(rows, seed) if seen is None else seen
    chain = seen == "chain"
    if chain:
        seen = [set(range(i + 1)) for n in rows for i in range(n)]
    words = words or max(1, -(-max(rows) // 64))
    mask = np.full((N, words), -1, np.int64)
    mask[lead:lead + sum(rows)] = S.words(seen, words)
    return dict(q=(torch.randn(N, H, dk, generator=g) * std).to(dt).to(DEV), k=k.to(dt).to(DEV), v=v.to(dt).to(DEV), tables=tables.to(DEV),
                hist=hist, rows=rows, lead=lead, seen=seen, mask=None if chain else torch.tensor(mask, device=DEV), bs=bs,
                starts=lead + np.concatenate([[0], np.cumsum(rows)]))


def workspace(g, c, more=0):
    N, H, dk = c["q"].shape
    Hkv, dv = c["v"].shape[1], c["v"].shape[3]
    return g.tree_workspace(N + more, len(c["rows"]) + more, max(c["rows"]) + more, H, Hkv, dk, dv,
                            (c["tables"].shape[1] + more) * c["bs"], c["q"].dtype)


def run(g, c, scale, fill=255, ws=None, max_rows=None, **arms):
    N, H, _ = c["q"].shape
    if ws is None:
        ws = workspace(g, c)
        ws.fill_(fill)
    out = torch.full((N, H, c["v"].shape[3]), 9.0, dtype=c["q"].dtype, device=DEV)
    g.attn_tree_paged(c["q"], c["k"], c["v"], c["tables"], i32(c["hist"]), i32(c["starts"]), c["mask"], out, scale,
                      max_rows or max(c["rows"]), ws, **arms)
    return out


def rows_of(c, pool, b):
    n = c["hist"][b] + c["rows"][b]
    x = pool[c["tables"][b, :-(-n // c["bs"])].long()].double().cpu().numpy()
    return np.ascontiguousarray(x.transpose(1, 0, 2, 3)).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def verify(c, scale, out, tc=True, skip=(), **arms):
    worst = 0.0
    kw = {k: (v.double().cpu().numpy() if torch.is_tensor(v) else v) for k, v in arms.items()}
    kw["slopes"] = kw.pop("alibi_slopes", None)
    for b, n in enumerate(c["rows"]):
        if b in skip or n == 0:
            continue
        s = slice(int(c["starts"][b]), int(c["starts"][b + 1]))
        seen = c["seen"][s.start - c["lead"]:s.stop - c["lead"]]
        o = S.attend(c["q"][s].double().cpu().numpy(), rows_of(c, c["k"], b), rows_of(c, c["v"], b), c["hist"][b], seen, scale, **kw)
        worst = max(worst, excess(out[s], o, c["q"].dtype == BF16, tc, c["q"].shape[-1], c["hist"][b] + n, arms.get("softcap", 0.0)))
    check(worst, 1.0)
    end = int(c["starts"][-1])
    assert (out[:c["lead"]] == 9.0).all() and (out[end:] == 9.0).all()  # no sequence's rows


SHAPES = [
    # rows, history, H, Hkv, bs
    ([1], [0], 1, 1, 8),                                       # the least there is
    ([1, 1, 1], [0, 1, 500], 8, 2, 16),                        # a step without a draft
    ([7, 0, 3], [100, 50, 0], 14, 2, 16),                      # groups of 7 heads, an idle sequence, no history
    ([5, 9], [127, 128], 4, 4, 32),                            # the history ends at a tile's edge, and before it
    ([40, 64, 1, 33], [129, 1000, 3, 2048], 8, 2, 16),         # more rows than a tile
    ([130, 2], [70, 300], 4, 4, 64),                           # three mask words, two row tiles of one head
    ([3], [2900], 2, 1, 128),                                  # few rows, keys over many CTAs
    ([6, 4], [40, 40], 130, 1, 8),                             # more heads than a tile has rows
    ([2] * 90, [3 * i for i in range(90)], 3, 3, 16),          # many sequences
    ([80, 150, 20, 0, 65], [900, 333, 50, 7, 0], 8, 2, 16),    # three and five row tiles, pairs and single ones
    ([700], [200], 2, 1, 32),                                  # eleven mask words
]


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128), (256, 256)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=range(len(SHAPES)))
def test_tensor_cores(gpu_lib, dims, shape):
    g = gpu_lib
    rows, hist, H, Hkv, bs = shape
    c = case(rows, hist, H, Hkv, *dims, bs=bs, seed=len(rows) + bs, lead=2, pad=3)
    scale = 1 / math.sqrt(dims[0])
    out = run(g, c, scale)
    assert g.attn_get_device_error() == g.OK
    verify(c, scale, out)
    assert torch.equal(out, run(g, c, scale, fill=0))  # the same bits again


@pytest.mark.parametrize("dt,dims,bs", [(F32, (16, 16), 16), (F32, (32, 32), 8), (F32, (64, 64), 16), (F32, (128, 128), 12),
                                        (F32, (192, 128), 16), (F32, (256, 256), 32), (BF16, (16, 16), 16), (BF16, (32, 32), 1),
                                        (BF16, (64, 64), 12), (BF16, (128, 128), 256), (BF16, (192, 128), 4), (BF16, (256, 256), 24)], ids=str)
@pytest.mark.parametrize("rows,hist,H,Hkv", [([5, 0, 1], [63, 9, 0], 6, 2), ([70, 9, 33], [130, 700, 64], 4, 1),
                                             ([3], [1500], 100, 1)])
def test_simt(gpu_lib, dt, dims, bs, rows, hist, H, Hkv):
    g = gpu_lib
    c = case(rows, hist, H, Hkv, *dims, bs=bs, dt=dt, seed=bs, lead=1, pad=2)
    scale = 1 / math.sqrt(dims[0])
    out = run(g, c, scale)
    assert g.attn_get_device_error() == g.OK
    verify(c, scale, out, tc=False)
    assert torch.equal(out, run(g, c, scale, fill=0))


PATHS = [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64)]


@pytest.mark.parametrize("dt,d", PATHS)
def test_a_scale_below_zero_and_of_zero(gpu_lib, dt, d):
    g = gpu_lib
    c = case([5, 9], [60, 200], 4, 2, d, d, dt=dt)
    for scale in (-0.1, 0.0):
        o = run(g, c, scale)
        assert g.attn_get_device_error() == g.OK
        worst = 0.0
        for b, n in enumerate(c["rows"]):
            s = slice(int(c["starts"][b]), int(c["starts"][b + 1]))
            want = S.attend(c["q"][s].double().cpu().numpy(), rows_of(c, c["k"], b), rows_of(c, c["v"], b), c["hist"][b], c["seen"][s], scale)
            want = (want[0], want[1], np.abs(want[2]))
            worst = max(worst, excess(o[s], want, dt == BF16, False, d, c["hist"][b] + n))
        check(worst, 1.0)


@pytest.mark.parametrize("dt,d", PATHS)
def test_masks(gpu_lib, dt, d):
    """A chain, rows that see nothing drafted or nothing at all, sets that are no trees, bits past the rows."""
    g = gpu_lib
    rows, hist = [70, 5, 8], [50, 0, 300]
    c = case(rows, hist, 4, 2, d, d, dt=dt, seen="chain")
    verify(c, 0.1, run(g, c, 0.1), tc=dt == BF16)
    r = np.random.default_rng(3)
    seen = [set(np.nonzero(r.random(n) < 0.3)[0].tolist()) for n in rows for _ in range(n)]
    seen[0] = seen[70] = seen[72] = seen[76] = set()
    seen[1] = set(range(70))
    c = case(rows, hist, 4, 2, d, d, dt=dt, seen=seen, words=3)
    for row, n in ((5, 70), (71, 5), (80, 8)):  # bits of rows that there are not
        for j in range(n, 192):
            if c["mask"][row, j // 64].item() >> (j % 64) & 1 == 0:
                c["mask"][row, j // 64] += -(1 << 63) if j % 64 == 63 else 1 << (j % 64)
    out = run(g, c, 0.1)
    verify(c, 0.1, out, tc=dt == BF16)
    assert (out[70] == 0).all() and (out[72] == 0).all()  # no history, no bit
    for window in (1, 4, 40):  # (a row that sees no drafted row stands where the first one does)
        verify(c, 0.1, run(g, c, 0.1, window=window), tc=dt == BF16, window=window)
    assert g.attn_get_device_error() == g.OK


ARMS = [dict(window=3), dict(window=40), dict(window=400), dict(softcap=15.0), dict(sinks=True), dict(alibi_slopes=True),
        dict(window=30, softcap=20.0, sinks=True), dict(window=100, softcap=20.0, sinks=True, alibi_slopes=True)]


@pytest.mark.parametrize("dt,d", PATHS)
@pytest.mark.parametrize("arms", ARMS, ids=lambda a: "-".join(a) + str(a.get("window", "")))
def test_arms(gpu_lib, dt, d, arms):
    g = gpu_lib
    H = 6
    a = dict(arms)
    if "sinks" in a:
        a["sinks"] = torch.linspace(-2, 5, H, device=DEV)
    if "alibi_slopes" in a:
        a["alibi_slopes"] = torch.tensor([2.0 ** -(h + 1) for h in range(H)], device=DEV)
    for seen in (None, "chain"):
        c = case([20, 1, 66, 9], [150, 30, 513, 0], H, 2, d, d, dt=dt, seed=d, seen=seen)
        if "window" in a:  # blocks that the window has left may be gone
            for b, h in enumerate(c["hist"]):
                c["tables"][b, :max(0, h - a["window"] + 1) // c["bs"]] = -1
        out = run(g, c, 0.11, **a)
        assert g.attn_get_device_error() == g.OK
        verify_arms(c, 0.11, out, dt == BF16, a)


def verify_arms(c, scale, out, tc, a):
    """verify(), with table entries that are gone read as block 0 (no row sees what lies there)."""
    keep = c["tables"]
    c["tables"] = keep.clamp(min=0)
    verify(c, scale, out, tc, **a)
    c["tables"] = keep


@pytest.mark.parametrize("dt,d", PATHS)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("of", ["k", "v"])
def test_what_a_row_does_not_see_does_not_reach_it(gpu_lib, dt, d, of, what):
    """A drafted row, and a history row that the window has left for some rows, hold no number."""
    g = gpu_lib
    c = case([30, 12], [100, 270], 4, 2, d, d, dt=dt, seed=5)
    holders = []
    for b, j in ((0, 4), (1, 7)):
        at = c["hist"][b] + j
        c[of][int(c["tables"][b, at // 16]), 1, at % 16, 3] = what
        holders.append(j)
    for window in (0, 64):
        out = run(g, c, 0.1, window=window).double()
        assert g.attn_get_device_error() == g.OK
        for b, n in enumerate(c["rows"]):
            s = slice(int(c["starts"][b]), int(c["starts"][b + 1]))
            seen = c["seen"][s]
            o = S.attend(c["q"][s].double().cpu().numpy(), rows_of(c, c["k"], b), rows_of(c, c["v"], b), c["hist"][b], seen, 0.1, window=window)
            free = [i for i in range(n) if holders[b] not in seen[i]]
            assert 0 < len(free) < n
            got = out[s][free]
            want = tuple(x[free] for x in o)
            check(excess(got, want, dt == BF16, dt == BF16, d, c["hist"][b] + n), 1.0)
            # the other KV head's rows are finite, and a row that sees an infinite value is not
            assert torch.isfinite(out[s][:, :2]).all()
            if of == "v":
                bound = [i for i in range(n) if i not in free]
                col = out[s][bound][:, 2:, 3]
                assert not torch.isfinite(col).any()
                assert torch.isfinite(out[s][bound][:, 2:, :3]).all()
    # a history row at the lower end of the window: hidden from the deep rows, seen by the first
    c = case([30], [200], 4, 2, d, d, dt=dt, seed=6, seen="chain")
    at = 200 - 50 + 1 + 4  # the window of 50: rows up to depth 5 see it
    c[of][int(c["tables"][0, at // 16]), 0, at % 16, 5] = what
    out = run(g, c, 0.1, window=50).double()
    o = S.attend(c["q"].double().cpu().numpy(), rows_of(c, c["k"], 0), rows_of(c, c["v"], 0), 200, c["seen"], 0.1, window=50)
    check(excess(out[5:], tuple(x[5:] for x in o), dt == BF16, dt == BF16, d, 230), 1.0)


@pytest.mark.parametrize("dt,d", PATHS)
def test_what_a_row_does_not_see_with_every_arm(gpu_lib, dt, d):
    """The rows worked out again have the arms too."""
    g = gpu_lib
    H = 4
    a = dict(window=90, softcap=20.0, sinks=torch.linspace(-1, 3, H, device=DEV),
             alibi_slopes=torch.tensor([2.0 ** -(h + 2) for h in range(H)], device=DEV))
    c = case([30, 12], [100, 270], H, 2, d, d, dt=dt, seed=5)
    for b, j in ((0, 4), (1, 7)):
        at = c["hist"][b] + j
        c["v"][int(c["tables"][b, at // 16]), :, at % 16, 3] = float("nan")
    out = run(g, c, 0.1, **a).double()
    kw = dict(window=90, softcap=20.0, sinks=a["sinks"].double().cpu().numpy(), slopes=a["alibi_slopes"].double().cpu().numpy())
    worst = 0.0
    for b, j in ((0, 4), (1, 7)):
        s = slice(int(c["starts"][b]), int(c["starts"][b + 1]))
        o = S.attend(c["q"][s].double().cpu().numpy(), rows_of(c, c["k"], b), rows_of(c, c["v"], b), c["hist"][b], c["seen"][s], 0.1, **kw)
        free = [i for i in range(c["rows"][b]) if j not in c["seen"][s.start + i]]
        worst = max(worst, excess(out[s][free], tuple(x[free] for x in o), dt == BF16, dt == BF16, d, c["hist"][b] + c["rows"][b], 20.0))
    check(worst, 1.0)


@pytest.mark.parametrize("dt,d", PATHS)
@pytest.mark.parametrize("window", [0, 20])
def test_the_same_where_a_unit_has_all_keys_of_its_rows(gpu_lib, dt, d, window):
    """More row tiles than the GPU takes at a time, so that most are written without a join."""
    g = gpu_lib
    r = np.random.default_rng(d)
    rows, hist = r.integers(1, 13, 200).tolist(), r.integers(0, 60, 200).tolist()
    c = case(rows, hist, 8, 4, d, d, dt=dt, seed=7)
    verify(c, 0.1, run(g, c, 0.1, window=window), tc=dt == BF16, window=window)
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
            worst = max(worst, excess(out[s][free], tuple(x[free] for x in o), dt == BF16, dt == BF16, d, hist[b] + n))
    check(worst, 1.0)


@pytest.mark.parametrize("dt,d", PATHS)
def test_scores_of_minus_infinity(gpu_lib, dt, d):
    """Keys that score -infinity weigh zero; a row of such keys alone gets zeros."""
    g = gpu_lib
    c = case([6, 6], [0, 40], 2, 1, d, d, dt=dt, seen=[{i} for i in range(6)] + [set(range(i + 1)) for i in range(6)])
    c["q"][:, :, 0] = 1.0
    for b, j in ((0, 2), (1, 41), (1, 3)):
        c["k"][int(c["tables"][b, j // 16]), 0, j % 16, 0] = -float("inf")
    out = run(g, c, 0.1)
    assert g.attn_get_device_error() == g.OK
    assert (out[2] == 0).all()
    verify(c, 0.1, out, tc=dt == BF16)


@pytest.mark.parametrize("dt,d", PATHS)
@pytest.mark.parametrize("what", ["negative", "long", "order", "many", "past", "entry"])
def test_bad_sequences(gpu_lib, dt, d, what):
    """Flagged; the others are as ever."""
    g = gpu_lib
    c = case([4, 9, 5], [60, 100, 30], 4, 2, d, d, dt=dt, lead=1, pad=2)
    good, max_rows, skip, left = dict(c), 9, {1}, slice(5, 14)
    if what == "negative":
        c["hist"] = [60, -1, 30]
    elif what == "long":
        c["hist"] = [60, c["tables"].shape[1] * 16 - 8, 30]
    elif what == "order":
        c["starts"] = np.array([1, 5, 3, 19])  # no sequence is taken
        skip, left = {0, 1, 2}, slice(0, 21)
    elif what == "many":
        max_rows = 8
    elif what == "past":
        c["starts"] = np.array([1, 5, 14, 22])
        skip, left = {2}, slice(14, 19)
    elif what == "entry":
        c["tables"] = c["tables"].clone()
        c["tables"][1, 2] = c["k"].shape[0]
        left = slice(0, 0)
    out = run(g, c, 0.1, ws=workspace(g, good), max_rows=max_rows)
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    assert g.attn_get_device_error() == g.OK
    verify(good, 0.1, out, tc=dt == BF16, skip=skip)
    assert (out[left] == 9.0).all()


@pytest.mark.parametrize("dt,d", PATHS)
def test_starts_that_go_back_and_forth(gpu_lib, dt, d):
    """Overlapping sequences, whose tiles would be more than the workspace has room for: nothing is written
    behind it."""
    g = gpu_lib
    c = case([100], [40], 4, 1, d, d, dt=dt)
    B, H = 40, 4
    starts = i32([0 if b % 2 == 0 else 100 for b in range(B + 1)])
    tables = c["tables"].expand(B, -1).contiguous()
    need = g.attn_tree_paged_workspace_bytes(100, B, 100, tables.shape[1] * 16, H, 1, d, d, dt)
    ws = torch.full((need + (1 << 22),), 77, dtype=torch.uint8, device=DEV)
    out = torch.full((100, H, d), 9.0, dtype=dt, device=DEV)
    g.attn_tree_paged(c["q"], c["k"], c["v"], tables, i32([40] * B), starts, c["mask"], out, 0.1, 100, ws[:need])
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    assert (out == 9.0).all() and (ws[need:] == 77).all()


def test_no_offsets_are_zeros(gpu_lib):
    g = gpu_lib
    c = case([9, 30], [0, 0], 4, 2, 128, 128)
    out = torch.empty(39, 4, 128, dtype=BF16, device=DEV)
    g.attn_tree_paged(c["q"], c["k"], c["v"], c["tables"], None, i32(c["starts"]), c["mask"], out, 0.1, 30, workspace(g, c))
    assert torch.equal(out, run(g, c, 0.1))


@pytest.mark.parametrize("long", [0, 75])
def test_more_sequences_than_a_launch_takes(gpu_lib, long):
    g = gpu_lib
    B = 2100
    r = np.random.default_rng(0)
    rows = r.integers(0, 3, B)
    rows[::400] = long or 1  # (more than a row tile: pairs in each launch)
    c = case(rows.tolist(), r.integers(0, 40, B).tolist(), 2, 1, 64, 64, pad=1)
    out = run(g, c, 0.1)
    assert g.attn_get_device_error() == g.OK
    verify(c, 0.1, out)


def test_no_rows_no_sequences(gpu_lib):
    g = gpu_lib
    c = case([3], [10], 2, 1, 64, 64)
    out = torch.full((3, 2, 64), 9.0, dtype=BF16, device=DEV)
    g.attn_tree_paged(c["q"], c["k"], c["v"], c["tables"], i32([10]), i32([0, 0]), c["mask"], out, 0.1, 3, workspace(g, c))
    g.attn_tree_paged(c["q"][:0], c["k"], c["v"], c["tables"], i32([10]), i32([0, 0]), c["mask"][:0], out[:0], 0.1, 3, None)
    g.attn_tree_paged(c["q"], c["k"], c["v"], c["tables"][:0], i32([]), i32([0]), c["mask"], out, 0.1, 3, None)
    assert g.attn_get_device_error() == g.OK
    assert (out == 9.0).all()


@pytest.mark.parametrize("dt,d", PATHS)
def test_captured_and_on_two_streams(gpu_lib, dt, d):
    """Graphs and streams with workspaces of their own; one workspace for calls of several sizes in a row."""
    g = gpu_lib
    big = case([20, 40], [300, 900], 8, 2, d, d, dt=dt, seed=1)
    small = case([1, 2, 3], [5, 0, 77], 8, 2, d, d, dt=dt, seed=2)
    want = [run(g, c, 0.1) for c in (big, small)]
    ws = workspace(g, big, more=5)
    for c, w in ((big, want[0]), (small, want[1]), (big, want[0])):
        assert torch.equal(run(g, c, 0.1, ws=ws), w)
    graphs = []
    for c in (big, small):
        gr, ws_c = torch.cuda.CUDAGraph(), workspace(g, c)
        out = torch.zeros_like(want[len(graphs)])
        hist, starts = i32(c["hist"]), i32(c["starts"])
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            g.attn_tree_paged(c["q"], c["k"], c["v"], c["tables"], hist, starts, c["mask"], out, 0.1, max(c["rows"]), ws_c)
        graphs.append((gr, out, ws_c, hist, starts))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (gr, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for (gr, out, *_), w in zip(graphs, want):
        assert torch.equal(out, w)
    assert g.attn_get_device_error() == g.OK


def test_rows_of_one_are_the_paged_decode(gpu_lib):
    """Up to the order of its sums and the rounding of the probabilities."""
    g = gpu_lib
    c = case([1] * 5, [0, 10, 300, 2500, 100], 8, 2, 128, 128)
    out = run(g, c, 0.1)
    other = torch.empty_like(out)
    lens = i32(np.array(c["hist"]) + 1)
    g.attn_decode_paged(c["q"], c["k"], c["v"], c["tables"], lens, other, 0.1, g.decode_workspace(5, 8, 128, c["tables"].shape[1] * 16))
    verify(c, 0.1, other, tc=False)
    verify(c, 0.1, out)


@pytest.mark.parametrize("rows", [[5, 9], [90, 70]])  # (the second: pairs)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_wait_that_runs_out(gpu_lib, rows, d):
    """The test hook: the first K tile never comes; the call returns, says so, and the next one is right."""
    g = gpu_lib
    c = case(rows, [100, 400], 8, 2, d, d)
    want = run(g, c, 0.1)
    g.gqa_debug_withhold_first_tile(True)
    try:
        run(g, c, 0.1)
        assert g.attn_get_device_error() == g.ERR_DEVICE_TIMEOUT
    finally:
        g.gqa_debug_withhold_first_tile(False)
    assert torch.equal(run(g, c, 0.1), want)
    assert g.attn_get_device_error() == g.OK
