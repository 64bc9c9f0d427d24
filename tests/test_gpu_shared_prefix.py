"""Decode of sequences that share prefixes (GPU) against the fp64 oracle; the tolerance is
dense_bound.py's."""
import math

import numpy as np
import pytest
import torch

from dense_bound import excess
from margins import check
from oracle import rows as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def case(members, prefix_blocks, own, H, Hkv, dk, dv, bs=16, dt=torch.bfloat16, seed=1, alone=0, spare=1, std=1.5):
    """members[g] sequences behind prefix_blocks[g] shared blocks; own[b] rows of its own for
    each sequence (negative: that many rows of the prefix are not reached); `alone` sequences
    behind the last group share nothing. Unused slots of the pool hold NaN."""
    g = torch.Generator().manual_seed(seed)
    B = sum(members) + alone
    first, lens = [], []
    for n, p in list(zip(members, prefix_blocks)) + [(alone, 0)]:
        first += [p] * n
    lens = [first[b] * bs + own[b] for b in range(B)]
    need = [max(0, -(-lens[b] // bs) - first[b]) for b in range(B)]
    mbps = max(f + n for f, n in zip(first, need)) + spare
    nb = sum(prefix_blocks) + sum(need) + 2
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.full((B, mbps), -1, dtype=torch.int32)
    k = torch.full((nb, Hkv, bs, dk), float("nan")).to(dt)
    v = torch.full((nb, Hkv, bs, dv), float("nan")).to(dt)
    at = b = 0
    for n, p in list(zip(members, prefix_blocks)) + [(alone, 0)]:
        shared = perm[at:at + p]
        at += p
        for _ in range(n):
            tables[b, :p] = shared
            tables[b, p:p + need[b]] = perm[at:at + need[b]]
            at += need[b]
            for j in range(0, lens[b], bs):  # the rows that some sequence holds
                e, rows = int(tables[b, j // bs]), min(bs, lens[b] - j)
                new = torch.isnan(k[e, 0, :rows, 0])
                k[e, :, :rows][:, new] = torch.randn(Hkv, int(new.sum()), dk, generator=g).to(dt)
                v[e, :, :rows][:, new] = torch.randn(Hkv, int(new.sum()), dv, generator=g).to(dt)
            b += 1
    starts = [0] + list(np.cumsum(members))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(q=(torch.randn(B, H, dk, generator=g) * std).to(dt).to(DEV), k=k.to(DEV), v=v.to(DEV),
                tables=tables.to(DEV), lens=i32(lens), starts=i32(starts), shared=i32(list(prefix_blocks)), bs=bs)


def run(g, c, scale, fill=255, **arms):
    B, H, _ = c["q"].shape
    Hkv, dv = c["v"].shape[1], c["v"].shape[3]
    ws = g.shared_prefix_workspace(B, H, Hkv, dv, c["tables"].shape[1] * c["bs"], c["shared"].numel())
    ws.fill_(fill)
    out = torch.full((B, H, dv), float("nan"), dtype=c["q"].dtype, device=DEV)
    g.attn_decode_shared_prefix(c["q"], c["k"], c["v"], c["tables"], c["lens"], c["starts"], c["shared"], out, scale,
                                ws, **arms)
    return out


def rows_of(c, pool, b):
    n = int(c["lens"][b])
    blocks = c["tables"][b, :-(-n // c["bs"])].long()
    x = pool[blocks].double().cpu().numpy()
    return np.ascontiguousarray(x.transpose(1, 0, 2, 3)).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def verify(c, scale, out, tc=True, skip=(), **arms):
    worst = 0.0
    kw = {k: (v.double().cpu().numpy() if torch.is_tensor(v) else v) for k, v in arms.items()}
    kw["slopes"] = kw.pop("alibi_slopes", None)
    for b in range(c["q"].shape[0]):
        if b in skip:
            continue
        n = int(c["lens"][b])
        q = c["q"][b:b + 1].double().cpu().numpy()
        o = R.attend(q, rows_of(c, c["k"], b), rows_of(c, c["v"], b), scale, position=n - 1, **kw)
        worst = max(worst, excess(out[b:b + 1], o, c["q"].dtype == torch.bfloat16, tc, q.shape[-1], n,
                                  arms.get("softcap", 0.0)))
    check(worst, 1.0)


SHAPES = [
    # members, prefix blocks, own rows, H, Hkv, bs, alone
    ([2], [1], [1, 1], 1, 1, 8, 0),                                  # the least there is to share
    ([4], [8], [1, 16, 17, 100], 4, 2, 16, 0),                       # exactly one key tile
    ([3, 2], [9, 40], [5, 1, 30, 64, 2], 14, 2, 16, 2),              # groups of 7 heads, two prefixes, two alone
    ([2, 1, 3, 0, 2], [3, 5, 0, 4, 33], [1, 2, 3, 4, 5, 6, 7, 8], 8, 8, 32, 1),  # one member, no prefix, no member
    ([40], [20], [(7 * i) % 50 + 1 for i in range(40)], 8, 2, 64, 0),  # more rows than a tile
    ([5], [2], [0, -1, -60, -127, 3], 8, 1, 128, 0),                 # members that end in the prefix
    ([2], [70], [2500, 1], 2, 1, 8, 0),                              # own rows past a 2048-row split
    ([3], [300], [1, 2, 3], 130, 1, 16, 0),                          # more heads than a tile has rows
]


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=range(len(SHAPES)))
def test_shared_prefix(gpu_lib, dims, shape):
    g = gpu_lib
    members, prefix, own, H, Hkv, bs, alone = shape
    own = own + [9, 200][:alone]
    c = case(members, prefix, own, H, Hkv, *dims, bs=bs, alone=alone, seed=len(own) + bs)
    scale = 1 / math.sqrt(dims[0])
    out = run(g, c, scale)
    assert g.attn_get_device_error() == g.OK
    verify(c, scale, out)
    assert torch.equal(out, run(g, c, scale, fill=0))  # the same bits again


ARMS = [dict(window=5), dict(window=100), dict(window=400), dict(softcap=15.0), dict(sinks=True), dict(alibi_slopes=True),
        dict(window=300, softcap=20.0, sinks=True, alibi_slopes=True)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("arms", ARMS, ids=lambda a: "-".join(a) + str(a.get("window", "")))
def test_arms(gpu_lib, d, arms):
    g = gpu_lib
    H = 6
    a = dict(arms)
    if "sinks" in a:
        a["sinks"] = torch.linspace(-2, 5, H, device=DEV)
    if "alibi_slopes" in a:
        a["alibi_slopes"] = torch.tensor([2.0 ** -(h + 1) for h in range(H)], device=DEV)
    c = case([4, 3], [20, 9], [1, 90, 200, 7, 16, -20, 50, 33], H, 2, d, d, alone=1, seed=d)
    out = run(g, c, 0.11, **a)
    assert g.attn_get_device_error() == g.OK
    verify(c, 0.11, out, **a)


@pytest.mark.parametrize("how", ["f32", "odd block", "width", "wide", "narrow"])
def test_shapes_without_the_tensor_cores(gpu_lib, how):
    """Every sequence reads all of its rows."""
    g = gpu_lib
    dt = torch.float32 if how in ("f32", "narrow") else torch.bfloat16
    d = {"width": 32, "wide": 256, "narrow": 16}.get(how, 64)
    c = case([3, 2], [4, 2], [1, 20, 700, 9, 3], 4, 2, d, d, bs=12 if how == "odd block" else 16, dt=dt)
    for arms in ({}, dict(window=30, softcap=9.0)):
        out = run(g, c, 0.125, **arms)
        assert g.attn_get_device_error() == g.OK
        verify(c, 0.125, out, tc=False, **arms)


def test_no_groups_is_the_paged_decode(gpu_lib):
    g = gpu_lib
    c = case([3], [0], [40, 5, 2100], 4, 2, 64, 64)
    out = run(g, c, 0.125)  # a group without a prefix
    verify(c, 0.125, out)
    c["starts"], c["shared"] = c["starts"][:1], c["shared"][:0]
    assert torch.equal(run(g, c, 0.125), out)  # no group at all
    want = torch.empty_like(out)
    ws = g.decode_workspace(3, 4, 64, c["tables"].shape[1] * c["bs"])
    g.attn_decode_paged(c["q"], c["k"], c["v"], c["tables"], c["lens"], want, 0.125, workspace=ws)
    verify(c, 0.125, want, tc=False)


@pytest.mark.parametrize("H,Hkv,alone", [(2, 1, 400), (2, 2, 900), (10, 2, 500)])
def test_many_groups_and_sequences(gpu_lib, H, Hkv, alone):
    """More groups than the planner keeps in shared memory, more sequences than its threads,
    of which it takes 256 or 1024; rows enough that the parts of one are joined by one thread
    a column (the last)."""
    g = gpu_lib
    n = 150
    members = [(i % 4) * 3 for i in range(n)]
    B = sum(members)
    c = case(members, [i % 5 for i in range(n)], [1 + (i * 7) % 40 for i in range(B)] + [3] * alone, H, Hkv, 64, 64, bs=8,
             alone=alone, seed=9)
    out = run(g, c, 0.125)
    assert g.attn_get_device_error() == g.OK
    verify(c, 0.125, out)


def test_bad_groups_lengths_and_entries(gpu_lib):
    g = gpu_lib
    c = case([4], [10], [3, 20, 7, 1], 4, 2, 64, 64, spare=0)
    good = {k: v.clone() for k, v in c.items() if torch.is_tensor(v)}
    # groups out of order, past the batch, below it, a prefix longer than a table row: nothing
    # is shared, the result stands
    for starts, shared in (([0, 5], [10]), ([-1, 4], [10]), ([3, 1], [10]), ([0, 3, 1, 4], [2, 2, 2]), ([0, 4], [-1]),
                           ([0, 4], [c["tables"].shape[1] + 1])):
        c["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        c["shared"] = torch.tensor(shared, dtype=torch.int32, device=DEV)
        out = run(g, c, 0.125)
        assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
        verify(c, 0.125, out)
    c.update({k: v.clone() for k, v in good.items()})
    # lengths out of range: zeros for them alone
    c["lens"][1], c["lens"][3] = 0, c["tables"].shape[1] * c["bs"] + 1
    out = run(g, c, 0.125)
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    assert (out[1] == 0).all() and (out[3] == 0).all()
    verify(c, 0.125, out, skip=(1, 3))
    # a bad entry in the prefix: flagged, no read out of range (the group's results are unspecified)
    c.update({k: v.clone() for k, v in good.items()})
    for e in (-1, c["k"].shape[0], 2 ** 31 - 1):
        c["tables"][0, 4] = e
        run(g, c, 0.125)
        assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    # a bad entry among a sequence's own blocks: the others stand
    c.update({k: v.clone() for k, v in good.items()})
    c["tables"][1, 10] = c["k"].shape[0]
    out = run(g, c, 0.125)
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    c["tables"] = good["tables"]
    verify(c, 0.125, out, skip=(1,))


def test_nan_reaches_its_rows(gpu_lib):
    g = gpu_lib
    c = case([3], [20], [5, 9, 1], 4, 2, 64, 64)
    c["q"][1, 2, 7] = float("nan")
    out = run(g, c, 0.125)
    bad = torch.isnan(out).all(-1)
    assert bad.nonzero().tolist() == [[1, 2]] and int(torch.isnan(out).sum()) == 64


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_hold_no_number(gpu_lib, d):
    """Keys and values without a number reach the sequences that see them, and no other: a
    member that ends before them in the prefix, one whose window hides them, rows of the
    first block below the window."""
    g = gpu_lib
    bad = [float("nan"), float("inf"), -float("inf")]
    # behind the end of members 1 and 3, within the prefix
    c = case([4], [20], [5, -30, 40, -200], 4, 2, d, d)
    for i, x in enumerate(bad):
        c["v"][c["tables"][0, 18].item(), :, 3 + i], c["k"][c["tables"][0, 18].item(), :, 3 + i] = x, bad[0]
    out = run(g, c, 0.11)
    assert g.attn_get_device_error() == g.OK
    assert torch.isnan(out[[0, 2]]).all()
    verify(c, 0.11, out, skip=(0, 2))
    # windows: members of unequal lengths see the prefix from rows 20, 131, 133 and 320 (none) on
    c = case([4], [20], [0, 111, 113, 300], 4, 2, d, d)
    assert c["lens"].tolist() == [320, 431, 433, 620]
    for row, x in ((0, bad[0]), (19, bad[1]), (132, bad[0])):
        e = c["tables"][0, row // 16].item()
        c["v"][e, :, row % 16], c["k"][e, :, row % 16] = x, bad[0]
    out = run(g, c, 0.11, window=300)
    assert g.attn_get_device_error() == g.OK
    assert torch.isnan(out[[0, 1]]).all()  # row 132 is theirs
    verify(c, 0.11, out, skip=(0, 1), window=300)
    # rows 0 and 19 are hidden from all
    e = c["tables"][0, 132 // 16].item()
    c["v"][e, :, 132 % 16], c["k"][e, :, 132 % 16] = 0.25, 0.5
    out = run(g, c, 0.11, window=300)
    verify(c, 0.11, out, window=300)


def test_entries_that_a_member_no_longer_has(gpu_lib):
    """The shared entries come from a member that shares: not from one that ends before them,
    nor from one whose window has left them behind and whose blocks are gone."""
    g = gpu_lib
    c = case([4], [20], [-200, 5, 60, 16], 4, 2, 128, 128)
    c["tables"][0, -(-int(c["lens"][0]) // 16):] = -1
    out = run(g, c, 0.11)
    assert g.attn_get_device_error() == g.OK
    verify(c, 0.11, out)
    c = case([4], [20], [500, 5, 60, 16], 4, 2, 128, 128)
    keep = c["tables"].clone()
    c["tables"][0, :32] = -1  # rows below 820 - 300 = 520
    c["tables"][1:, :1] = -1  # rows below 325 - 300 = 25
    out = run(g, c, 0.11, window=300)
    assert g.attn_get_device_error() == g.OK
    c["tables"] = keep
    verify(c, 0.11, out, window=300)


def test_two_streams_at_once(gpu_lib):
    """Two calls in flight at once, each with a workspace of its own."""
    g = gpu_lib
    cs = [case([4, 3], [20, 9], [1, 90, 200, 7, 16, 20, 50], 8, 2, 128, 128, seed=s) for s in (1, 2)]
    want = [run(g, c, 0.11) for c in cs]
    torch.cuda.synchronize()
    outs, spaces, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c in cs:
        B, H, _ = c["q"].shape
        spaces.append(g.shared_prefix_workspace(B, H, 2, 128, c["tables"].shape[1] * c["bs"], 2))
        outs.append(torch.empty_like(want[0]))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, ws, out, st in zip(cs, spaces, outs, streams):
            g.attn_decode_shared_prefix(c["q"], c["k"], c["v"], c["tables"], c["lens"], c["starts"], c["shared"], out,
                                        0.11, ws, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert g.attn_get_device_error() == g.OK


def test_a_decode_loop_in_a_graph(gpu_lib):
    """Rows appended and attended step by step, as a server does, the step captured once and
    replayed; against the eager paged decode of the same history."""
    g = gpu_lib
    H, Hkv, d, bs, steps = 8, 2, 64, 16, 20
    c = case([3, 2], [9, 4], [1, 3, 15, 16, 2], H, Hkv, d, d, bs=bs, spare=3)
    B = 5
    # room for the rows to come: fresh blocks for every free entry of the tables
    extra = int((c["tables"] < 0).sum())
    nb = c["k"].shape[0]
    c["tables"][c["tables"] < 0] = torch.arange(nb, nb + extra, dtype=torch.int32, device=DEV)
    pad = torch.full((extra, Hkv, bs, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    kp, vp = torch.cat([c["k"], pad]), torch.cat([c["v"], pad])
    lens, starts = c["lens"].clone(), torch.arange(B + 1, dtype=torch.int32, device=DEV)
    qkv = torch.zeros(B, (H + 2 * Hkv) * d, dtype=torch.bfloat16, device=DEV)
    q = qkv[:, :H * d].unflatten(-1, (H, d))
    k = qkv[:, H * d:(H + Hkv) * d].unflatten(-1, (Hkv, d))
    v = qkv[:, (H + Hkv) * d:].unflatten(-1, (Hkv, d))
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    rope = g.rope_init(d, 1e6, layout="half")
    qo, out = torch.empty(B, H, d, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, d, dtype=torch.bfloat16, device=DEV)
    cap = c["tables"].shape[1] * bs
    ws = g.shared_prefix_workspace(B, H, Hkv, d, cap, 2)

    def step():
        g.kv_append_paged_rows(q, k, v, qo, kp, vp, c["tables"], starts, lens, lens, rope=rope, q_weight=w, k_weight=w)
        g.attn_decode_shared_prefix(qo, kp, vp, c["tables"], lens, c["starts"], c["shared"], out, 0.125, ws)

    gen = torch.Generator().manual_seed(3)
    qkv.copy_(torch.randn(qkv.shape, generator=gen))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ws2, want = g.decode_workspace(B, H, d, cap), torch.empty_like(out)
    for i in range(steps):
        qkv.copy_(torch.randn(qkv.shape, generator=gen))
        graph.replay()
        assert lens.tolist() == [n + 2 + i for n in c["lens"].tolist()]
        g.attn_decode_paged(qo, kp, vp, c["tables"], lens, want, 0.125, workspace=ws2)
        # both within the stores' rounding and the tensor cores' rounding of P, which averages
        # over the keys: 2^-8 of the values' own size (at most 5 here) bounds it
        assert float((out.float() - want.float()).abs().max()) <= 2.0 ** -8 * 5 + 2.0 ** -7 * float(want.abs().max())
    assert g.attn_get_device_error() == g.OK


def test_withheld_tile_is_reported(gpu_lib):
    g = gpu_lib
    c = case([3], [30], [5, 9, 1], 4, 2, 128, 128)
    want = run(g, c, 0.1)
    torch.cuda.synchronize()
    g.gqa_debug_withhold_first_tile(1)
    try:
        run(g, c, 0.1)
        assert g.attn_get_device_error() == g.ERR_DEVICE_TIMEOUT
    finally:
        g.gqa_debug_withhold_first_tile(0)
    assert torch.equal(run(g, c, 0.1), want)
    assert g.attn_get_device_error() == g.OK


def test_workspace_refusals(gpu_lib):
    g = gpu_lib
    c = case([2], [2], [1, 1], 2, 1, 64, 64)
    out = torch.empty(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    n = g.attn_decode_shared_prefix_workspace_bytes(2, 2, 1, 64, c["tables"].shape[1] * c["bs"], 1)
    for ws in (None, torch.empty(n - 1, dtype=torch.uint8, device=DEV)):
        with pytest.raises(g.GqaError) as e:
            g.attn_decode_shared_prefix(c["q"], c["k"], c["v"], c["tables"], c["lens"], c["starts"], c["shared"], out,
                                        0.125, ws)
        assert e.value.status == g.ERR_WORKSPACE
