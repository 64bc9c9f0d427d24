"""Norm and rotation of query and key rows, and the ragged paged append (GPU),
against the fp64 oracle.

Tolerance, per element: the store's rounding (2^-8 of the value for bf16, 2^-24 for
fp32) plus the fp32 arithmetic's error, relative to the length of the element's pair:
the sum of squares (at most 16 fused terms in a lane and 5 butterfly steps, halved by the
square root), its four further operations, two products and three in the rotation make
at most 20 roundings of 2^-24; cos and sin are within 2 ulp (4 more) of an angle off by at
most 3e-7, and a frequency held to 2^-48 moves the angle at position p by p * 2^-48.
"""
import math

import numpy as np
import pytest
import torch

from margins import check
from oracle import rows as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
STORE = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def excess(got, want, size, dt, pos):
    """The largest error over its allowance."""
    far = (24 * 2.0 ** -24 + 3e-7) + np.abs(np.asarray(pos, np.float64))[..., None, None] * 2.0 ** -48
    err = np.abs(got.double().cpu().numpy() - want)
    # the allowance's last term keeps 0 / 0 out: subnormal results
    return float((err / (STORE[dt] * np.abs(want) + far * (1 + STORE[dt]) * size + 1e-37)).max())


def gen(seed):
    return torch.Generator().manual_seed(seed)


def packed(shape_heads, lead, d, dt, g):
    """q, k, v as slices of one projection's output, as a decoder layer has them."""
    widths = [h * d for h in shape_heads]
    x = (torch.randn(*lead, sum(widths), generator=g) * 1.3).to(dt).to(DEV)
    return [t.unflatten(-1, (h, d)) for t, h in zip(x.split(widths, -1), shape_heads)]


def weight(d, dt, g):
    return (1 + 0.2 * torch.randn(d, generator=g)).to(dt).to(DEV)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


ROPES = [  # (layout, rot_offset, rot_dim as a share of d, scaling)
    ("half", 0, 1.0, {}),
    ("interleaved", 0, 1.0, {}),
    ("half", 0, 0.5, dict(scaling="turns", factor=8.0, original_max=4096, low=1.0, high=4.0)),
    ("interleaved", 8, 0.5, dict(scaling="index", factor=4.0, original_max=4096, low=1.0, high=32.0)),
    ("half", 3, 0.25, dict(scaling="linear", factor=2.0)),   # pairs across chunks, an odd offset
    ("interleaved", 5, 0.25, {}),
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 16, 64, 72, 96, 128, 256])
@pytest.mark.parametrize("rope", ROPES, ids=lambda r: f"{r[0]}-{r[1]}-{r[2]}")
def test_norm_rope(gpu_lib, dt, d, rope):
    g = gpu_lib
    layout, off, share, scaling = rope
    rot = max(2, int(d * share) // 2 * 2)
    off = min(off, d - rot)
    gg = gen(d * 7 + rot + off)
    B, T, H, Hkv = 3, 5, 7, 2
    q, k, _ = packed([H, Hkv, Hkv], (B, T), d, dt, gg)
    wq, wk = weight(d, dt, gg), weight(d, dt, gg)
    pos = torch.tensor([0, 1, 4097, 131071, (1 << 24) + 5], dtype=torch.int32).repeat(B, 1).to(DEV)
    pos[1] = -pos[1]
    pos[2, 4] = (1 << 31) - 1
    r = g.rope_init(rot, 1e6, layout=layout, rot_offset=off, **scaling)
    qo, ko = torch.empty(B, T, H, d, dtype=dt, device=DEV), torch.empty(B, Hkv, T, d, dtype=dt, device=DEV)
    before = q.clone()
    g.attn_qk_norm_rope(q, k, qo, ko.transpose(1, 2), pos, r, q_weight=wq, k_weight=wk, eps=1e-5)
    assert torch.equal(q, before)
    w = R.frequencies(rot, 1e6, **scaling)
    p = pos.cpu().numpy()
    for got, x, wt in ((qo, q, wq), (ko.transpose(1, 2), k, wk)):
        want, size = R.rotate(R.norm(f64(x), f64(wt), 1e-5), p, w, layout, off, r.magnitude)
        check(excess(got, want, size, dt, p), 1.0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_parts_alone(gpu_lib, dt):
    """Norm of one of the two, rotation alone, norm alone, queries or keys alone, in place."""
    g = gpu_lib
    gg = gen(5)
    B, T, H, Hkv, d = 2, 3, 4, 2, 64
    q, k, v = packed([H, Hkv, Hkv], (B, T), d, dt, gg)
    wk = weight(d, dt, gg)
    pos = torch.arange(B * T, dtype=torch.int32, device=DEV).view(B, T) + 9
    r = g.rope_init(64, 1e4, layout="half")
    w, p = R.frequencies(64, 1e4), pos.cpu().numpy()
    q0, k0, v0 = f64(q), f64(k), v.clone()
    # keys normed, queries only turned; both in place in the packed buffer, whose values stay
    g.attn_qk_norm_rope(q, k, q, k, pos, r, k_weight=wk)
    want, size = R.rotate(q0, p, w, "half")
    check(excess(q, want, size, dt, p), 1.0, "queries, rotation alone")
    want, size = R.rotate(R.norm(k0, f64(wk), 1e-6), p, w, "half")
    check(excess(k, want, size, dt, p), 1.0, "keys, norm and rotation")
    assert torch.equal(v, v0)
    # norm alone, keys alone
    ko = torch.empty(B, T, Hkv, d, dtype=dt, device=DEV)
    k1 = f64(k)
    g.attn_qk_norm_rope(None, k, None, ko, None, None, k_weight=wk)
    want = R.norm(k1, f64(wk), 1e-6)
    check(excess(ko, want, np.abs(want), dt, 0 * p), 1.0, "norm alone")
    # neither: a copy
    g.attn_qk_norm_rope(q, None, (qo := torch.empty_like(q.contiguous())), None, None, None)
    assert torch.equal(qo, q)


def test_rows_of_zeros_and_special_values(gpu_lib):
    """A row of zeros stays zeros under the norm (eps keeps it finite); NaN and infinity
    stay in their own row, and outside their own pair without a norm."""
    g = gpu_lib
    for layout in ("half", "interleaved"):
        for dt in (torch.bfloat16, torch.float32):
            x = torch.randn(1, 4, 3, 64, generator=gen(1)).to(dt).to(DEV)
            x[0, 0] = 0
            x[0, 1, 1, 3] = float("nan")
            x[0, 2, 2, 60] = float("inf")
            y, z = torch.empty_like(x), torch.empty_like(x)
            pos = torch.arange(4, dtype=torch.int32, device=DEV)[None]
            r = g.rope_init(32, 1e4, layout=layout)
            w = torch.ones(64, dtype=dt, device=DEV)
            g.attn_qk_norm_rope(x, None, y, None, pos, r, q_weight=w)
            g.attn_qk_norm_rope(x, None, z, None, pos, r)
            assert (y[0, 0] == 0).all()
            bad = ~torch.isfinite(y).all(-1)
            assert bad.nonzero().tolist() == [[0, 1, 1], [0, 2, 2]]
            at = (~torch.isfinite(z)).nonzero().tolist()
            pair = [3, 19] if layout == "half" else [2, 3]
            assert at == [[0, 1, 1, pair[0]], [0, 1, 1, pair[1]], [0, 2, 2, 60]]


@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (64, 1, 32, 8), (1, 777, 14, 2), (2, 3001, 5, 1)])
def test_sizes(gpu_lib, shape):
    """One row to many: the number of items per token changes, the result does not."""
    g = gpu_lib
    B, T, H, Hkv = shape
    d, dt = 128, torch.bfloat16
    gg = gen(T)
    q, k, _ = packed([H, Hkv, Hkv], (B, T), d, dt, gg)
    wq, wk = weight(d, dt, gg), weight(d, dt, gg)
    pos = torch.randint(0, 1 << 20, (B, T), generator=gg, dtype=torch.int32).to(DEV)
    r = g.rope_init(128, 1e6, layout="half")
    qo, ko = torch.empty(B, T, H, d, dtype=dt, device=DEV), torch.empty(B, T, Hkv, d, dtype=dt, device=DEV)
    g.attn_qk_norm_rope(q, k, qo, ko, pos, r, q_weight=wq, k_weight=wk)
    w, p = R.frequencies(128, 1e6), pos.cpu().numpy()
    for got, x, wt in ((qo, q, wq), (ko, k, wk)):
        want, size = R.rotate(R.norm(f64(x), f64(wt), 1e-6), p, w, "half")
        check(excess(got, want, size, dt, p), 1.0)


@pytest.mark.parametrize("shape", [
    # type, tokens, H, Hkv, d, layout, rotated columns, offset: tokens side by side in a warp,
    # 8 (64 columns of bf16), 4 (128, or 64 of fp32), 2 (256); none a multiple of that
    (torch.bfloat16, 4867, 3, 1, 64, "half", 64, 0),
    (torch.bfloat16, 5003, 8, 2, 32, "half", 8, 4),
    (torch.bfloat16, 4865, 1, 1, 64, "interleaved", 32, 16),
    (torch.bfloat16, 2435, 8, 2, 128, "half", 64, 64),
    (torch.float32, 2433, 3, 2, 64, "interleaved", 64, 0),
    (torch.float32, 2439, 5, 1, 64, "half", 22, 3),
    (torch.bfloat16, 1217, 6, 1, 256, "half", 256, 0),
    (torch.bfloat16, 5001, 2, 1, 64, None, 0, 0),
], ids=str)
def test_many_tokens_of_few_rows(gpu_lib, shape):
    g = gpu_lib
    dt, T, H, Hkv, d, layout, rot, off = shape
    gg = gen(T)
    q, k, _ = packed([H, Hkv, Hkv], (1, T), d, dt, gg)
    wq, wk = weight(d, dt, gg), weight(d, dt, gg)
    pos = torch.randint(0, 1 << 20, (1, T), generator=gg, dtype=torch.int32).to(DEV)
    r = g.rope_init(rot, 1e6, layout=layout, rot_offset=off) if layout else None
    qo, ko = torch.empty(1, T, H, d, dtype=dt, device=DEV), torch.empty(1, T, Hkv, d, dtype=dt, device=DEV)
    g.attn_qk_norm_rope(q, k, qo, ko, pos, r, q_weight=wq, k_weight=wk)
    p = pos.cpu().numpy()
    for got, x, wt in ((qo, q, wq), (ko, k, wk)):
        want = R.norm(f64(x), f64(wt), 1e-6)
        size = np.abs(want)
        if layout:
            want, size = R.rotate(want, p, R.frequencies(rot, 1e6), layout, off)
        check(excess(got, want, size, dt, p), 1.0)
    # the same bits as a few tokens at a time
    for a, b in ((0, 5), (T - 700, T)):
        q2, k2 = torch.empty_like(qo[:, a:b]), torch.empty_like(ko[:, a:b])
        g.attn_qk_norm_rope(q[:, a:b], k[:, a:b], q2, k2, pos[:, a:b].contiguous(), r, q_weight=wq, k_weight=wk)
        assert torch.equal(q2, qo[:, a:b]) and torch.equal(k2, ko[:, a:b])


def test_same_bits_as_the_present_rotation(gpu_lib):
    """Adjacent pairs, no norm, no scaling: attn_rope_interleaved_qk's operation."""
    g = gpu_lib
    gg = gen(3)
    q = torch.randn(2, 50, 6, 64, generator=gg).to(torch.bfloat16).to(DEV)
    k = torch.randn(2, 50, 2, 64, generator=gg).to(torch.bfloat16).to(DEV)
    pos = torch.randint(0, 40000, (2, 50), generator=gg, dtype=torch.int32).to(DEV)
    qa, ka, qb, kb = q.clone(), k.clone(), q.clone(), k.clone()
    g.attn_rope_interleaved_qk(qa, ka, pos, 1e6)
    g.attn_qk_norm_rope(qb, kb, qb, kb, pos, g.rope_init(64, 1e6))
    assert torch.equal(qa, qb) and torch.equal(ka, kb)


# ---------------------------------------------------------------------------- append

def append_case(dt, counts, lens, H=6, Hkv=2, dk=64, dv=64, bs=16, pad=0, seed=1, spare_blocks=2):
    gg = gen(seed)
    B, N = len(counts), sum(counts) + pad
    need = [(n + c + bs - 1) // bs for n, c in zip(lens, counts)]
    mbps = max(need) + spare_blocks
    nb = sum(need) + 3
    perm = torch.randperm(nb, generator=gg).to(torch.int32)
    tables = torch.full((B, mbps), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = perm[at:at + n]
        at += n
    widths = [H * dk, Hkv * dk, Hkv * dv]
    x = (torch.randn(N, sum(widths), generator=gg) * 1.3).to(dt).to(DEV)
    q, k, v = x.split(widths, -1)
    c = dict(q=q.unflatten(-1, (H, dk)), k=k.unflatten(-1, (Hkv, dk)), v=v.unflatten(-1, (Hkv, dv)),
             tables=tables.to(DEV), starts=torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV),
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV), bs=bs, counts=counts, hist=lens,
             kp=torch.randn(nb, Hkv, bs, dk, generator=gg).to(dt).to(DEV),
             vp=torch.randn(nb, Hkv, bs, dv, generator=gg).to(dt).to(DEV),
             wq=weight(dk, dt, gg), wk=weight(dk, dt, gg))
    return c


def append_check(c, dt, qo, kp, vp, lens_out, w, layout, magnitude, old_q, norm=True, off=0):
    """q_out, pools and lengths against the oracle; every slot and row not written as it was."""
    want_k, want_v = f64(c["kp"]), c["vp"].clone()
    seen_k = np.zeros(want_k.shape, bool)
    at = 0
    for b, n in enumerate(c["counts"]):
        for i in range(n):
            p = c["hist"][b] + i
            want, size = R.rotate(R.norm(f64(c["q"][at]), f64(c["wq"]) if norm else None, 1e-6), p, w, layout, off,
                                  magnitude)
            assert excess(qo[at], want, size, dt, p) <= 1.0
            blk, s = int(c["tables"][b, p // c["bs"]]), p % c["bs"]
            want, size = R.rotate(R.norm(f64(c["k"][at]), f64(c["wk"]) if norm else None, 1e-6), p, w, layout, off,
                                  magnitude)
            assert excess(kp[blk, :, s], want, size, dt, p) <= 1.0
            seen_k[blk, :, s] = True
            want_v[blk, :, s] = c["v"][at]
            at += 1
    assert torch.equal(qo[at:], old_q[at:])  # rows of padding
    keep = torch.from_numpy(~seen_k).to(kp.device)
    assert torch.equal(kp[keep], c["kp"][keep])
    assert torch.equal(vp, want_v)
    assert lens_out.tolist() == [n + k for n, k in zip(c["hist"], c["counts"])]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [
    ([1, 1, 1], [0, 15, 16], {}),                      # a decode step, blocks starting and ending
    ([0, 5, 0, 17, 1, 0], [3, 14, 0, 31, 7, 9], dict(pad=6)),  # ragged, empty sequences, padding
    ([40], [0], dict(dk=128, dv=64, bs=8, H=3, Hkv=1)),  # one prompt, value width of its own
    ([2, 3], [100, 1], dict(dk=72, dv=24, bs=5)),       # odd widths, odd blocks
    ([33] * 40, list(range(40)), dict(H=2, Hkv=1, dk=32, dv=32)),  # more than one step of the search
])
def test_append_rows(gpu_lib, dt, shape):
    g = gpu_lib
    counts, lens, kw = shape
    c = append_case(dt, counts, lens, **kw)
    dk = c["q"].shape[-1]
    r = g.rope_init(dk, 1e6, layout="half")
    w = R.frequencies(dk, 1e6)
    old = torch.full(c["q"].shape, 7.0, dtype=dt, device=DEV)
    qo, kp, vp = old.clone(), c["kp"].clone(), c["vp"].clone()
    out = torch.full_like(c["lens"], -5)
    g.kv_append_paged_rows(c["q"], c["k"], c["v"], qo, kp, vp, c["tables"], c["starts"], c["lens"], out, rope=r,
                           q_weight=c["wq"], k_weight=c["wk"])
    assert g.attn_get_device_error() == g.OK
    append_check(c, dt, qo, kp, vp, out, w, "half", 1.0, old)
    # the lengths in place, keys alone: the same pools
    kp2, vp2, lens = c["kp"].clone(), c["vp"].clone(), c["lens"].clone()
    g.kv_append_paged_rows(None, c["k"], c["v"], None, kp2, vp2, c["tables"], c["starts"], lens, lens, rope=r,
                           k_weight=c["wk"])
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2) and torch.equal(lens, out)
    assert g.attn_get_device_error() == g.OK


@pytest.mark.parametrize("H,Hkv,dk,dv,B", [(3, 1, 64, 64, 9), (1, 1, 128, 64, 9), (2, 1, 64, 128, 70)])
def test_append_many_rows(gpu_lib, H, Hkv, dk, dv, B):
    """Many rows, several to a warp, sequences that start within one, empty ones, one that does
    not fit its table, padding: the same bits as sequence by sequence."""
    g = gpu_lib
    rng = np.random.default_rng(B)
    counts = [int(x) for x in rng.multinomial(10203, np.ones(B) / B)]
    counts[3] = 0
    lens = [int(x) for x in rng.integers(0, 40, B)]
    c = append_case(torch.bfloat16, counts, lens, H=H, Hkv=Hkv, dk=dk, dv=dv, pad=13, seed=B)
    c["tables"][5, lens[5] // c["bs"]] = -1  # sequence 5: its first new block is missing
    r = g.rope_init(dk, 1e6, layout="half")
    N = c["q"].shape[0]
    out = []
    for whole in (True, False):
        kp, vp, lens_out = c["kp"].clone(), c["vp"].clone(), torch.full_like(c["lens"], -7)
        qo = torch.full((N, H, dk), 9.0, dtype=torch.bfloat16, device=DEV)
        if whole:
            g.kv_append_paged_rows(c["q"], c["k"], c["v"], qo, kp, vp, c["tables"], c["starts"], c["lens"], lens_out,
                                   rope=r, q_weight=c["wq"], k_weight=c["wk"])
        for b in [] if whole else range(B):
            a, z = int(c["starts"][b]), int(c["starts"][b + 1])
            starts = torch.tensor([0, z - a], dtype=torch.int32, device=DEV)
            g.kv_append_paged_rows(c["q"][a:z], c["k"][a:z], c["v"][a:z], qo[a:z], kp, vp, c["tables"][b:b + 1], starts,
                                   c["lens"][b:b + 1], lens_out[b:b + 1], rope=r, q_weight=c["wq"], k_weight=c["wk"])
        assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
        out.append((kp, vp, lens_out, qo))
    a, z = int(c["starts"][5]), int(c["starts"][6])  # (its q rows are unspecified)
    out[0][3][a:z] = out[1][3][a:z] = 0
    for x, y in zip(*out):
        assert torch.equal(x, y)
    want = [n + k for n, k in zip(lens, counts)]
    want[5] = lens[5]
    assert out[0][2].tolist() == want
    assert bool((out[0][3][int(c["starts"][-1]):] == 9).all())


def test_append_one_row_matches_the_present_append(gpu_lib):
    g = gpu_lib
    c = append_case(torch.bfloat16, [1, 1, 1, 1], [5, 40, 0, 63])
    kp, vp, lens = c["kp"].clone(), c["vp"].clone(), c["lens"].clone()
    q = c["q"].contiguous().clone()
    g.kv_append_paged(q, c["k"].contiguous(), c["v"].contiguous(), kp, vp, c["tables"], lens, lens, 1e4)
    kp2, vp2, lens2, q2 = c["kp"].clone(), c["vp"].clone(), c["lens"].clone(), c["q"].contiguous().clone()
    g.kv_append_paged_rows(q2, c["k"], c["v"], q2, kp2, vp2, c["tables"], c["starts"], lens2, lens2,
                           rope=g.rope_init(64, 1e4))
    assert torch.equal(vp, vp2) and torch.equal(lens, lens2)
    # angles reduced in fp64 there, in fp32 here: a stored bf16 may fall on the neighbour
    for a, b in ((q, q2), (kp, kp2)):
        assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 1e-5).all())


def test_append_errors_skip_rows_and_keep_the_length(gpu_lib):
    g = gpu_lib
    dt = torch.bfloat16
    counts, lens = [2, 20, 3, 4], [1, 10, 4, 5]
    c = append_case(dt, counts, lens, spare_blocks=0)
    good = c["tables"].clone()
    c["tables"][1, 1] = 10 ** 6      # rows 16 .. 29 of sequence 1
    lens_in = c["lens"].clone()
    lens_in[2] = -1
    lens_in[3] = c["tables"].shape[1] * 16 - 2  # two rows past the capacity
    kp, vp, out = c["kp"].clone(), c["vp"].clone(), torch.zeros_like(lens_in)
    qo = torch.zeros_like(c["q"])
    c["tables"][3, -1] = good[3, 0]  # a valid block for its last rows
    g.kv_append_paged_rows(c["q"], c["k"], c["v"], qo, kp, vp, c["tables"], c["starts"], lens_in, out)
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    assert out.tolist() == [3, 10, -1, int(lens_in[3])]
    # what is written: sequence 0's rows, the good ones of 1 and of 3, nothing else
    want = c["vp"].clone()
    for b, ps in ((0, [1, 2]), (1, range(10, 16)), (3, [int(lens_in[3]), int(lens_in[3]) + 1])):
        for i, p in enumerate(ps):
            want[int(c["tables"][b, p // 16]), :, p % 16] = c["v"][int(c["starts"][b]) + i]
    assert torch.equal(vp, want)
    # starts out of order, below zero or past the buffer: flagged, lengths kept, nothing read out of range
    for starts in ([0, 5, 2, 9, 29], [-3, 2, 4, 6, 8], [0, 2, 4, 6, 10 ** 6]):
        out.zero_()
        bad = torch.tensor(starts, dtype=torch.int32, device=DEV)
        g.kv_append_paged_rows(c["q"], c["k"], c["v"], qo, kp, vp, good, bad, c["lens"], out)
        assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
        for b in range(4):
            n = starts[b + 1] - starts[b]
            fine = 0 <= starts[b] <= starts[b + 1] <= c["q"].shape[0] and lens[b] + n <= good.shape[1] * 16 and all(
                int(e) >= 0 for e in good[b, lens[b] // 16:(lens[b] + n + 15) // 16])
            assert int(out[b]) == lens[b] + (n if fine else 0)


def test_append_graph_replay_and_prefill(gpu_lib):
    """A chunk appended and attended in a captured graph, replayed on new rows: the same bits
    as the eager calls."""
    g = gpu_lib
    dt = torch.bfloat16
    B, S, H, Hkv, d, bs = 2, 24, 4, 2, 64, 16
    c = append_case(dt, [S] * B, [5, 30], H=H, Hkv=Hkv, dk=d, dv=d, bs=bs)
    r = g.rope_init(d, 1e6, layout="half")
    qo = torch.empty(B * S, H, d, dtype=dt, device=DEV)
    lens_out, out = torch.empty_like(c["lens"]), torch.empty(B, S, H, d, dtype=dt, device=DEV)
    kp, vp = c["kp"].clone(), c["vp"].clone()
    q, k, v = (c[n].contiguous().clone() for n in "qkv")

    def step():
        g.kv_append_paged_rows(q, k, v, qo, kp, vp, c["tables"], c["starts"], c["lens"], lens_out, rope=r,
                               q_weight=c["wq"], k_weight=c["wk"])
        g.attn_prefill_paged(qo.view(B, S, H, d), kp, vp, c["tables"], out, 0.125, position_offset=c["lens"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    q.copy_(torch.randn(q.shape, generator=gen(8)))
    k.copy_(torch.randn(k.shape, generator=gen(9)))
    graph.replay()
    got, got_kp = out.clone(), kp.clone()
    out.zero_()
    kp.copy_(c["kp"])
    step()
    assert torch.equal(out, got) and torch.equal(kp, got_kp)
    assert g.attn_get_device_error() == g.OK
    assert lens_out.tolist() == [5 + S, 30 + S]


def test_on_another_stream(gpu_lib):
    g = gpu_lib
    c = append_case(torch.bfloat16, [7, 9], [3, 4])
    r = g.rope_init(64, 1e6)
    res = []
    for st in (torch.cuda.current_stream(), torch.cuda.Stream()):
        qo, kp, vp, out = torch.zeros_like(c["q"]), c["kp"].clone(), c["vp"].clone(), torch.zeros_like(c["lens"])
        st.wait_stream(torch.cuda.current_stream())
        g.kv_append_paged_rows(c["q"], c["k"], c["v"], qo, kp, vp, c["tables"], c["starts"], c["lens"], out, rope=r,
                               stream=st)
        torch.cuda.current_stream().wait_stream(st)
        res.append((qo, kp, vp, out))
    assert all(torch.equal(a, b) for a, b in zip(*res))
