"""Accepted rows kept (GPU): copies of rows, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import step as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def case(B, layers, rows, Hkv, dk, dv, bs, dt, seed, hist=90, paths=None):
    r = np.random.default_rng(seed)
    lens, n = r.integers(0, hist + 1, B), r.integers(0, rows + 1, B)
    if paths is None:
        paths = [sorted(r.choice(n[b], r.integers(0, n[b] + 1), replace=False).tolist()) for b in range(B)]
    else:
        n[:] = rows
    mbps = -(-(hist + rows) // bs) + 1
    nb = B * mbps + 2
    tables = np.full((B, mbps), -1)
    perm = r.permutation(nb)
    for b in range(B):
        used = -(-(lens[b] + n[b]) // bs)
        tables[b, :used] = perm[b * mbps:b * mbps + used]
    t = torch.Generator().manual_seed(seed)
    most = max([1] + [len(p) for p in paths])
    path = np.full((B, most), -3)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    pool = lambda d: [torch.randn(nb, Hkv, bs, d, generator=t).to(dt).to(DEV) for _ in range(layers)]  # noqa: E731
    return dict(lens=lens, starts=np.concatenate([[4], 4 + np.cumsum(n)]), tables=tables, paths=paths, path=path, k=pool(dk),
                v=pool(dv) if dv else None)


def run(g, c, same=False):
    lens = i32(c["lens"])
    out = lens if same else torch.full_like(lens, -1)
    g.kv_commit_rows(c["k"], c["v"], i32(c["tables"]), lens, i32(c["starts"]), i32(c["path"]), i32([len(p) for p in c["paths"]]), out)
    return out.cpu().numpy()


def wanted(c, pool, skip=()):
    x = pool.double().cpu().numpy()
    for b, p in enumerate(c["paths"]):
        if b not in skip:
            x = S.commit(x, c["tables"][b], int(c["lens"][b]), p)
    return x


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("B,layers,rows,Hkv,dk,dv,bs,dt", [
    (1, 1, 1, 1, 16, 16, 16, torch.bfloat16),
    (5, 3, 20, 2, 64, 64, 16, torch.bfloat16),
    (4, 2, 300, 2, 128, 64, 8, torch.float32),      # paths longer than a stage
    (9, 70, 12, 1, 32, 32, 12, torch.bfloat16),     # more layers than a launch, an odd block size
    (3, 2, 40, 8, 256, 256, 64, torch.bfloat16),
    (3, 2, 40, 1, 576, 0, 16, torch.bfloat16),      # latent rows, no values
    (700, 1, 6, 3, 64, 64, 1, torch.float32),
])
def test_commit(gpu_lib, B, layers, rows, Hkv, dk, dv, bs, dt, same):
    g = gpu_lib
    c = case(B, layers, rows, Hkv, dk, dv, bs, dt, seed=rows)
    want = [wanted(c, x) for x in c["k"] + (c["v"] or [])]
    got = run(g, c, same)
    assert g.attn_get_device_error() == g.OK
    np.testing.assert_array_equal(got, c["lens"] + [len(p) for p in c["paths"]])
    for x, y in zip(c["k"] + (c["v"] or []), want):
        np.testing.assert_array_equal(x.double().cpu().numpy(), y)


def test_overlapping_moves(gpu_lib):
    """Rows that are moved from and moved to: each place is read before it is overwritten."""
    g = gpu_lib
    paths = [list(range(1, 40)), list(range(39)), [0, 2, 4, 6, 8, 10, 12, 14, 16, 18, 20], [39], [], [0, 1, 5, 6, 7, 8, 9, 10, 11, 12, 39]]
    c = case(6, 2, 40, 2, 64, 64, 16, torch.bfloat16, seed=2, paths=paths)
    want = [wanted(c, x) for x in c["k"] + c["v"]]
    run(g, c)
    for x, y in zip(c["k"] + c["v"], want):
        np.testing.assert_array_equal(x.double().cpu().numpy(), y)


def test_one_tensor_of_all_layers(gpu_lib):
    g = gpu_lib
    c = case(5, 3, 20, 2, 64, 32, 16, torch.bfloat16, seed=4)
    want = [wanted(c, x) for x in c["k"] + c["v"]]
    c["k"], c["v"] = torch.stack(c["k"]), torch.stack(c["v"])
    run(g, c)
    assert g.attn_get_device_error() == g.OK
    for x, y in zip([*c["k"], *c["v"]], want):
        np.testing.assert_array_equal(x.double().cpu().numpy(), y)
    with pytest.raises(ValueError):  # layers that do not lie one behind the other
        g.kv_commit_rows(c["k"][::2], None, i32(c["tables"]), i32(c["lens"]), i32(c["starts"]), i32(c["path"]), i32([0] * 5), i32([0] * 5))


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("what", ["order", "twice", "past", "below", "count", "length", "capacity", "entry", "starts"])
def test_bad_paths(gpu_lib, what, same):
    """Flagged; the sequence is left as it is, the others are served."""
    g = gpu_lib
    c = case(4, 2, 20, 2, 64, 64, 16, torch.bfloat16, seed=7, paths=[[0, 3, 5], [1, 4, 9], [2, 7], [6]])
    b = 1
    if what in ("order", "twice", "past", "below"):
        c["path"][b, :3] = {"order": [1, 9, 4], "twice": [1, 4, 4], "past": [1, 4, 20], "below": [-1, 4, 9]}[what]
    elif what == "count":
        c["paths"][b] = [1, 4, 9, 9]  # one more than path has room for
    elif what == "length":
        c["lens"][b] = -1
    elif what == "capacity":
        c["lens"][b] = c["tables"].shape[1] * 16 - 19
    elif what == "entry":
        c["tables"][b, (c["lens"][b] + 9) // 16] = len(c["k"][0])
    elif what == "starts":
        b = 3
        c["starts"][4] = c["starts"][3] - 1
    want = [wanted(c, x, skip=(b,)) for x in c["k"] + c["v"]]
    got = run(g, c, same)
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    n = [len(p) for p in c["paths"]]
    n[b] = 0
    np.testing.assert_array_equal(got, c["lens"] + n)
    for x, y in zip(c["k"] + c["v"], want):
        np.testing.assert_array_equal(x.double().cpu().numpy(), y)


def test_captured(gpu_lib):
    g = gpu_lib
    c = case(5, 3, 20, 2, 64, 64, 16, torch.bfloat16, seed=3)
    want = [wanted(c, x) for x in c["k"] + c["v"]]
    keep = [x.clone() for x in c["k"] + c["v"]]
    lens, args = i32(c["lens"]), (i32(c["starts"]), i32(c["path"]), i32([len(p) for p in c["paths"]]))
    tables, out = i32(c["tables"]), i32(c["lens"] * 0)
    g.kv_commit_rows(c["k"], c["v"], tables, lens, *args, out)  # (first use outside the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.kv_commit_rows(c["k"], c["v"], tables, lens, *args, out)
    for x, y in zip(c["k"] + c["v"], keep):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(c["k"] + c["v"], want):
        np.testing.assert_array_equal(x.double().cpu().numpy(), y)
