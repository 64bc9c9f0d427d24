"""Steps of speculative decoding as a program runs them (GPU): plan, append by slots, attention of the
drafted rows, commit, several steps in a row with the arrays in place; each step's attention against fp64
attention over a plain list of every sequence's rows, its cache against that list."""
import numpy as np
import pytest
import torch

from dense_bound import excess
from margins import check
from oracle import rows as R
from oracle import step as S
from test_gpu_qk_rows import excess as rows_excess

pytestmark = pytest.mark.gpu
DEV = "cuda"
THETA = 1e4


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Program:
    """What a serving program keeps: pools for each layer, tables, the free list, lengths."""

    def __init__(self, g, B, layers, H, Hkv, d, bs, mbps, nb, dt, most, N):
        self.g, self.B, self.H, self.Hkv, self.d, self.bs, self.most, self.N, self.dt = g, B, H, Hkv, d, bs, most, N, dt
        pool = lambda: [torch.full((nb, Hkv, bs, d), float("nan"), dtype=dt, device=DEV) for _ in range(layers)]  # noqa: E731
        self.k, self.v = pool(), pool()
        self.tables, self.blocks, self.lens = i32(np.full((B, mbps), -1)), i32(np.zeros(B)), i32(np.zeros(B))
        self.free_list, self.free = i32(np.random.default_rng(0).permutation(nb)), i32([nb, 0])
        self.starts, self.positions = i32(np.zeros(B + 1)), i32(np.zeros(N))
        self.slots = torch.zeros(N, dtype=torch.int64, device=DEV)
        self.mask = torch.zeros(N, (most + 63) // 64, dtype=torch.int64, device=DEV)
        self.new, self.parents = i32(np.zeros(B)), i32(np.zeros(N))
        self.path, self.n_path = i32(np.zeros((B, most))), i32(np.zeros(B))
        self.rope = g.rope_init(d, THETA, layout="half")
        self.ws = g.tree_workspace(N, B, most, H, Hkv, d, d, mbps * bs, dt)
        new = lambda h: [torch.zeros(N, h, d, dtype=dt, device=DEV) for _ in range(layers)]  # noqa: E731
        self.q, self.kn, self.vn = new(H), new(Hkv), new(Hkv)
        self.q_rot, self.out = new(H), new(H)

    def forward(self):
        g = self.g
        g.kv_plan_rows(self.lens, self.new, self.tables, self.blocks, self.blocks, self.free_list, self.free, self.free, self.starts,
                       self.positions, self.slots, self.bs, parents=self.parents, tree_mask=self.mask)
        for x in range(len(self.k)):
            g.kv_append_slots(self.q[x], self.kn[x], self.vn[x], self.q_rot[x], self.k[x], self.v[x], self.slots, self.positions, self.rope)
            g.attn_tree_paged(self.q_rot[x], self.k[x], self.v[x], self.tables, self.lens, self.starts, self.mask, self.out[x], 0.1,
                              self.most, self.ws)

    def accept(self):
        self.g.kv_commit_rows(self.k, self.v, self.tables, self.lens, self.starts, self.path, self.n_path, self.lens)


def accepted_paths(r, new, parents, starts):
    """For each sequence a way down its tree, and how many of it are kept."""
    out = []
    for b, n in enumerate(new):
        path, at = [], -1
        while True:
            below = [i for i in range(n) if parents[starts[b] + i] == at]
            if not below or (path and r.random() < 0.2):
                break
            at = int(r.choice(below))
            path.append(at)
        out.append(path)
    return out


@pytest.mark.parametrize("dt,H,Hkv,d,captured", [(torch.bfloat16, 8, 2, 64, False), (torch.bfloat16, 8, 2, 128, True),
                                                  (torch.float32, 4, 2, 32, False), (torch.bfloat16, 2, 1, 256, True)])
def test_steps(gpu_lib, dt, H, Hkv, d, captured):
    g, r = gpu_lib, np.random.default_rng(d)
    B, layers, bs, most, N = 5, 2, 16, 24, 100
    p = Program(g, B, layers, H, Hkv, d, bs, 20, 90, dt, most, N)
    freqs = R.frequencies(d, THETA)
    rows = [[[np.zeros((0, Hkv, d)), np.zeros((0, Hkv, d))] for _ in range(layers)] for _ in range(B)]  # each layer's keys and values
    t = torch.Generator().manual_seed(d)
    graph = None
    if captured:  # (a first step without rows: the calls' first use is outside the capture)
        p.forward()
        p.accept()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.forward()
    for step in range(7):
        new = r.integers(0, most + 1, B) if step else np.array([20, 1, 24, 0, 13])
        if step == 4:  # a request is over, its rows and blocks go
            rows[2] = [[np.zeros((0, Hkv, d)), np.zeros((0, Hkv, d))] for _ in range(layers)]
            p.lens[2] = 0
            new[2] = 0
        new = np.minimum(new, N // B)
        starts = np.concatenate([[0], np.cumsum(new)])
        parents = np.full(N, -1)
        for b in range(B):
            for i in range(1, new[b]):
                parents[starts[b] + i] = r.integers(max(0, i - 4), i) if step else i - 1  # (prompts first: chains)
        p.new.copy_(i32(new))
        p.parents.copy_(i32(parents))
        for x in range(layers):
            for tensor in (p.q[x], p.kn[x], p.vn[x]):
                tensor.copy_(torch.randn(tensor.shape, generator=t))
        if graph is not None:
            graph.replay()
        else:
            p.forward()
        assert g.attn_get_device_error() == g.OK
        assert int(p.free[1]) == 0 and (p.starts.cpu().numpy() == starts).all()
        seen = S.ancestors(parents, starts)
        worst = 0.0
        for b in range(B):
            n, s = int(new[b]), slice(int(starts[b]), int(starts[b + 1]))
            hist = len(rows[b][0][0])
            assert int(p.lens[b]) == hist
            at = np.array([hist + len(seen[i]) - 1 for i in range(s.start, s.stop)], np.int64)
            assert (p.positions[s].cpu().numpy() == at).all()
            for x in range(layers):
                if n == 0:
                    continue
                # the rows as they lie in the cache
                blk, row = p.slots[s] // bs, p.slots[s] % bs
                kc = p.k[x][blk, :, row].double().cpu().numpy()
                vc = p.v[x][blk, :, row].double().cpu().numpy()
                want, size = R.rotate(p.kn[x][s].double().cpu().numpy(), at, freqs, "half")
                check(rows_excess(p.k[x][blk, :, row], want, size, dt, at), 1.0)
                assert torch.equal(p.v[x][blk, :, row], p.vn[x][s])
                k = np.concatenate([rows[b][x][0], kc]).transpose(1, 0, 2)
                v = np.concatenate([rows[b][x][1], vc]).transpose(1, 0, 2)
                o = S.attend(p.q_rot[x][s].double().cpu().numpy(), k, v, hist, seen[s], 0.1)
                tc = dt == torch.bfloat16
                worst = max(worst, excess(p.out[x][s], o, tc, tc, d, hist + n))
        check(worst, 1.0, f"step {step}")
        paths = accepted_paths(r, new, parents, starts) if step else [list(range(n)) for n in new]
        path = np.full((B, most), -1)
        for b, x in enumerate(paths):
            path[b, :len(x)] = x
            for y in range(layers):
                for kind, pool in ((0, p.k[y]), (1, p.v[y])):
                    s = p.slots[int(starts[b]):int(starts[b + 1])][torch.tensor(x, dtype=torch.long, device=DEV)]
                    rows[b][y][kind] = np.concatenate([rows[b][y][kind], pool[s // bs, :, s % bs].double().cpu().numpy()])
        p.path.copy_(i32(path))
        p.n_path.copy_(i32([len(x) for x in paths]))
        p.accept()
        assert g.attn_get_device_error() == g.OK
        table = p.tables.cpu().numpy()
        for b in range(B):  # the cache holds the accepted rows, one behind the other
            n = len(rows[b][0][0])
            assert int(p.lens[b]) == n
            for y in range(layers):
                for kind, pool in ((0, p.k[y]), (1, p.v[y])):
                    at = np.arange(n)
                    have = pool[table[b, at // bs], :, at % bs].double().cpu().numpy() if n else np.zeros((0, Hkv, d))
                    np.testing.assert_array_equal(have, rows[b][y][kind])
