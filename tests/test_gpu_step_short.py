"""A step for which blocks are wanting (GPU), through all four calls: the sequences that are served are as ever, and
nothing reads or writes blocks that a sequence had once and others hold by now."""
import numpy as np
import pytest
import torch

from dense_bound import excess
from margins import check
from oracle import step as S
from test_gpu_step import Program, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def forward(p, t, new, captured=None):
    """One step of chains of new[b] rows; returns the packed rows' starts."""
    starts = np.concatenate([[0], np.cumsum(new)])
    parents = np.full(p.N, -1)
    for b, n in enumerate(new):
        parents[starts[b]:starts[b] + n] = np.arange(n) - 1
    p.new.copy_(i32(new))
    p.parents.copy_(i32(parents))
    for x in range(len(p.k)):
        for tensor in (p.q[x], p.kn[x], p.vn[x]):
            tensor.copy_(torch.randn(tensor.shape, generator=t))
        p.out[x].fill_(9.0)
    if captured is None:
        p.forward()
    else:
        captured.replay()
    return starts


def accept(p, n, first=0):
    """Sequence b keeps rows first .. first + n[b] - 1 of its drafted ones."""
    path = np.full((p.B, p.most), -1)
    for b, k in enumerate(n):
        path[b, :k] = first + np.arange(k)
    p.path.copy_(i32(path))
    p.n_path.copy_(i32(n))
    p.accept()


def verify(p, starts, served):
    """The outputs of the sequences served, against attention over the rows that their tables name."""
    worst, table = 0.0, p.tables.cpu().numpy()
    for b in served:
        n, hist = int(starts[b + 1] - starts[b]), int(p.lens[b])
        if n == 0:
            continue
        s, at = slice(int(starts[b]), int(starts[b + 1])), np.arange(hist + n)
        assert (p.slots[s].cpu().numpy() == table[b, (hist + np.arange(n)) // p.bs] * p.bs + (hist + np.arange(n)) % p.bs).all()
        for x in range(len(p.k)):
            k, v = (y[table[b, at // p.bs], :, at % p.bs].double().cpu().numpy().transpose(1, 0, 2) for y in (p.k[x], p.v[x]))
            assert torch.equal(p.v[x][table[b, at[hist:] // p.bs], :, at[hist:] % p.bs], p.vn[x][s])
            o = S.attend(p.q_rot[x][s].double().cpu().numpy(), k, v, hist, [set(range(i + 1)) for i in range(n)], 0.1)
            tc = p.dt == torch.bfloat16
            worst = max(worst, excess(p.out[x][s], o, tc, tc, p.d, hist + n))
    check(worst, 1.0)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dt,H,Hkv,d", [(torch.bfloat16, 8, 2, 64), (torch.bfloat16, 4, 2, 128), (torch.float32, 4, 2, 32)])
def test_a_step_for_which_blocks_are_wanting(gpu_lib, dt, H, Hkv, d, captured):
    g = gpu_lib
    p = Program(g, 3, 2, H, Hkv, d, 16, 8, 8, dt, 64, 96)
    t = torch.Generator().manual_seed(d)
    graph = None
    if captured:
        p.forward()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.forward()
    # prompts of 2, 2 and 1 blocks; 0 and 1 idle, 2 drafts on two blocks more and keeps one row; its blocks go back
    # and the others take them
    for new, kept in (([24, 24, 10], [24, 24, 10]), ([0, 0, 24], [0, 0, 1]), ([24, 40, 1], [21, 36, 1])):
        starts = forward(p, t, new, graph)
        assert int(p.free[1]) == 0
        verify(p, starts, range(3))
        accept(p, kept)
        assert g.attn_get_device_error() == g.OK
    table = p.tables.cpu().numpy()
    assert int(p.free[0]) == 0 and p.blocks.tolist() == [3, 4, 1] and p.lens.tolist() == [45, 60, 12]
    # sequence 2 wants a block that there is not
    pools = [x.clone() for x in p.k + p.v]
    starts = forward(p, t, [3, 4, 20], graph)
    assert int(p.free[1]) == 1 and p.blocks.tolist() == [3, 4, 1]
    assert (p.slots[int(starts[2]):int(starts[3])] == -1).all()
    assert g.attn_get_device_error() == g.OK  # (a step that runs short is no error, in none of the calls)
    verify(p, starts, [0, 1])
    own = p.tables.cpu().numpy()[2, 0]
    for x, y in zip(p.k + p.v, pools):
        assert torch.equal(x[own].nan_to_num(), y[own].nan_to_num())
    # rows of it that are accepted all the same: flagged, nothing moves
    pools = [x.clone() for x in p.k + p.v]
    accept(p, [0, 0, 15], first=4)
    assert g.attn_get_device_error() == g.ERR_DEVICE_BOUNDS
    assert p.lens.tolist() == [45, 60, 12]
    for x, y in zip(p.k + p.v, pools):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())
    accept(p, [3, 4, 0])
    assert g.attn_get_device_error() == g.OK
    # request 0 is over, and sequence 2 is served
    p.lens[0] = 0
    starts = forward(p, t, [0, 0, 20], graph)
    assert g.attn_get_device_error() == g.OK and p.free.tolist() == [2, 0]
    verify(p, starts, [2])
    accept(p, [0, 0, 20])
    assert g.attn_get_device_error() == g.OK
    assert p.lens.tolist() == [0, 64, 32]
    assert p.tables[1].tolist()[:4] == table[1].tolist()[:4]
