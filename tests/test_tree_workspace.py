"""attn_tree_paged_workspace_bytes against what the call asks for (CPU): the size for all rows that a table row can name is
enough, one byte less or the size for shorter tables is not."""
import random

import pytest
import torch

INV, WS = 1, 4
P = 16  # a non-null, aligned stand-in: never dereferenced
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    from causal_gqa_attention_row_gb300 import build
    build.build()
    import causal_gqa_attention_row_gb300 as g
    g.load()
    return g


def call(g, N, B, rows, mbps, bs, H, Hkv, dk, dv, dt, ws, size):
    return g.load().attn_tree_paged(P, P, P, P, P, P, None, P, N, B, rows, 0, mbps, 1000, bs, H, Hkv, dk, dv, 0.1, dt, ws, size,
                                    None, None)


@pytest.mark.parametrize("dt,dk,dv", [(BF16, 64, 64), (BF16, 192, 128), (BF16, 256, 256), (F32, 64, 64), (BF16, 32, 32)], ids=str)
def test_the_call_asks_for_the_size_of_its_tables(g, dt, dk, dv):
    """(a misaligned workspace of enough bytes is refused as misaligned, one that is too small as too small; both before
    any launch)"""
    r = random.Random(dk)
    for _ in range(300):
        H, Hkv = r.choice([(8, 2), (14, 2), (4, 4), (130, 1)])
        N, B, rows = r.randint(1, 3000), r.randint(1, 600), r.randint(1, 200)
        mbps, bs = r.randint(1, 300), r.choice([8, 16, 64, 128])
        size = g.attn_tree_paged_workspace_bytes(N, B, rows, mbps * bs, H, Hkv, dk, dv, dt)
        args = N, B, rows, mbps, bs, H, Hkv, dk, dv, 1 if dt == BF16 else 0
        assert call(g, *args, P + 8, size) == INV
        if dt == F32 or dk == 32:  # (on one kernel whatever the block size is)
            assert call(g, *args, P, size - 1) == WS


def test_a_size_for_shorter_tables_is_refused(g):
    """One sequence of 100 keys in a table of 256 blocks of 16: the table counts."""
    args = 1, 1, 1, 256, 16, 14, 2, 64, 64, 1
    short, whole = (g.attn_tree_paged_workspace_bytes(1, 1, 1, n, 14, 2, 64, 64, BF16) for n in (100, 4096))
    assert short < whole
    assert call(g, *args, P, short) == WS and call(g, *args, P + 8, whole) == INV
