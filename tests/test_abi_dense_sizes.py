"""Sizes at the ends of what attn_decode_shared_prefix counts in 32 bits (CPU): refused before
any launch."""
import pytest

INV, WS = 1, 4
P = 16  # a non-null, 16-byte aligned stand-in: never dereferenced


@pytest.fixture(scope="module")
def g():
    from causal_gqa_attention_row_gb300 import build
    build.build()
    import causal_gqa_attention_row_gb300 as g
    g.load()
    return g


def shared(g, B, mbps, bs, size=1 << 50):
    return g.load().attn_decode_shared_prefix(P, P, P, P, P, P, P, P, B, 1, mbps, 50, bs, 8, 2, 64, 64, 0.1, 1, P, size,
                                              None, None)


@pytest.mark.parametrize("B,mbps,bs", [(256, (1 << 23) - 1, 128), (1 << 20, 1 << 16, 16)])
def test_more_key_tiles_than_32_bits_count(g, B, mbps, bs):
    assert B * (mbps * bs // 128 + 2) > 2 ** 31 - 1 and mbps * bs <= (2 ** 31 - 1) // 2
    assert shared(g, B, mbps, bs) == INV
