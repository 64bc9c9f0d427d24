"""Frequencies of the scaled rotations (CPU): the library's host function against the
formulas in fp64, and its refusals."""
import math

import numpy as np
import pytest

from oracle import rows


@pytest.fixture(scope="module")
def g():
    from causal_gqa_attention_row_gb300 import build
    build.build()
    import causal_gqa_attention_row_gb300 as g
    g.load()
    return g


CASES = [
    dict(rot_dim=128, theta=1e6),
    dict(rot_dim=2, theta=1e4),
    dict(rot_dim=64, theta=1e4, scaling="linear", factor=4.0),
    dict(rot_dim=128, theta=5e5, scaling="turns", factor=8.0, original_max=8192, low=1.0, high=4.0),
    dict(rot_dim=128, theta=1e4, scaling="index", factor=16.0, original_max=4096, low=1.0, high=32.0),
    dict(rot_dim=16, theta=1e4, scaling="index", factor=2.0, original_max=64, low=1.0, high=32.0),
    dict(rot_dim=256, theta=1e6, scaling="none", divisors=[1.0 + 0.03 * t for t in range(128)]),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: f"{c.get('scaling', 'none')}-{c['rot_dim']}")
def test_frequencies(g, c):
    table, _ = g.rope_frequencies(**c)
    got = table.double().sum(1).numpy()
    want = rows.frequencies(**c)
    # a float pair holds a double to 2^-48; pow, and the blend of two terms, 4 ulp of a double
    assert np.all(np.abs(got - want) <= want * (2.0 ** -48 + 4 * 2.0 ** -52))


def test_magnitude(g):
    assert g.rope_frequencies(8, 1e4)[1] == 1.0
    kw = dict(factor=8.0, original_max=4096, low=1.0, high=32.0)
    assert g.rope_frequencies(8, 1e4, scaling="index", **kw)[1] == np.float32(0.1 * math.log(8.0) + 1.0)
    assert g.rope_frequencies(8, 1e4, scaling="index", magnitude=0.5, **kw)[1] == 0.5
    assert g.rope_frequencies(8, 1e4, scaling="turns", **kw)[1] == 1.0


@pytest.mark.parametrize("c", [
    dict(rot_dim=7, theta=1e4), dict(rot_dim=0, theta=1e4), dict(rot_dim=258, theta=1e4),
    dict(rot_dim=8, theta=0.0), dict(rot_dim=8, theta=float("nan")), dict(rot_dim=8, theta=float("inf")),
    dict(rot_dim=8, theta=1e4, scaling="linear", factor=0.0),
    dict(rot_dim=8, theta=1e4, scaling="turns", factor=2.0, original_max=0.0),
    dict(rot_dim=8, theta=1e4, scaling="turns", factor=2.0, original_max=64, low=4.0, high=4.0),
    dict(rot_dim=8, theta=1.0, scaling="index", factor=2.0, original_max=64, low=1.0, high=4.0),
    dict(rot_dim=8, theta=1e4, magnitude=float("inf")),
    dict(rot_dim=8, theta=1e4, divisors=[1.0, 0.0, 1.0, 1.0]),
])
def test_refusals(g, c):
    with pytest.raises(g.GqaError) as e:
        g.rope_frequencies(**c)
    assert e.value.status == g.ERR_INVALID_ARG
