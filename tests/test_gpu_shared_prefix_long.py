"""A shared prefix of more than 2^20 key tiles (GPU): its table repeats three blocks, so that the
result is the softmax over 384 keys with the number of times that each is seen as a factor."""
import numpy as np
import pytest
import torch

from margins import check

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_a_prefix_of_134_million_keys(gpu_lib):
    g = gpu_lib
    B, H, Hkv, d, bs, n = 3, 4, 1, 64, 128, (1 << 20) + 5  # n blocks of 128 keys, a key tile each
    gen = torch.Generator().manual_seed(9)
    q = torch.randn(B, H, d, generator=gen).bfloat16()
    kp, vp = (torch.randn(3, Hkv, bs, d, generator=gen).bfloat16() for _ in range(2))
    tables = (torch.arange(n + 1, dtype=torch.int32) % 3).repeat(B, 1)
    own = np.array([1, 77, 128])
    lens = torch.tensor(n * bs + own, dtype=torch.int32)
    groups, shared = torch.tensor([0, B], dtype=torch.int32), torch.tensor([n], dtype=torch.int32)
    out = torch.empty(B, H, d, dtype=torch.bfloat16, device=DEV)
    ws = g.shared_prefix_workspace(B, H, Hkv, d, (n + 1) * bs, 1)
    g.attn_decode_shared_prefix(*(t.to(DEV) for t in (q, kp, vp, tables, lens, groups, shared)), out, 0.125, ws)
    assert g.attn_get_device_error() == g.OK

    k, v = (t.double().numpy().reshape(3 * bs, d) for t in (kp, vp))
    worst = 0.0
    for b in range(B):
        times = np.repeat(np.bincount(np.arange(n) % 3, minlength=3).astype(float), bs)
        times[n % 3 * bs:n % 3 * bs + own[b]] += 1
        s = 0.125 * (q[b].double().numpy() @ k.T)
        w = times * np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        want, size = w @ v, w @ np.abs(v)
        # the store and P in bf16: 2^-8 each; the sums: with one group on 304 slots a key range has
        # at most 2^20 / 152 < 2^13 tiles, each of which adds at most two fp32 steps of 2^-23 to the row
        # sum and to the output: 2 x 2^13 x 2 x 2^-23 = 2^-8 of the size; exponentials and scores far less
        err = np.abs(out[b].double().cpu().numpy() - want)
        worst = max(worst, (err / (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -16) * size)).max())
    check(worst, 1.0)
