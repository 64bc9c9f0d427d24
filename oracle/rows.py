"""fp64 oracle of the query/key row calls and of the attentions without a causal rule.

TEST INFRASTRUCTURE: see the package docstring. Plain numpy loops over heads and
sequences from the formulas, sharing no code with the kernels; arrays are float64.
"""
import math

import numpy as np


def frequencies(rot_dim, theta, scaling="none", factor=1.0, original_max=0.0, low=1.0, high=4.0, divisors=None):
    """Frequency of each pair: theta^(-2t / rot_dim) over its divisor, lowered by the scaling."""
    out = []
    for t in range(rot_dim // 2):
        w = theta ** (-2.0 * t / rot_dim)
        if divisors is not None:
            w = w / divisors[t]
        if scaling == "linear":
            w = w / factor
        elif scaling == "turns":
            n = original_max * w / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (n - low) / (high - low)))
            w = keep * w + (1.0 - keep) * w / factor
        elif scaling == "index":
            def place(turns):
                return rot_dim * math.log(original_max / (2.0 * math.pi * turns)) / (2.0 * math.log(theta))
            first, last = max(0, math.floor(place(high))), min(rot_dim - 1, math.ceil(place(low)))
            ramp = min(1.0, max(0.0, (t - first) / max(last - first, 0.001)))
            w = w * (1.0 - ramp) + w / factor * ramp
        out.append(w)
    return np.array(out)


def norm(x, weight, eps):
    """x [..., d] over its root mean square, times weight."""
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def rotate(x, positions, freqs, layout, rot_offset=0, magnitude=1.0):
    """x [..., heads, d], positions [...]: returns the rotated rows and, per element,
    the length of its pair times the magnitude (the scale of a rounding error), the
    element's own size outside the rotated slice."""
    out, size = x.copy(), np.abs(x)
    half = len(freqs)
    for t in range(half):
        i, j = (rot_offset + 2 * t, rot_offset + 2 * t + 1) if layout == "interleaved" else (rot_offset + t,
                                                                                             rot_offset + t + half)
        angle = np.asarray(positions, np.float64)[..., None] * freqs[t]
        a, b = x[..., i], x[..., j]
        out[..., i] = magnitude * (a * np.cos(angle) - b * np.sin(angle))
        out[..., j] = magnitude * (a * np.sin(angle) + b * np.cos(angle))
        size[..., i] = size[..., j] = magnitude * np.hypot(a, b)
    return out, size


def attend(q, k, v, scale, window=0, softcap=0.0, sinks=None, slopes=None, position=None):
    """q [S, H, dk], k [Hkv, n, dk], v [Hkv, n, dv] of one sequence, every row seeing every
    key (with a window or ALiBi slopes: all rows at `position`). No keys: zeros. Returns
    the output, and sum_j w_j |v_j| and the largest scale * sum_i |q_i k_ji| of each row:
    the sizes that the arithmetic's errors go by."""
    S, H, _ = q.shape
    first = max(0, position - window + 1) if window > 0 else 0  # the keys below take no part, whatever they hold
    k, v = k[:, first:], v[:, first:]
    n, dv = v.shape[1], v.shape[2]
    out, size, reach = np.zeros((S, H, dv)), np.zeros((S, H, dv)), np.zeros((S, H, 1))
    if n == 0:
        return out, size, reach
    G = H // k.shape[0]
    j = first + np.arange(n)
    for h in range(H):
        kh, vh = k[h // G], v[h // G]
        s = scale * (q[:, h] @ kh.T)
        reach[:, h, 0] = scale * (np.abs(q[:, h]) @ np.abs(kh).T).max(-1)
        if softcap > 0:
            s = softcap * np.tanh(s / softcap)
        if slopes is not None:
            s = s + slopes[h] * (j - position)
        m = s.max(-1, keepdims=True)
        if sinks is not None:
            m = np.maximum(m, sinks[h])
        w = np.exp(s - m)
        den = w.sum(-1, keepdims=True) + (0.0 if sinks is None else np.exp(sinks[h] - m))
        out[:, h] = w @ vh / den
        size[:, h] = w @ np.abs(vh) / den
    return out, size, reach
