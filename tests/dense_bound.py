"""How far a result of the attentions without a causal rule may be from the fp64 oracle.

Per element, with A = sum_j w_j |v_j| and R = max_j scale * sum_i |q_i k_ji| (both from the
oracle), dk the width and n the number of keys:
* the store: 2^-8 of the value for bf16, 2^-24 for fp32;
* on the tensor cores the probabilities are rounded to bf16: 2^-8 A;
* a score is off by at most dk * 2^-22 * R (products exact, one fp32 step per addition; the
  tensor cores may drop a bit or two more), the exponential by 2^-20 with its argument's
  rounding, a capped score by 1e-6 of the cap: each moves a probability by as much, and
  the quotient of the two sums by twice that;
* the two sums of n terms: n * 2^-23.
"""
import numpy as np


def excess(got, oracle, bf16, tensor_cores, dk, n, softcap=0.0):
    """The largest error over its allowance."""
    out, size, reach = oracle
    err = np.abs(got.double().cpu().numpy() - out)
    p = 2 * (dk * 2.0 ** -22 * reach + 2.0 ** -20 + 1e-6 * softcap) + max(n, 1) * 2.0 ** -23
    if tensor_cores:
        p = p + 2.0 ** -8
    store = 2.0 ** -8 if bf16 else 2.0 ** -24
    tol = store * np.abs(out) + (1 + store) * p * size
    worst = (err / (tol + 1e-37)).max()
    return float("inf") if np.isnan(worst) else float(worst)
