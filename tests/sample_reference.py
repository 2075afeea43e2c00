"""The draw of dllm_sample from its definition, in 64 bits (numpy).

``margin`` says how near u lies to where another token would be drawn, as a
share of the kept mass: the kernel's cumulative masses are good to about 2^-40
of the whole, so a test's inputs must keep a margin above that (they do by
many orders unless values tie exactly, which 64 bits and the kernel's whole
counts both hold exactly)."""
import numpy as np


def order_of(x):
    """Tokens by falling value, ties to the lowest token (-0 == +0)."""
    return np.argsort(-(x + 0.0), kind="stable")


def sample(x, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, prob, margin) of a row x (float64 values of bf16)."""
    x = np.asarray(x, dtype=np.float64)
    m = x.max() if len(x) else -np.inf
    if np.isnan(x).any() or not np.isfinite(m) or not T >= 0:
        return -1, float("nan"), 1.0
    at = order_of(x)
    if T == 0:
        return int(at[0]), 1.0, 1.0
    w = np.exp((x[at] - m) / T) if np.isfinite(T) else (x[at] > -np.inf).astype(np.float64)
    n = int((w > 0).sum())
    if top_k > 0:
        n = min(n, top_k)
    if min_p > 0:
        n = min(n, int((w >= min(min_p, 1.0)).sum()))
    c = np.cumsum(w[:n])
    margin = 1.0
    if top_p < 1:
        z = c[-1]
        k = int((c < top_p * z).sum())
        margin = min(margin, float(np.abs(c - top_p * z).min()) / z)
        n = min(n, k + 1)
    mass = c[n - 1]
    t = u * mass if u >= 0 else -1.0
    i = min(int((c[:n] <= t).sum()), n - 1)
    margin = min(margin, float(np.abs(c[:n] - t).min()) / mass)
    return int(at[i]), float(w[i] / mass), margin
