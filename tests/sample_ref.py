"""Sampling under settings in 64 bits, from the definition: the kept tokens'
probabilities of a row and the token that a uniform draws, and the probability
rule on a chain. Logits are float64 arrays (of the bf16 or fp32 values)."""
import numpy as np


def distribution(z, T=1.0, k=0, p=1.0, m=0.0):
    """Probabilities of a row's tokens (zeros: none has a weight)."""
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    z[np.abs(z) < 2.0 ** -90] = 0.0
    top = z.max()
    if top == -np.inf:
        return np.zeros_like(z)
    if T == 0.0:
        T, k = 1.0, 1
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        w = np.where(z == np.inf, 1.0, 0.0) if top == np.inf else np.exp((z - top) / max(T, 2.0 ** -90))
    w[w < 2.0 ** -64] = 0.0
    order = np.lexsort((np.arange(len(z)), -z))
    s = w[order]
    s[s < m] = 0.0
    if k > 0:
        s[k:] = 0.0
    if p < 1.0:
        c = np.cumsum(s)
        n = int(np.searchsorted(c, p * c[-1], side="left")) + 1  # the fewest that reach it
        s[max(n, 1):] = 0.0
    out = np.zeros_like(w)
    out[order] = s
    return out / out.sum()


def pick(w, u):
    """The first index whose running sum exceeds u times the sum; -1 without weights."""
    c = np.cumsum(w)
    if not c[-1] > 0:
        return -1
    u = 0.0 if np.isnan(u) else min(max(float(u), 0.0), 1.0)
    at = int(np.searchsorted(c, u * c[-1], side="right"))
    return min(at, int(np.nonzero(w)[0][-1]))


def chain(draft, target, tokens, u, r, n, fd, ft):
    """One request: (acc_len, tokens). fd, ft: (T, k, p, m)."""
    L, V = draft.shape
    out = []
    for j in range(n + 1):
        p = distribution(target[j], *ft)
        if j == n:
            out.append(pick(p, r))
            break
        q = distribution(draft[j], *fd)
        x = int(tokens[j])
        ok = 0 <= x < V
        ratio = (min(1.0, p[x] / q[x]) if q[x] > 0 else 1.0) if ok else 0.0
        if not float(u[j]) < ratio:
            out.append(pick(np.maximum(p - q, 0.0), r))
            break
        out.append(x)
    return len(out), out + [-1] * (L + 1 - len(out))
