"""The calls over many sequences in numpy float64: trees, append, attention, acceptance, adapters."""
import numpy as np


def half_step(kind):
    """Largest relative error of one rounding to the type."""
    return 2.0 ** -8 if kind == "bf16" else 2.0 ** -11


def random_tree(rng, n, roots=1):
    """Parents: `roots` nodes under the cache, the others under any node before them, recent ones more often."""
    return np.array([-1 if i < roots else int(i - 1 - min(i - 1, rng.geometric(0.3) - 1)) for i in range(n)], np.int32)


def chain(n):
    return np.arange(-1, n - 1, dtype=np.int32)


def ancestors(parent):
    """[n, n]: node j is node i or lies before it."""
    see = np.eye(len(parent), dtype=bool)
    for i, p in enumerate(parent):
        if p >= 0:
            see[i] |= see[p]
    return see


def depths(parent):
    return ancestors(parent).sum(1) - 1


def append(qkv, nq, nkv, hd, qn, kn, eps, theta, positions):
    """(q [n, nq, hd], k [n, nkv, hd], v, size [n, nq + nkv, hd]): size bounds the two products of a rotated element."""
    x = qkv.astype(np.float64).reshape(len(qkv), nq + 2 * nkv, hd)
    qk = x[:, :nq + nkv]
    if qn is not None:
        w = np.concatenate([np.broadcast_to(qn, (nq, hd)), np.broadcast_to(kn, (nkv, hd))]).astype(np.float64)
        qk = qk / np.sqrt((qk * qk).mean(-1, keepdims=True) + eps) * w
    ang = positions[:, None, None] * theta ** (-np.arange(0, hd, 2) / hd)
    a, b = qk[..., :hd // 2], qk[..., hd // 2:]
    y = np.concatenate([a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)], -1)
    size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    return y[:, :nq], y[:, nq:], x[:, nq + nkv:], size


def attention(q, k, v, start, parent, weights):
    """(out [n, nq, hd], bound): q [n, nq, hd] over k, v [nkv, start + n, hd]. The bound on a result in f16: half a
    step of the output; `weights`, the weights' own rounding; a score's error d from the f32 sums of hd products and
    its scaling, which changes a weight and the weights' sum by a factor 1 + d each; f32 sums over the keys; the
    exponential's 2^-21."""
    n, nq, hd = q.shape
    nkv, length = k.shape[:2]
    see = np.ones((n, length), bool)
    see[:, start:] = ancestors(parent)
    out, bound = np.zeros((n, nq, hd)), np.zeros((n, nq, hd))
    for h in range(nq):
        kk, vv = k[h // (nq // nkv)], v[h // (nq // nkv)]
        s = q[:, h] @ kk.T / np.sqrt(hd)
        s = np.where(see, s, -np.inf)
        e = np.exp(s - s.max(1, keepdims=True))
        p = e / e.sum(1, keepdims=True)
        out[:, h] = p @ vv
        size = np.where(see, np.abs(q[:, h]) @ np.abs(kk).T / np.sqrt(hd), 0).max(1, keepdims=True)
        d = (hd + 4) * 2.0 ** -24 * size
        bound[:, h] = 2.0 ** -11 * np.abs(out[:, h]) + 2.0 ** -25 + (weights + 2 * d + (length + 64) * 2.0 ** -24 + 2.0 ** -20) * (p @ np.abs(vv))
    return out, bound


def accept(parent, tokens, ids, root):
    """(accepted nodes, the wanted token that no node has)."""
    path, want, node = [], root, -1
    while True:
        fit = [i for i in range(len(parent)) if parent[i] == node and tokens[i] == want]
        if not fit:
            return path, want
        node = fit[0]
        path.append(node)
        want = int(ids[node])


def adapters(base, x, a, b, scale):
    """(base + scale (x A^T) B^T, bound): f32 sums over K and the rank, x A^T in two f16 terms (2^-22), f32 results."""
    base, x, a, b = (t.astype(np.float64) for t in (base, x, a, b))
    out = base + scale * (x @ a.T) @ b.T
    down = np.abs(x) @ np.abs(a).T
    bound = scale * ((x.shape[1] + a.shape[0] + 16) * 2.0 ** -24 * down + 2.0 ** -21 * np.abs(x @ a.T)) @ np.abs(b).T
    return out, bound + 2.0 ** -22 * np.abs(out) + 2.0 ** -23 * np.abs(base)
