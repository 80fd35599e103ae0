"""Plain 64-bit definitions of the drafted-tree operators (imported only by tests): loops over sequences and
tokens, none of the package's code."""
import numpy as np


def path_of(parent, t):
    """Token t and its ancestors, nearest first."""
    out = []
    while t >= 0:
        out.append(t)
        up = int(parent[t])
        t = up if -1 <= up < t else -1
    return out


def ring_rows(n_swa, head, W):
    """Committed rows, newest first."""
    if n_swa == W:
        return [(head - 1 - i) % W for i in range(W)]
    return list(range(n_swa - 1, -1, -1))


def tree_attention(q, k_main, v_main, idx, k_swa, v_swa, n_swa, k_draft, v_draft, parent, n_draft, head, scale, T):
    """out, lse, sum of p |v| (for tolerances), largest sum of |q k| scale; all float64."""
    B, H, _ = q.shape
    W = k_swa.shape[1]
    out = np.zeros((B, H, v_main.shape[-1]))
    absum = np.zeros_like(out)
    lse = np.full((B, H), -np.inf)
    dot = 0.0
    for b in range(B):
        s, t = divmod(b, T)
        if n_draft is not None and t >= n_draft[s]:
            continue
        path = path_of(parent[s], t)
        ring = ring_rows(int(n_swa[s]), int(head[s]), W)[:max(0, W - len(path))]
        path = path[:W]
        sel = [e for e in idx[b] if 0 <= e < k_main.shape[1]]
        k = np.concatenate([k_main[s, sel], k_swa[s, ring], k_draft[s, path]])
        v = np.concatenate([v_main[s, sel], v_swa[s, ring], v_draft[s, path]])
        x = q[b] @ k.T * scale
        dot = max(dot, float((np.abs(q[b]) @ np.abs(k).T).max()) * scale)
        m = x.max(1, keepdims=True)
        p = np.exp(x - m)
        l = p.sum(1, keepdims=True)
        out[b] = (p / l) @ v
        absum[b] = (p / l) @ np.abs(v)
        lse[b] = (m + np.log(l))[:, 0]
    return out, lse, absum, dot


def attention_weights(q, k_main, idx, lse, scale, T):
    B, K = idx.shape
    w = np.zeros((B, K))
    for b in range(B):
        for j in range(K):
            e = idx[b, j]
            if 0 <= e < k_main.shape[1]:
                x = q[b] @ k_main[b // T, e] * scale
                fin = lse[b] != -np.inf
                w[b, j] = np.exp(x[fin] - lse[b][fin]).sum()
    return w


def evict(n, trigger, keep, sink, recent, mass):
    """Entries of one sequence that stay, ascending."""
    if n <= trigger:
        return list(range(n))
    middle = list(range(sink, n - recent))
    best = sorted(middle, key=lambda e: (-int(mass[e]), e))[:keep - sink - recent]
    return sorted(list(range(sink)) + best + list(range(n - recent, n)))


def block_means(k_idx, n, block, rounded):
    nb = -(-k_idx.shape[0] // block)
    out = np.zeros((nb, k_idx.shape[1]))
    for j in range(-(-n // block)):
        m = k_idx[j * block:min(n, (j + 1) * block)].mean(0)
        out[j] = np.rint(m) if rounded else m
    return out
