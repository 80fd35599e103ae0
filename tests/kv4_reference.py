"""Plain 64-bit definitions of the 4-bit main cache and of the norm with rotary positions (imported only by tests): none of
the package's code, every group and row by itself."""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:119])


def nearest(x, table):
    """Index of the entry of `table` nearest to x >= 0, at a tie the even one; the last where x is beyond it."""
    d = np.abs(table - np.minimum(x, table[-1]))
    best = np.flatnonzero(d == d.min())
    return int(best[0] if best[0] % 2 == 0 else best[-1])


def groups(d):
    return -(-d // 16)


def entry_bytes(dk, dv):
    return -(-9 * (groups(dk) + groups(dv)) // 16) * 16


def quantise(x, exp):
    """Codes [groups, 16] and scale bytes [groups] of one key or value [d]."""
    x = np.concatenate([np.asarray(x, dtype=np.float64), np.zeros(-len(x) % 16)]).reshape(-1, 16) * 2.0 ** -exp
    codes, scales = np.zeros(x.shape, dtype=np.int64), np.zeros(len(x), dtype=np.int64)
    for g, y in enumerate(x):
        top = np.abs(y).max()
        if not np.isfinite(top):
            scales[g] = 127
            continue
        scales[g] = max(1, nearest(top / 6.0, SCALES))
        for i, v in enumerate(y):
            codes[g, i] = nearest(abs(v) / SCALES[scales[g]], LEVELS) + (8 if v < 0 else 0)
    return codes, scales


def values(codes, scales, d, exp):
    """The numbers [d] that codes and scale bytes stand for."""
    s = np.where(scales == 127, np.nan, SCALES[np.minimum(scales, 126)])[:, None]
    return (LEVELS[codes % 8] * np.where(codes >= 8, -1.0, 1.0) * s).reshape(-1)[:d] * 2.0 ** exp


def pack(k, v, k_exp, v_exp):
    """An entry's bytes, of one key and one value."""
    parts = [quantise(k, k_exp), quantise(v, v_exp)]
    codes = np.concatenate([c.reshape(-1) for c, _ in parts])
    out = np.zeros(entry_bytes(len(k), len(v)), dtype=np.uint8)
    out[:len(codes) // 2] = codes[0::2] | codes[1::2] << 4
    scales = np.concatenate([s for _, s in parts])
    out[len(codes) // 2:len(codes) // 2 + len(scales)] = scales
    return out


def unpack(entry, dk, dv, k_exp, v_exp):
    """Key and value of an entry's bytes."""
    gk, gv = groups(dk), groups(dv)
    raw = np.asarray(entry, dtype=np.int64)
    codes = np.stack([raw[:8 * (gk + gv)] & 15, raw[:8 * (gk + gv)] >> 4], 1).reshape(-1, 16)
    scales = raw[8 * (gk + gv):9 * (gk + gv)]
    return values(codes[:gk], scales[:gk], dk, k_exp), values(codes[gk:], scales[gk:], dv, v_exp)


def attention(q, keys, vals, idx, k_swa, v_swa, n_swa, scale, T):
    """out, lse, sum of p |v| and the largest sum of |q k| scale; keys and vals [S, N, d] as numbers."""
    B, H, _ = q.shape
    out = np.zeros((B, H, vals.shape[-1]))
    absum, lse, dot = np.zeros_like(out), np.full((B, H), -np.inf), 0.0
    for b in range(B):
        sel = [e for e in idx[b] if 0 <= e < keys.shape[1]]
        n = min(max(int(n_swa[b]), 0), k_swa.shape[1])
        k = np.concatenate([keys[b // T, sel], k_swa[b, :n]])
        v = np.concatenate([vals[b // T, sel], v_swa[b, :n]])
        if len(k) == 0:
            continue
        x = q[b] @ k.T * scale
        dot = max(dot, float((np.abs(q[b]) @ np.abs(k).T).max()) * scale)
        m = x.max(1, keepdims=True)
        p = np.exp(x - m)
        l = p.sum(1, keepdims=True)
        out[b] = (p / l) @ v
        absum[b] = (p / l) @ np.abs(v)
        lse[b] = (m + np.log(l))[:, 0]
    return out, lse, absum, dot


def norm_rope(x, gain, eps, center, angle, mag, off, inter):
    """x [rows, heads, dim], gain broadcast to it, angle [rows, rot / 2] (None: nothing is turned); (y, the norm alone)."""
    x = x.astype(np.float64)
    if center:
        x = x - x.mean(-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain
    plain = y.copy()
    if angle is None:
        return y, plain
    rot = 2 * angle.shape[1]
    at = np.arange(rot).reshape(-1, 2).T if inter else np.arange(rot).reshape(2, -1)
    a, b = plain[..., off + at[0]], plain[..., off + at[1]]
    c, s = (np.cos(angle) * mag).astype(np.float64)[:, None], (np.sin(angle) * mag).astype(np.float64)[:, None]
    y[..., off + at[0]], y[..., off + at[1]] = a * c - b * s, b * c + a * s
    return y, plain
