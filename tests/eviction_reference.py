"""Plain numpy reference, in float64, of the caches that evict tokens: rotary positions on several axes, attention with the
weight that each key draws, the eviction.  Shares no code with the library."""
import numpy as np


def turn(x, rope_pos, inv_freq, axis, interleaved):
    """x [T, H, D] float64 -> turned, and |a| + |b| of each element's pair (0 where it stays)."""
    half = len(inv_freq)
    out, mag = x.copy(), np.zeros_like(x)
    for i in range(half):
        angle = rope_pos[axis[i]].astype(np.float64) * np.float64(inv_freq[i])
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return out, mag


def attend(q, kc, vc, table_row, limits, scale):
    """q [m, Hq, D] float64; row i sees the sequence's first limits[i] tokens that lie in valid blocks.  Returns the outputs,
    softmax |v|, each key's weight summed over rows and heads [Hkv, n], and a bound on a weight's relative error when
    scores, exponentials and sums are taken in 32 bits."""
    m, hq, d = q.shape
    P, B, hkv, _ = kc.shape
    n = int(max(limits, default=0))
    g = hq // hkv
    out, mag, w, rel = np.zeros_like(q), np.zeros_like(q), np.zeros((hkv, n)), 0.0
    blocks = np.array([table_row[j // B] for j in range(n)], dtype=np.int64)
    ok = (blocks >= 0) & (blocks < P)
    at = np.where(ok, blocks, 0), np.arange(n) % B
    for h in range(hkv):
        k, v = kc[at[0], at[1], h], vc[at[0], at[1], h]
        k[~ok], v[~ok] = 0, 0
        for i in range(m):
            see = ok & (np.arange(n) < limits[i])
            if not see.any():
                continue
            k1, v1 = k[see], v[see]
            for e in range(h * g, (h + 1) * g):
                s = scale * (k1 @ q[i, e])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[i, e], mag[i, e] = p @ v1, p @ np.abs(v1)
                w[h, see] += p
                # a score is off by (D + 8) roundings of its terms' magnitudes, a 2^x by its argument's rounding
                terms = scale * (np.abs(k1) @ np.abs(q[i, e])).max()
                rel = max(rel, 2 * (d + 8) * 2.0 ** -23 * terms + 8 * 2.0 ** -23 * (np.abs(s).max() + np.log(len(s)) + 1))
    return out, mag, w, rel + 2.0 ** -20


def kept(weights, places, n, budget, keep_first, recent_from):
    """Indices of the tokens of one head that stay, of its first n."""
    def rank(j):
        if places[j] < keep_first or places[j] >= recent_from:
            return (0, 0.0, j)
        x = float(weights[j])
        return (1, np.inf if np.isnan(x) else -x + 0.0, j)
    return sorted(sorted(range(n), key=rank)[:budget])


def evict(kc, vc, table, lens, weights, places, next_pos, budget, keep_first, keep_recent):
    """In place; returns the new lengths."""
    P, B, hkv, _ = kc.shape
    for s, n in enumerate(lens):
        if n <= budget:
            continue
        for h in range(hkv):
            stay = set(kept(weights[s, h], places[s, h], n, budget, keep_first, int(next_pos[s]) - keep_recent))
            src = [j for j in range(budget, n) if j in stay]
            dst = [j for j in range(budget) if j not in stay]
            for a, b in zip(src, dst):
                weights[s, h, b], places[s, h, b] = weights[s, h, a], places[s, h, a]
                x, y = table[s, a // B], table[s, b // B]
                if 0 <= x < P and 0 <= y < P:
                    kc[y, b % B, h], vc[y, b % B, h] = kc[x, a % B, h], vc[x, a % B, h]
    return np.minimum(lens, budget)
