"""Plain numpy reference, in float64, of the e4m3 pools with a scale per (block, kv head): the quantising write, the
read back and attention over the values read back.  Shares no code with the library."""
import numpy as np

E4M3 = np.array([np.nan if c & 127 == 127 else
                 (-1.0 if c & 128 else 1.0) * ((c & 7) / 8 * 2.0 ** -6 if (c >> 3) & 15 == 0
                                               else (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7))
                 for c in range(256)])
_POS = E4M3[:127]


def nearest_code(x):
    """Code of the nearest e4m3 value (ties to the even code, beyond 448 the largest), NaN to 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=448.0)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POS[hi] - a, a - _POS[lo]
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(_POS[hi] == a, hi, code)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), code & 128 | 127, code).astype(np.uint8)


def scale_of(amax):
    """Smallest power of two s with amax <= 448 s, at least 2^-100."""
    e = -100
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def slots(table, seq, pos, block, num_blocks):
    out, errors = [], 0
    for s, p in zip(seq, pos):
        slot = -1
        if p >= 0:
            ok = 0 <= s < table.shape[0] and p // block < table.shape[1]
            pb = table[s, p // block] if ok else -1
            if 0 <= pb < num_blocks:
                slot = int(pb) * block + p % block
            else:
                errors += 1
        out.append(slot)
    return np.array(out, np.int64), errors


def write(new, codes, scales, slot):
    """In place: rows `new` [T, H, D] float64 into codes [P, B, H, D] and scales [P, H] (float64)."""
    block = codes.shape[1]
    by_block = {}
    for t, s in enumerate(slot):
        if s >= 0:
            by_block.setdefault(int(s) // block, {})[int(s) % block] = t  # the last token of a slot is stored
    for b, rows in by_block.items():
        offs = sorted(rows)
        x = new[[rows[o] for o in offs]]
        for h in range(codes.shape[2]):
            v = x[:, h]
            fin = np.abs(v[np.isfinite(v)])
            base = 0.0 if 0 in rows else scales[b, h]
            s = max(base, scale_of(fin.max() if fin.size else 0.0))
            if 0 not in rows and s > base:
                keep = [o for o in range(block) if o not in rows]
                codes[b, keep, h] = nearest_code(E4M3[codes[b, keep, h]] * (base / s))
            codes[b, offs, h] = nearest_code(v / s)
            scales[b, h] = s


def values(codes, scales):
    return E4M3[codes] * scales[:, None, :, None]


def attend(q, k, v, scale):
    """q [G, D], k and v [n, D]: (softmax(scale q k^T) v, softmax(...) |v|); zeros without keys."""
    if k.shape[0] == 0:
        return np.zeros_like(q), np.zeros_like(q)
    s = scale * q @ k.T
    p = np.exp(s - s.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    return p @ v, p @ np.abs(v)


def context(codes, scales, table_row, n, num_blocks):
    """Values of the first n tokens of a sequence that lie in valid blocks: [m, H, D]."""
    block = codes.shape[1]
    rows = [(int(table_row[j // block]), j % block) for j in range(n)]
    rows = [(b, o) for b, o in rows if 0 <= b < num_blocks]
    if not rows:
        return np.zeros((0,) + codes.shape[2:])
    b, o = np.array(rows).T
    return E4M3[codes[b, o]] * scales[b][:, :, None]


def attend_rows(q, kc, ks, vc, vs, table_row, limits, scale):
    """q [m, Hq, D], row i attends the sequence's first limits[i] tokens: (out, softmax |v|), each [m, Hq, D]."""
    m, hq, d = q.shape
    hkv = kc.shape[2]
    g = hq // hkv
    out, mag = np.zeros_like(q), np.zeros_like(q)
    for i in range(m):
        k = context(kc, ks, table_row, limits[i], kc.shape[0])
        v = context(vc, vs, table_row, limits[i], kc.shape[0])
        for h in range(hkv):
            o, a = attend(q[i, h * g:(h + 1) * g], k[:, h], v[:, h], scale)
            out[i, h * g:(h + 1) * g], mag[i, h * g:(h + 1) * g] = o, a
    return out, mag


def floor_rows(vc, vs, table_row, limits, hq):
    """R sum_j |code_j| of each row's tokens, [m, Hq, D]: R the power of two not below any of their V scales."""
    P, block, hkv, d = vc.shape
    out = np.zeros((len(limits), hq, d))
    for i, n in enumerate(limits):
        rows = [(int(table_row[j // block]), j % block) for j in range(n)]
        rows = [(b, o) for b, o in rows if 0 <= b < P]
        if not rows:
            continue
        b, o = np.array(rows).T
        r = 2.0 ** np.ceil(np.log2(np.maximum(vs[b].max(axis=0), 2.0 ** -110)))
        out[i] = np.repeat(r[:, None] * np.abs(E4M3[vc[b, o]]).sum(axis=0), hq // hkv, axis=0)
    return out
