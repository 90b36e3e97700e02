"""fp64 numpy oracle of the rotary positions and of the 8-bit cache (include/lfm2sc_hybrid.h), written from its formulas;
TEST INFRASTRUCTURE ONLY.  The one place that is not fp64 is where the header fixes fp32 steps: a block's scale and the
quotient that is rounded to a code (numpy's float32 arithmetic is IEEE, so codes are the exact ones).

A cache is a dict: page, block, int8, k / v code values [pages, heads, page, D] (float64, token-major for both), ks / vs
scales [pages, heads, page / block] (float32).
"""
import numpy as np

from oracle.hybrid import _probabilities, f64

F32 = np.float32
MIN_SCALE = F32(2.0 ** -100)


# ---------------------------------------------------------------- rotary
def rotary(x, D, freqs, positions, interleaved=False, inverse=False, magnitude=1.0):
    """Rows x [T, heads*D] at positions [T]."""
    x, f = f64(x), f64(freqs)
    T, R = x.shape[0], 2 * f.size
    a = np.asarray(positions, dtype=np.float64)[:, None] * f
    c, s = magnitude * np.cos(a)[:, None], magnitude * np.sin(a)[:, None] * (-1.0 if inverse else 1.0)
    y = x.reshape(T, -1, D).copy()
    i, j = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    u, v = y[:, :, i].copy(), y[:, :, j].copy()
    y[:, :, i] = u * c - v * s
    y[:, :, j] = v * c + u * s
    return y.reshape(T, -1)


def packed_positions(cu, T, starts=None):
    """Position of every row, and whether it belongs to a sequence."""
    pos, mine = np.zeros(T, dtype=np.int64), np.zeros(T, dtype=bool)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        pos[a:b] = np.arange(b - a) + (0 if starts is None else starts[i])
        mine[a:b] = True
    return pos, mine


# ---------------------------------------------------------------- codes
def round_code(x, int8):
    """x (float32, in steps of the scale) as the value of its code."""
    x = np.asarray(x, dtype=np.float64)
    if int8:
        return np.clip(np.rint(np.where(np.isnan(x), 0.0, x)), -127, 127)
    with np.errstate(invalid="ignore"):
        a = np.clip(x, -448, 448)
        step = 2.0 ** (np.maximum(np.frexp(np.where(np.isfinite(a), a, 0.0))[1], -5) - 4)
        return np.clip(np.rint(a / step) * step, -448, 448)


def fresh(top, int8):
    if not top > 0:
        return F32(0)
    if int8:
        return max(F32(top) / F32(127), MIN_SCALE)
    m, e = np.frexp(np.float64(top))                         # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return max(F32(2.0) ** F32(e - 9 + (m > 0.875)), MIN_SCALE)


def joined(old, top, int8):
    """(scale, old / scale) of a block that keeps tokens of scale `old`."""
    if not (old >= MIN_SCALE and np.isfinite(old)):
        return fresh(top, int8), 0.0
    with np.errstate(over="ignore"):
        need = F32(top) * (F32(1) / F32(old))
    if not need < F32(1.1e12):
        return fresh(top, int8), 0.0
    n = 0
    while not (float(need) * 2.0 ** -n < 127.5 if int8 else float(need) * 2.0 ** -n <= 448):
        n += 1
    return F32(old) * F32(2.0) ** F32(n), 2.0 ** -n


def _magnitude(x):
    a = np.abs(x)
    return float(np.where(np.isfinite(a), a, 0.0).max(initial=0.0))


def write(cache, k, v, page_table, seq_len, lens):
    """Appends rows k, v [sum lens, heads*D] in place."""
    S, B, int8 = cache["page"], cache["block"], cache["int8"]
    P, H, _, D = cache["k"].shape
    cap = page_table.shape[1] * S
    for x, codes, scales in ((f64(k), cache["k"], cache["ks"]), (f64(v), cache["v"], cache["vs"])):
        row = 0
        for i, n in enumerate(lens):
            rows = x[row:row + n].reshape(n, H, D)
            row += n
            end = min(max(int(seq_len[i]), 0), cap)
            start = end - n
            for b in range(max(start, 0) // B, -(-end // B) if n else 0):
                t = np.arange(max(b * B, start, 0), min((b + 1) * B, end))
                page = page_table[i, b * B // S]
                if t.size == 0 or not 0 <= page < P:
                    continue
                kept = np.arange(b * B, max(min(start, (b + 1) * B), b * B)) % S
                for h in range(H):
                    new = rows[t - start, h]
                    top = _magnitude(new)
                    at = (page, h, b * B % S // B)
                    if kept.size:
                        scale, ratio = joined(scales[at], top, int8)
                        codes[page, h, kept] = round_code(codes[page, h, kept] * ratio, int8)
                    else:
                        scale = fresh(top, int8)
                    inv = F32(1) / scale if scale > 0 else F32(0)
                    with np.errstate(invalid="ignore", over="ignore"):
                        codes[page, h, t % S] = round_code(new.astype(F32) * inv, int8)
                    scales[at] = scale


def values(cache, pages, n):
    """k, v [n, heads, D] in float64 of the first n tokens of a list of pages (numbers outside the pool: the nearest)."""
    P = cache["k"].shape[0]
    pages = np.clip(np.asarray(pages[:-(-n // cache["page"])], dtype=np.int64), 0, P - 1)
    out = []
    for codes, scales in ((cache["k"], cache["ks"]), (cache["v"], cache["vs"])):
        x = codes[pages] * np.repeat(scales[pages].astype(np.float64), cache["block"], axis=2)[..., None]
        out.append(x.transpose(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])[:n])
    return out


def attention(q, cache, prefix_pages, prefix_len, page_table, suffix_len, L, scale):
    """out [N*L, Hq*D], spread = sum p |v|, and the largest |score| terms sum |q||k| scale, for lfm2sc_attn_cached8."""
    q = f64(q)
    _, Hkv, _, D = cache["k"].shape
    N, Hq = page_table.shape[0], q.shape[1] // D
    out, spread, most = np.zeros_like(q), np.zeros_like(q), 0.0
    pk, pv = values(cache, prefix_pages, prefix_len) if prefix_len else (np.zeros((0, Hkv, D)),) * 2
    for i in range(N):
        n = min(max(int(suffix_len[i]), 0), page_table.shape[1] * cache["page"])
        ok, ov = values(cache, page_table[i], n) if n else (np.zeros((0, Hkv, D)),) * 2
        k, v = np.concatenate([pk, ok]), np.concatenate([pv, ov])
        for s in range(L):
            seen = prefix_len + max(0, n - L + s + 1)
            for h in range(Hq):
                g = h // (Hq // Hkv)
                c = slice(h * D, h * D + D)
                row = q[i * L + s, c]
                p, _ = _probabilities((scale * row @ k[:seen, g].T)[None])
                if seen:
                    most = max(most, float((scale * np.abs(row) @ np.abs(k[:seen, g]).T).max()))
                out[i * L + s, c] = p[0] @ v[:seen, g]
                spread[i * L + s, c] = p[0] @ np.abs(v[:seen, g])
    return out, spread, most
