"""fp64 numpy oracle of include/lfm2sc_hybrid.h, written from its formulas; TEST INFRASTRUCTURE ONLY.

Arrays are numpy arrays or CPU tensors (widened exactly to float64).  Packed rows [T, heads*D]; nothing is computed for
rows of no sequence (NaN there).  The `*_bounds` outputs are the magnitudes that rounding errors of the operands scale
with; see the functions.
"""
import numpy as np


def f64(x):
    if x is None:
        return None
    return x.detach().cpu().double().numpy() if hasattr(x, "detach") else np.asarray(x, dtype=np.float64)


def _sequences(cu, T):
    cu = [min(max(int(c), 0), T) for c in np.asarray(cu)]
    return [(a, b) for a, b in zip(cu, cu[1:]) if b > a]


def _probabilities(s):
    """Row softmax of scores with -inf masks, and ln of the sum; a row without a key has no weight."""
    top = s.max(1, keepdims=True, initial=-np.inf)
    ref = np.where(np.isneginf(top), 0.0, top)
    e = np.exp(s - ref)
    z = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (ref + np.log(z))[:, 0]
    return e / np.where(z > 0, z, 1.0), lse


def attention(q, k, v, cu, D, scale):
    """out [T, Hq*D], lse [Hq, T], and spread [T, Hq*D] = sum_j p_j |v_j|."""
    q, k, v = f64(q), f64(k), f64(v)
    T, Hq, Hkv = q.shape[0], q.shape[1] // D, k.shape[1] // D
    out, spread, lse = np.full((T, Hq * D), np.nan), np.full((T, Hq * D), np.nan), np.full((Hq, T), np.nan)
    for a, b in _sequences(cu, T):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            c, kc = slice(h * D, h * D + D), slice(g * D, g * D + D)
            s = scale * q[a:b, c] @ k[a:b, kc].T
            s[np.triu_indices(b - a, 1)] = -np.inf
            p, lse[h, a:b] = _probabilities(s)
            out[a:b, c] = p @ v[a:b, kc]
            spread[a:b, c] = p @ np.abs(v[a:b, kc])
    return out, lse, spread


def attention_backward(q, k, v, cu, D, scale, d_out, half_step=0.0):
    """dq, dk, dv and, for each, a bound of what rounding p, ds (relative half_step each) and out (half_step of its value
    and of its terms, which delta = d_out.out inherits) can move it by."""
    q, k, v, d_out = f64(q), f64(k), f64(v), f64(d_out)
    T, Hq, Hkv = q.shape[0], q.shape[1] // D, k.shape[1] // D
    out, _, spread = attention(q, k, v, cu, D, scale)
    dq, bq = np.full((T, Hq * D), np.nan), np.full((T, Hq * D), np.nan)
    dk, dv, bk, bv = (np.full((T, Hkv * D), np.nan) for _ in range(4))
    for a, b in _sequences(cu, T):
        for x in (dk, dv, bk, bv):
            x[a:b] = 0.0
        for h in range(Hq):
            g = h // (Hq // Hkv)
            c, kc = slice(h * D, h * D + D), slice(g * D, g * D + D)
            s = scale * q[a:b, c] @ k[a:b, kc].T
            s[np.triu_indices(b - a, 1)] = -np.inf
            p, _ = _probabilities(s)
            do = d_out[a:b, c]
            ds = p * (do @ v[a:b, kc].T - (do * out[a:b, c]).sum(1, keepdims=True))
            e = half_step * (np.abs(ds) + p * (np.abs(do) * (spread[a:b, c] + np.abs(out[a:b, c]))).sum(1, keepdims=True))
            dq[a:b, c] = scale * ds @ k[a:b, kc]
            bq[a:b, c] = scale * e @ np.abs(k[a:b, kc])
            dk[a:b, kc] += scale * ds.T @ q[a:b, c]
            bk[a:b, kc] += scale * e.T @ np.abs(q[a:b, c])
            dv[a:b, kc] += p.T @ do
            bv[a:b, kc] += half_step * p.T @ np.abs(do)
    return (dq, dk, dv), (bq, bk, bv)


def cached(q, k_pages, v_pages, prefix_pages, prefix_len, page_table, suffix_len, L, scale):
    """out [N*L, Hq*D] and spread as in attention(); a row that sees no key gives zeros."""
    q, k_pages, v_pages = f64(q), f64(k_pages), f64(v_pages)
    P, S, Hkv, D = k_pages.shape
    Hq = q.shape[1] // D
    out, spread = np.zeros((q.shape[0], Hq * D)), np.zeros((q.shape[0], Hq * D))

    def keys(pool, pages, n):
        pages = np.clip(np.asarray(pages, dtype=np.int64), 0, P - 1)
        return pool[pages].reshape(-1, Hkv, D)[:n]

    for i, n in enumerate(np.asarray(suffix_len)):
        n = min(max(int(n), 0), np.asarray(page_table).shape[1] * S)
        k, v = (np.concatenate([keys(x, prefix_pages, prefix_len) if prefix_len else np.zeros((0, Hkv, D)),
                                keys(x, np.asarray(page_table)[i], n)]) for x in (k_pages, v_pages))
        for s in range(L):
            see = prefix_len + max(0, n - L + 1 + s)
            for h in range(Hq):
                g, c = h // (Hq // Hkv), slice(h * D, h * D + D)
                if see == 0:
                    continue
                p, _ = _probabilities(scale * q[i * L + s, None, c] @ k[:see, g].T)
                out[i * L + s, c] = (p @ v[:see, g])[0]
                spread[i * L + s, c] = (p @ np.abs(v[:see, g]))[0]
    return out, spread


def _weights(row):
    """A row's entries as weights: NaN and negative ones count as 0."""
    return np.nan_to_num(row, nan=0.0, posinf=np.inf, neginf=0.0).clip(min=0.0)


def accept_drafts(target, tokens, u_accept, u_sample, draft=None, num_drafts=None):
    """(accept_len, next_token) of each sequence."""
    target, draft, tokens = f64(target), f64(draft), np.asarray(tokens)
    N, L = tokens.shape
    V = target.shape[1]
    lens, picks = [], []
    for n in range(N):
        drafts = L if num_drafts is None else min(max(int(num_drafts[n]), 0), L)
        a = 0
        while a < drafts:
            x = int(tokens[n, a])
            inside = 0 <= x < V
            p = target[n * (L + 1) + a, x] if inside else 0.0
            q = draft[n * L + a, x] if draft is not None and inside else 1.0
            if not float(u_accept[n, a]) * q < p:
                break
            a += 1
        p = _weights(target[n * (L + 1) + a])
        r = p
        if a < drafts:
            if draft is not None:
                with np.errstate(invalid="ignore"):
                    r = p - _weights(draft[n * L + a])
                r = np.where(r > 0, r, 0.0)
            else:
                r = p.copy()
                if 0 <= tokens[n, a] < V:
                    r[tokens[n, a]] = 0.0
            if not r.sum() > 0:
                r = p
        cum = np.cumsum(r)
        over = np.flatnonzero((cum > float(u_sample[n]) * cum[-1]) & (r > 0))
        some = np.flatnonzero(r > 0)
        lens.append(a)
        picks.append(int(over[0]) if over.size else int(some[-1]) if some.size else -1)
    return np.array(lens), np.array(picks)
