"""Plain 64-bit forms of the serving operators on the int8 KV cache (test code
only): attention of drafted tokens, the commit of a path, the attention weight
of cached rows and the choice of the rows to keep.  NumPy, one head at a time."""
import numpy as np


def draft_codes(K, V, mean, ks, vs):
    """int8 codes of drafts [T, d] with a head's header: fp32, one rounding a step."""
    k = np.clip(np.rint(((K - mean).astype(np.float32) / ks).astype(np.float32)), -127, 127)
    v = np.clip(np.rint((V / vs).astype(np.float32)), -127, 127)
    return k, v


def visible(T, L, mask=None, mode="tree"):
    """[T, L + drafts] truth values.  mode: tree (mask [T, T]), chain, all, cached
    (no drafts), cached_causal."""
    cached = np.ones((T, L), dtype=bool)
    if mode == "cached":
        return cached
    if mode == "cached_causal":
        return np.arange(L)[None] <= (L - T + np.arange(T))[:, None]
    d = {"tree": mask, "chain": np.tril(np.ones((T, T), dtype=bool)),
         "all": np.ones((T, T), dtype=bool)}[mode]
    return np.concatenate([cached, d], axis=1)


def attend(qc, scale, kc, vc, vs, see):
    """One head: O [T, d], lse [T], A = sum_j P_j |v_j| / sum P (the size of what is
    summed) and the largest |t| in log2 units."""
    s = (qc.astype(np.float64) @ kc.astype(np.float64).T) * scale
    s = np.where(see, s, -np.inf)
    top = s.max(axis=1, initial=-np.inf)
    live = top > -np.inf
    p = np.exp(s - np.where(live, top, 0.0)[:, None])
    z = p.sum(axis=1)
    v = vc.astype(np.float64) * vs.astype(np.float64)
    inv = np.where(live, 1.0 / np.where(live, z, 1.0), 0.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(live, top + np.log(z), -np.inf)
    big = np.abs(np.where(see, s, 0.0)).max(initial=0.0) / np.log(2.0)
    return (p @ v) * inv, lse, (p @ np.abs(v)) * inv, big


def commit(K, V, path, n, L, seen, ks, vs, mean, amax, kc, vc):
    """One sequence, in place: K, V [H, T, d] fp32; kc, vc [H, cap, d]."""
    mean, amax = mean.copy(), amax.copy()
    for t in range(n):
        j = path[t]
        diff = (K[:, j] - mean).astype(np.float32)
        kc[:, L + t] = np.clip(np.rint((diff / ks).astype(np.float32)), -127, 127)
        mean = (mean + (diff / np.float32(seen + t + 1)).astype(np.float32)).astype(np.float32)
        qv = np.clip(np.rint((V[:, j] / vs).astype(np.float32)), -127, 127)
        vc[:, L + t] = qv
        amax = np.maximum(amax, np.abs(qv)).astype(np.float32)
    return mean, amax


def weight(qc, qs, kc, ks, lse, see, sm):
    """One query head: sum over its tokens of exp(s - lse), [L]; and the largest |t|."""
    s = (qc.astype(np.float64) @ kc.astype(np.float64).T) * qs.astype(np.float64)[:, None]
    s = s * ks.astype(np.float64)[None] * sm
    live = (lse > -np.inf)[:, None] & see
    p = np.where(live, np.exp(np.where(live, s - np.where(lse > -np.inf, lse, 0)[:, None], 0.0)), 0.0)
    return p.sum(axis=0), np.abs(s).max(initial=0.0) / np.log(2.0)


def keep(w, L, budget, n_sink, n_recent):
    """Rows kept, ascending."""
    r = np.arange(L)
    guard = (r < n_sink) | (r >= L - n_recent)
    v = np.where(np.isnan(w[:L]), -np.inf, w[:L])
    return np.sort(np.lexsort((r, -v, ~guard))[:min(L, budget)])
