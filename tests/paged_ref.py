"""Plain forms of the paged cache's operators (test code only): the rotation and the
append in single fp32 operations, one page at a time; the attention in 64 bits, one
head at a time.  NumPy, and torch for e4m3 and bf16 roundings."""
import numpy as np
import torch

TOP = {"int8": np.float32(127.0), "e4m3": np.float32(448.0)}
f32 = np.float32


def bf16(x):
    """x rounded to bf16, as fp32."""
    return torch.from_numpy(np.array(x, np.float32, order="C")).to(torch.bfloat16).float().numpy()


def table(n, rot, base=10000.0):
    i = np.arange(rot // 2)
    a = np.arange(n)[:, None] * base ** (-2.0 * i / rot)
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def rotate(x, pos, tab, inter, inverse=False):
    """x fp32 [..., T, d], pos [T]: every product and sum rounded to fp32."""
    rot = tab.shape[1]
    c, s = tab[pos, :rot // 2], tab[pos, rot // 2:]
    s = -s if inverse else s
    y = x.copy()
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = (a * c).astype(f32) - (b * s).astype(f32), (b * c).astype(f32) + (a * s).astype(f32)
    if inter:
        y[..., :rot:2], y[..., 1:rot:2] = u, v
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = u, v
    return y


def encode(y, code):
    """fp32 values / scale -> codes (int8, or e4m3 bytes)."""
    if code == "int8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8)
    t = torch.from_numpy(np.clip(y, -448, 448).astype(np.float32))
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def decode(c, code):
    """Codes as the values they stand for, before the scale (float64)."""
    if code == "int8":
        return c.astype(np.float64)
    return torch.from_numpy(np.ascontiguousarray(c)).view(torch.float8_e4m3fn).double().numpy()


def append(x, first, code, page, table_row, pages, scales):
    """One sequence, K or V: x fp32 [Hkv, n, d] into rows first .. of the pages, in place."""
    H, n, d = x.shape
    top = TOP[code]
    r = 0
    while r < n:
        j, at = divmod(first + r, page)
        m = min(n - r, page - at)
        p = int(table_row[j])
        for h in range(H):
            new = x[h, r:r + m]
            a = f32(np.abs(new).max())
            old = scales[p, h]
            if not np.isfinite(a) or (at > 0 and not (np.isfinite(old) and old >= 0)):
                scales[p, h] = np.nan
                pages[p, h, at:at + m] = 0
                continue
            if at > 0 and old >= f32(2.0 ** -100):
                s = old
                while a > f32(top * s):
                    s = f32(s * 2)
                if s != old:
                    pages[p, h, :at] = encode((decode(pages[p, h, :at], code) * float(old) / float(s)).astype(f32), code)
            else:
                s = f32(0) if a < f32(2.0 ** -64) else f32(a * f32(f32(1) / top))
                if at > 0 and s > 0:
                    pages[p, h, :at] = 0
            scales[p, h] = s
            inv = f32(f32(1) / s) if s > 0 else f32(0)
            pages[p, h, at:at + m] = encode((new * inv).astype(f32), code)
        r += m


def rows(pages, scales, table_row, h, L, page, code):
    """A KV head's codes [L, d] and the scale of each row, float64."""
    no = [int(p) for p in table_row[:-(-L // page)]]
    if not no:
        return np.zeros((0, pages.shape[3])), np.zeros(0)
    c = decode(pages[no, h], code).reshape(-1, pages.shape[3])[:L]
    return c, np.repeat(scales[no, h].astype(np.float64), page)[:L]


def attend(q, kc, ks, vc, vs, see, sm):
    """One query head: O [n, d], lse [n]; A = sum P |v| / sum P (the size of what is
    summed), and the largest |t| in log2 units (scores and the V scale's exponent)."""
    s = (q.astype(np.float64) @ kc.T) * ks * sm
    s = np.where(see, s, -np.inf)
    top = s.max(axis=1, initial=-np.inf)
    live = top > -np.inf
    p = np.exp(s - np.where(live, top, 0.0)[:, None])
    z = p.sum(axis=1)
    vs = np.where(vs < 2.0 ** -48, 0.0, vs)
    v = vc * vs[:, None]
    inv = np.where(live, 1.0 / np.where(live, z, 1.0), 0.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(live, top + np.log(z), -np.inf)
    big = np.abs(np.where(see, s, 0.0)).max(initial=0.0) / np.log(2.0)
    big += np.abs(np.log2(np.maximum(vs, 2.0 ** -48))).max(initial=0.0)
    # the largest part of a single key in O, on which P's absolute error below fp16's normal range counts
    part = (p * vs).max(axis=1, initial=0.0)[:, None] * inv
    return (p @ v) * inv, lse, (p @ np.abs(v)) * inv, big, part
