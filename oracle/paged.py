"""fp64 definitions of the paged 8-bit key/value cache: rotation, append, attention.

Test infrastructure, like the rest of this package.  Pinned in ``tests/test_oracle_paged.py``.
"""
import numpy as np

E4M3_MAX = 448.0
BORDER = 449.0


def e4m3_table():
    """The value of every e4m3 byte."""
    t = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        t[b] = -v if b & 128 else v
    return t


def e4m3_step(x):
    """Distance of neighbouring e4m3 values around |x|."""
    _, e = np.frexp(np.abs(x))
    return 2.0 ** (np.maximum(e - 1, -6) - 3)


def to_e4m3(x):
    """Nearest e4m3 value, half to even, clipped at +-448; NaN for what is not finite."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    y = np.where(fine, x, 0.0)
    s = e4m3_step(y)
    return np.where(fine, np.clip(np.round(y / s) * s, -E4M3_MAX, E4M3_MAX), np.nan)


def scale_of(amax):
    """Least power of two s in 2^-32..2^32 with amax <= 449 s."""
    e = -32
    while e < 32 and amax > BORDER * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x, positions, inv_freq, sections, interleaved=False):
    """x [T, heads, d]; positions [axes, T]."""
    x = np.array(x, np.float64)
    half, i = len(inv_freq), 0
    for axis, count in enumerate(sections):
        for _ in range(count):
            f = np.asarray(positions[axis], np.float64) * float(inv_freq[i])
            c, s = np.cos(f)[:, None], np.sin(f)[:, None]
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            lo, hi = x[:, :, a].copy(), x[:, :, b].copy()
            x[:, :, a], x[:, :, b] = lo * c - hi * s, lo * s + hi * c
            i += 1
    return x


def append(x, cu, kv_lens, table, cache, scale):
    """Appends rows x [T, h, d] to `cache` (e4m3 values, [pages, h, page, d]) and `scale` [pages, h], in place.
    Returns {(page, head, slot): the unrounded row} of the new tokens."""
    page, n_pages, rows = cache.shape[2], cache.shape[0], {}
    for n in range(len(cu) - 1):
        new = cu[n + 1] - cu[n]
        start = kv_lens[n] - new
        if new == 0 or start < 0 or kv_lens[n] > table.shape[1] * page:
            continue
        for slot in range(start // page, (kv_lens[n] - 1) // page + 1):
            at = int(table[n, slot])
            if not 0 <= at < n_pages:
                continue
            lo, hi = max(start, slot * page), min(kv_lens[n], (slot + 1) * page)
            old = lo - slot * page
            for h in range(cache.shape[1]):
                part = x[cu[n] + lo - start:cu[n] + hi - start, h]
                fine = np.abs(part[np.isfinite(part)])
                s = scale_of(fine.max() if fine.size else 0.0)
                if old:
                    s = max(s, scale[at, h])
                    if s != scale[at, h]:
                        cache[at, h, :old] = to_e4m3(cache[at, h, :old] * (scale[at, h] / s))
                scale[at, h] = s
                cache[at, h, old:old + hi - lo] = to_e4m3(part / s)
                for i in range(hi - lo):
                    rows[at, h, old + i] = part[i]
    return rows


def attention(q, cu, kv_lens, table, k_cache, v_cache, k_scale, v_scale, scale=None):
    """(o [T, h_q, d], lse [T, h_q]) of the causal attention of every sequence's last rows over its cached tokens.  A
    row that sees no token has o = 0, lse = -inf.  Caches hold e4m3 values."""
    T, h_q, d = q.shape
    h_kv, page = k_cache.shape[1], k_cache.shape[2]
    scale = d ** -0.5 if scale is None else scale
    o, lse = np.zeros((T, h_q, d)), np.full((T, h_q), -np.inf)
    for n in range(len(cu) - 1):
        total, new = kv_lens[n], cu[n + 1] - cu[n]
        pages = np.asarray(table[n, :(total + page - 1) // page], np.int64)
        k = (k_cache[pages] * k_scale[pages][..., None, None]).transpose(1, 0, 2, 3).reshape(h_kv, -1, d)
        v = (v_cache[pages] * v_scale[pages][..., None, None]).transpose(1, 0, 2, 3).reshape(h_kv, -1, d)
        for i in range(new):
            seen = total - new + i + 1
            if seen <= 0:
                continue
            for h in range(h_q):
                g = h // (h_q // h_kv)
                s = (k[g, :seen] @ q[cu[n] + i, h]) * scale
                m = s.max()
                p = np.exp(s - m)
                o[cu[n] + i, h] = (p / p.sum()) @ v[g, :seen]
                lse[cu[n] + i, h] = m + np.log(p.sum())
    return o, lse
