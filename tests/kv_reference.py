"""Plain 64-bit references of the paged 8-bit key/value cache and of tree attention (numpy, no framework code)."""
import numpy as np

NAN_SCALE = 255


def e4m3_table() -> np.ndarray:
    """Value of each e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    t = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        t[c] = s * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    t[0x7F] = t[0xFF] = np.nan
    return t


E4M3 = e4m3_table()
_POS = E4M3[:0x7F]                                        # ascending: codes 0 .. 0x7E


def round_e4m3(y: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values of |y| <= 448, ties to the even code."""
    a = np.abs(y)
    hi = np.clip(np.searchsorted(_POS, a), 1, len(_POS) - 1)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def quantise(x: np.ndarray):
    """(codes, scale bytes) of vectors along the last axis, by the definition in the header."""
    x = x.astype(np.float64)
    codes = np.zeros(x.shape, np.uint8)
    scales = np.zeros(x.shape[:-1], np.uint8)
    for i in np.ndindex(x.shape[:-1]):
        v = x[i]
        if not np.isfinite(v).all():
            scales[i] = NAN_SCALE
            continue
        amax = np.abs(v).max()
        e = 0
        if amax > 0:
            e = -100
            while e < 120 and amax > 448.0 * 2.0 ** e:
                e += 1
        scales[i] = e + 127
        codes[i] = round_e4m3(v * 2.0 ** -e)
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    f = np.where(scales == NAN_SCALE, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return E4M3[codes] * f[..., None]


def lane_rows(pool: np.ndarray, table_row: np.ndarray, n: int) -> np.ndarray:
    """Rows 0 .. n-1 of a lane, [n, heads, ...], from a pool [pages, heads, page, ...]."""
    page = pool.shape[2]
    at = np.arange(n)
    return pool[table_row[at // page], :, at % page]


def visible(n: int, total: int, mask, first: int) -> np.ndarray:
    """[n, total] truth values: what node t of a lane sees (mask words [nodes, words] uint32, or None)."""
    see = np.ones((n, total), bool)
    for t in range(n):
        for i in range(n):
            see[t, total - n + i] = i <= t if mask is None else bool(mask[first + t, i // 32] >> np.uint32(i % 32) & 1)
    return see


def attention(q, k, v, see, scale):
    """One lane and head: q [n, D], k and v [L, D] float64, see [n, L]. Returns out [n, D], lse [n], and
    sum p |v| [n, D] (the scale that roundings of p act on)."""
    n, D = q.shape
    out, lse, mass = np.zeros((n, D)), np.full(n, -np.inf), np.zeros((n, D))
    for t in range(n):
        j = np.flatnonzero(see[t])
        if not len(j):
            continue
        with np.errstate(all="ignore"):
            s = k[j] @ q[t] * scale
            top = s.max()
            p = np.exp(s - top)
            total = p.sum()
            out[t] = p @ v[j] / total
            mass[t] = p @ np.abs(v[j]) / total
            lse[t] = top + np.log(total)
    return out, lse, mass
