"""fp64 definitions of the attention layer's operators, in numpy, token by token and head by head: the 8-bit cache
format, the paged cache's write and read-back, causal attention over it, and the residual RMS norm with its gradients.
Test infrastructure: shares no code with the CUDA path."""
import numpy as np

E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -117, 119


def _e4m3_table():
    """Value of each non-negative e4m3 code 0 .. 0x7e (0x7f is NaN): bias 7, 3 mantissa bits, subnormals at 2^-6."""
    v = []
    for c in range(0x7f):
        e, m = c >> 3, c & 7
        v.append(np.ldexp(m / 8.0, -6) if e == 0 else np.ldexp(1.0 + m / 8.0, e - 7))
    return np.array(v)


TABLE = _e4m3_table()


def e4m3_code(x):
    """Nearest e4m3 code of each value (ties to the even code, magnitudes beyond 448 saturate)."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(x), E4M3_MAX)
    hi = np.clip(np.searchsorted(TABLE, mag), 0, 0x7e)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = mag - TABLE[lo], TABLE[hi] - mag
    take_hi = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    code = np.where(take_hi, hi, lo)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def e4m3_value(code):
    code = np.asarray(code)
    v = TABLE[np.minimum(code & 0x7f, 0x7e)]
    v = np.where((code & 0x7f) == 0x7f, np.nan, v)
    return np.where(code & 0x80, -v, v)


def quantise_row(x):
    """(codes, scale byte) of one cache row."""
    x = np.asarray(x, dtype=np.float64)
    if not np.all(np.isfinite(x)):
        return np.zeros(x.shape, np.uint8), 255
    amax, e = np.max(np.abs(x)), EXP_MIN
    while e < EXP_MAX and amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return e4m3_code(x * 2.0 ** -e), e + 127


def row_value(code, byte):
    return np.full(np.shape(code), np.nan) if byte == 255 else e4m3_value(code) * 2.0 ** (int(byte) - 127)


def cache_rows(cache, scale, table, page, lo, hi):
    """Positions lo .. hi - 1 of the sequence with this block table, [hi - lo, Hkv, d] fp64.  ``cache`` fp64 values
    (bf16 cache) or uint8 codes."""
    out = []
    for pos in range(lo, hi):
        pg, r = table[pos // page], pos % page
        if scale is None:
            out.append(cache[pg, :, r])
        else:
            out.append(np.stack([row_value(cache[pg, h, r], scale[pg, h, r]) for h in range(cache.shape[1])]))
    return np.stack(out) if out else np.zeros((0, cache.shape[1], cache.shape[3]))


def attention(q, k, v, scale, window=0):
    """New tokens q [T, Hq, d] at the end of the keys k, v [L, Hkv, d]: (o [T, Hq, d], lse [T, Hq], and per output the
    weighted mean of |v| and per (token, head) the largest sum of |q_c k_c| scale over the keys it sees: what error
    bounds are made of)."""
    T, Hq, d = q.shape
    L, Hkv = k.shape[:2]
    G = Hq // Hkv
    o, lse = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    absv, mass = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    for t in range(T):
        pos = L - T + t
        lo = max(0, pos - window + 1) if window else 0
        for h in range(Hq):
            kk, vv = k[lo:pos + 1, h // G], v[lo:pos + 1, h // G]
            s = kk @ q[t, h] * scale
            m = np.max(s)
            p = np.exp(s - m)
            o[t, h] = p @ vv / p.sum()
            absv[t, h] = p @ np.abs(vv) / p.sum()
            lse[t, h] = m + np.log(p.sum())
            mass[t, h] = np.max(np.abs(kk) @ np.abs(q[t, h])) * abs(scale)
    return o, lse, absv, mass


def add_rmsnorm(x, residual, weight, eps):
    s = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=-1) + eps)
    return s, rstd, s * rstd[:, None] * weight


def add_rmsnorm_grads(dy, s, weight, rstd, ds=None):
    d = s.shape[-1]
    inner = np.sum(dy * weight * s, axis=-1)
    dx = rstd[:, None] * dy * weight - (rstd ** 3 * inner / d)[:, None] * s
    return (dx if ds is None else dx + ds), np.sum(dy * s * rstd[:, None], axis=0)
