"""The 8-bit cache's definition in plain numpy float64, for the tests: codes, scales, the quantising
store on a logical [nkv, positions, hd] array of values, and causal attention."""
import numpy as np

BLOCK = 32
CMAX = {"e4m3": 448.0, "int8": 127.0}
E_MIN = -32


def e4m3_values():
    """Value of each e4m3 code (s eeee mmm, bias 7, no infinities, 0x7f / 0xff NaN)."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + f / 8) * 2.0 ** (e - 7), f / 512)
    v[(c & 127) == 127] = np.nan
    return np.where(c > 127, -v, v)


def decode(kind, codes):
    """Values of uint8 codes, scale 1."""
    codes = np.asarray(codes, np.uint8)
    return codes.view(np.int8).astype(np.float64) if kind == "int8" else e4m3_values()[codes]


def encode(kind, x):
    """Code of the nearest value, ties to even, saturating (|x| not NaN)."""
    x = np.clip(np.asarray(x, np.float64), -CMAX[kind], CMAX[kind])
    if kind == "int8":
        return np.rint(x).astype(np.int8).view(np.uint8)
    a = np.abs(x)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    q = np.rint(a / step) * step  # a multiple of the binade's step; the next binade's first value at most
    vals = e4m3_values()[:127]
    code = np.searchsorted(vals, q)
    assert np.array_equal(vals[code], q)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def exponent(kind, amax):
    """Least e >= E_MIN with amax <= CMAX 2^e."""
    e = E_MIN
    while amax > CMAX[kind] * 2.0 ** e:
        e += 1
    return e


def store(kind, codes, scales, x, start):
    """In place on codes uint8 [nkv, positions, hd] and scales [nkv, blocks]: x [M, nkv, hd] at start."""
    M = x.shape[0]
    x = np.asarray(x, np.float64)
    for h in range(codes.shape[0]):
        for b in range(start // BLOCK, (start + M - 1) // BLOCK + 1):
            lo, hi = max(start, b * BLOCK), min(start + M, (b + 1) * BLOCK)
            new = x[lo - start:hi - start, h]
            finite = np.abs(new[np.isfinite(new)])
            s = 2.0 ** exponent(kind, finite.max() if finite.size else 0.0)
            if lo > b * BLOCK and scales[h, b] >= s:
                s = scales[h, b]
            elif lo > b * BLOCK:
                old = decode(kind, codes[h, b * BLOCK:lo]) * float(scales[h, b])
                codes[h, b * BLOCK:lo] = encode(kind, old / s)
            codes[h, lo:hi] = np.where(np.isnan(new), 0, encode(kind, np.nan_to_num(new, nan=0.0, posinf=1e30, neginf=-1e30) / s))
            scales[h, b] = s


def values(kind, codes, scales):
    """[nkv, positions, hd] float64."""
    return decode(kind, codes) * np.repeat(scales.astype(np.float64), BLOCK, axis=1)[:, :codes.shape[1], None]


def attention(q, k, v, start):
    """q [M, nq, hd], k / v [nkv, >= start + M, hd] float64: (out [M, nq, hd], sum p |v|, sum of
    exp(s - max), largest sum |q k| / sqrt(hd)), the last three for the error bound."""
    M, nq, hd = q.shape
    nkv = k.shape[0]
    G, L = nq // nkv, start + M
    out, mag, den = np.zeros((M, nq, hd)), np.zeros((M, nq, hd)), np.zeros((M, nq))
    big = 0.0
    see = np.arange(L)[None, :] <= start + np.arange(M)[:, None]
    for h in range(nq):
        kk, vv = k[h // G, :L], v[h // G, :L]
        s = q[:, h] @ kk.T / np.sqrt(hd)
        big = max(big, float((np.abs(q[:, h]) @ np.abs(kk).T / np.sqrt(hd))[see].max()))
        s = np.where(see, s, -np.inf)
        e = np.exp(s - s.max(1, keepdims=True))
        den[:, h] = e.sum(1)
        p = e / den[:, h, None]
        out[:, h], mag[:, h] = p @ vv, p @ np.abs(vv)
    return out, mag, den, big
