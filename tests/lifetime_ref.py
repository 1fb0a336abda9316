"""Plain 64-bit (and wider) references of the cache-lifetime operators:
rotary positions, running attention weights, eviction.  numpy only; they
share no code with the kernels."""
import numpy as np

BLOCK = 16


def rotate(x, positions, frequencies, axis, rotary_dim, interleaved):
    """x float64 [T, H, d] turned by positions int [A, T]; angles in extended
    precision.  Returns (turned, |x| + |y| of each element's pair)."""
    y = np.array(x, dtype=np.float64)
    mag = np.zeros_like(y)
    R = rotary_dim
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        ang = np.asarray(positions[axis[i]], dtype=np.longdouble) * np.longdouble(frequencies[i])
        c = np.cos(ang).astype(np.float64)[:, None]
        s = np.sin(ang).astype(np.float64)[:, None]
        u, w = x[:, :, a], x[:, :, b]
        y[:, :, a] = u * c - w * s
        y[:, :, b] = u * s + w * c
        mag[:, :, a] = mag[:, :, b] = np.abs(u) + np.abs(w)
    return y, mag


def e4m3_table():
    """The 256 E4M3 values (NaN for S.1111.111)."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = np.nan if (e == 15 and m == 7) else \
            (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = -x if s else x
    return v


E4M3 = e4m3_table()


def attention_weights(q, k, v, scale):
    """q [G, d], k and v [L, d] float64: (out [G, d], summed weights [L],
    largest |q| . |k| scale of a score)."""
    if k.shape[0] == 0:
        return np.zeros_like(q), np.zeros((0,)), 0.0
    s = scale * (q @ k.T)
    e = np.exp(s - s.max(axis=1, keepdims=True))
    p = e / e.sum(axis=1, keepdims=True)
    bound = float((abs(scale) * (np.abs(q) @ np.abs(k).T)).max())
    return p @ v, p.sum(axis=0), bound


def weights_tolerance(d, L, group, bound):
    """Bound on the error of a token's summed weight, relative to the sum's
    exact value.  A score is d products added in binary32 (each addition off
    by at most one unit, 2^-23 of the magnitudes' sum, so d 2^-23 bound), its
    conversion to log2 units and the subtraction of the maximum add 4 roundings
    of at most bound; a weight moves by e^(2 error) with the error of its
    score and of the maximum's; exp2 and the divisions add 8 roundings, the
    row sum and the sum over heads one each per term."""
    score = bound * (d * 2.0 ** -23 + 4 * 2.0 ** -24)
    return 2 * score + (8 + L + group) * 2.0 ** -24


def evict_choice(w, L, keep, sink, recent):
    """Positions one head keeps, ascending: w float32 [>= L] ranks."""
    n = min(L, keep)
    r = min(recent, n)
    f = min(sink, n - r)
    mid = list(range(f, L - r))

    def rank(t):  # larger first, lower position first, NaN last
        x = float(w[t])
        return (1, 0.0, t) if x != x else (0, -x, t)
    best = sorted(mid, key=rank)[:n - r - f]
    return list(range(f)) + sorted(best) + list(range(L - r, L))


def heads_sum(w):
    """fp32 [H, S] -> the heads' sum, in binary64 head by head, rounded once."""
    s = np.zeros(w.shape[1], dtype=np.float64)
    with np.errstate(all="ignore"):
        for h in range(w.shape[0]):
            s = s + w[h].astype(np.float64)
        return s.astype(np.float32)
