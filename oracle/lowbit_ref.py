"""Plain NumPy definitions of the 4-bit rows and the low-bit cache, in float64.

Test infrastructure only; nothing here is shared with the package.  Decisions that are
float32 by definition (a grid's scale, its quotients) are rounded to float32 once.
"""
import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


# ------------------------------------------------------------------ microscaled rows
def mx_quantize(x):
    """(codes (R, 32 nb) uint8, e (R, nb) uint8) of x (R, C) float64; not-finite blocks get 255."""
    R, C = x.shape
    nb = -(-C // 32)
    p = np.zeros((R, nb * 32))
    p[:, :C] = x
    b = p.reshape(R, nb, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    # floor(log2 top): frexp gives top = m 2^k with m in [0.5, 1)
    k = np.frexp(top)[1] - 1
    e = np.where(top > 0, np.maximum(k - 2, -127), -127) + 127
    y = np.abs(b) / np.exp2(e.astype(np.float64) - 127)[..., None]
    dist = np.abs(np.minimum(y, 6.0)[..., None] - LEVELS)
    best = dist.min(-1)
    near = dist == best[..., None]                     # one level, or two at a tie
    even = near & (np.arange(8) % 2 == 0)
    idx = np.where(near.sum(-1) == 2, even.argmax(-1), near.argmax(-1))
    codes = (idx | (np.signbit(b).astype(np.int64) << 3)).astype(np.uint8)
    codes[bad] = 0
    e = np.where(bad, 255, e).astype(np.uint8)
    return codes.reshape(R, nb * 32), e


def mx_values(codes, e):
    """float64 values of codes (R, 32 nb) and scales e (R, nb); NaN where e = 255."""
    v = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(e == 255, np.nan, np.exp2(e.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)


def mx_scale_index(row, block, nb):
    """Byte of (row, block) in the tiled scales of rows with nb blocks."""
    return ((row // 128) * (-(-nb // 4)) + block // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + block % 4


def mx_tile(e, fill=0):
    """Scales e (R, nb) in their tiles, a flat uint8 array; `fill` where no row is."""
    R, nb = e.shape
    out = np.full((-(-R // 128)) * (-(-nb // 4)) * 512, fill, dtype=np.uint8)
    for r in range(R):
        for k in range(-(-nb // 4) * 4):
            out[mx_scale_index(r, k, nb)] = e[r, k] if k < nb else 0
    return out


# ------------------------------------------------------------------ integer grids
def grid_quantize(x, bits, group, sym):
    """(codes (.., D) int64, s (.., G) float32, z (.., G) float32) of x (.., D) float64 holding
    float32 values; not-finite groups get s = NaN, z = 0 and codes 0."""
    f32 = np.float32
    D = x.shape[-1]
    g = group if group > 0 else D
    G = -(-D // g)
    maxq = 2 ** bits - 1
    codes = np.zeros(x.shape, dtype=np.int64)
    S = np.zeros(x.shape[:-1] + (G,), dtype=f32)
    Z = np.zeros_like(S)
    with np.errstate(all="ignore"):
        for i in range(G):
            v = x[..., i * g:(i + 1) * g]
            bad = ~np.isfinite(v).all(-1)
            lo, hi = np.minimum(v.min(-1), 0.0), np.maximum(v.max(-1), 0.0)

            def grid(lo, hi):
                if sym:
                    m = np.maximum(-lo, hi)
                    m = np.where(m == 0, 1.0, m)
                    return f32(f32(2 * m) / np.float64(maxq)), np.full(lo.shape, f32(2 ** (bits - 1)))
                flat = (lo == 0) & (hi == 0)
                lo, hi = np.where(flat, -1.0, lo), np.where(flat, 1.0, hi)
                s = f32(f32(hi - lo) / np.float64(maxq))
                return s, np.rint(f32(-lo / s.astype(np.float64)))

            s, z = grid(lo, hi)
            s1, z1 = grid(np.full_like(lo, -1.0), np.full_like(hi, 1.0))
            under = s == 0
            s, z = np.where(under, s1, s), np.where(under, z1, z)
            q = np.rint(f32(v / s.astype(np.float64)[..., None]))
            c = np.clip(q.astype(np.float64) + z[..., None], 0, maxq)
            bad = bad | ~np.isfinite(s)
            codes[..., i * g:(i + 1) * g] = np.where(bad[..., None], 0, np.nan_to_num(c)).astype(np.int64)
            S[..., i] = np.where(bad, f32(np.nan), s)
            Z[..., i] = np.where(bad, f32(0), z)
    return codes, S, Z


def grid_values(codes, S, Z, group):
    """float64 values s (code - z)."""
    D = codes.shape[-1]
    of = np.arange(D) // (group if group > 0 else D)
    return S.astype(np.float64)[..., of] * (codes - Z.astype(np.float64)[..., of])


# ------------------------------------------------------------------ rows of a call
def slots(tokens, table, cu, start, page_size, pages):
    """Slot of each row: -1 for padding, -2 for a position or page out of range."""
    out = np.full(tokens, -1, dtype=np.int64)
    for s in range(len(start)):
        for t in range(cu[s], min(cu[s + 1], tokens)):
            pos = int(start[s]) + t - int(cu[s])
            out[t] = -2
            if start[s] >= 0 and pos // page_size < table.shape[1]:
                page = int(table[s, pos // page_size])
                if 0 <= page < pages:
                    out[t] = page * page_size + pos % page_size
    return out
