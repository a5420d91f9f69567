"""4-bit floating point in NumPy fp64 (test infrastructure; shares no code with
the library).

Every decision is a comparison of exact numbers: a magnitude against
border * s * t, where border has 3 bits, s (E4M3) 4 and t (fp32) 24, so the
product is exact in fp64; likewise amax against border * 6 * t for the scale.
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(i % 8) * 2.0 ** -9 if i < 8 else (8 + i % 8) * 2.0 ** (i // 8 - 10) for i in range(127)])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def nearest(a, table, unit):
    """Index of the entry of `table` whose multiple of `unit` is nearest to
    a >= 0, ties to the even index, the last one where a is beyond it."""
    k = np.zeros(np.broadcast(a, unit).shape, dtype=np.int64)
    for i in range(len(table) - 1):
        border = (table[i] + table[i + 1]) / 2 * unit
        k += (a > border) | ((a == border) & (i % 2 == 1))
    return k


def quantize(X, fmt, bounds=None, tensor_scale=None):
    """X [rows, n] (exact in fp64), groups of rows between consecutive bounds.
    Returns codes uint8 [rows, nb * B], scale bytes uint8 [rows, nb], t fp32
    [groups] (None for mxfp4) and the values fp32 [rows, n]."""
    X = np.asarray(X, dtype=np.float64)
    rows, n = X.shape
    B = BLOCK[fmt]
    nb = -(-n // B)
    V = np.zeros((rows, nb * B))
    V[:, :n] = X
    V = V.reshape(rows, nb, B)
    bounds = [0, rows] if bounds is None else list(bounds)
    finite = np.isfinite(V)
    bad = ~finite.all(-1)
    A = np.where(finite, np.abs(V), 0.0)
    amax = A.max(-1) if n else np.zeros((rows, nb))
    codes = np.zeros(V.shape, dtype=np.uint8)
    byte = np.zeros((rows, nb), dtype=np.uint8)
    ts = []
    values = np.zeros(V.shape, dtype=np.float32)
    for g, (r0, r1) in enumerate(zip(bounds[:-1], bounds[1:])):
        if fmt == "mxfp4":
            t = np.float32(1)
            m = amax[r0:r1]
            e = np.full(m.shape, -127, dtype=np.int64)
            e[m > 0] = np.frexp(m[m > 0])[1] - 1 - 2
            e = np.clip(e, -127, 127)
            byte[r0:r1] = e + 127
            s = np.ldexp(1.0, e)
        else:
            if tensor_scale is not None:
                t = np.float32(tensor_scale[g])
            else:
                top = amax[r0:r1].max() if r1 > r0 else 0.0
                t = max(np.float32(top) / np.float32(2688), np.float32(2.0 ** -126))
            byte[r0:r1] = nearest(amax[r0:r1], E4M3, 6.0 * np.float64(t))
            s = E4M3[byte[r0:r1]]
        u = (s * np.float64(t))[..., None]
        k = nearest(A[r0:r1], E2M1, u)
        c = k + 8 * np.signbit(V[r0:r1])
        c[np.broadcast_to(u == 0, c.shape)] = 0
        c[bad[r0:r1]] = 0
        codes[r0:r1] = c
        with np.errstate(over="ignore"):
            v = (E2M1[c % 8] * np.where(c // 8, -1.0, 1.0) * s[..., None]).astype(np.float32) * t
        v[bad[r0:r1]] = np.nan
        values[r0:r1] = v
        ts.append(t)
    byte[bad] = 255 if fmt == "mxfp4" else 127
    return (codes.reshape(rows, nb * B), byte, None if fmt == "mxfp4" else np.array(ts, dtype=np.float32),
            values.reshape(rows, nb * B)[:, :n])


def pack(codes, n):
    """Two codes a byte, rows of 16 * ceil(n / 32) bytes."""
    rows = codes.shape[0]
    c = np.zeros((rows, -(-n // 32) * 32), dtype=np.uint8)
    w = min(c.shape[1], codes.shape[1])
    c[:, :w] = codes[:, :w]
    return c[:, 0::2] | c[:, 1::2] << 4


def scale_tiles(byte, bounds):
    """The tiles [bands, quads, 512] of scale bytes [rows, nb], one entry at a time."""
    nb = byte.shape[1]
    quads = -(-nb // 4)
    bands = sum(-(-(b - a) // 128) for a, b in zip(bounds[:-1], bounds[1:]))
    out = np.zeros((bands, quads, 512), dtype=np.uint8)
    first = 0
    for a, b in zip(bounds[:-1], bounds[1:]):
        for r in range(b - a):
            for j in range(nb):
                out[first + r // 128, j // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4] = byte[a + r, j]
        first += -(-(b - a) // 128)
    return out


def unpack(packed, tiles, n, fmt, bounds):
    """code * s of a packed matrix (fp64)."""
    rows = packed.shape[0]
    c = np.empty((rows, 2 * packed.shape[1]), dtype=np.int64)
    c[:, 0::2], c[:, 1::2] = packed & 15, packed >> 4
    v = E2M1[c % 8] * np.where(c // 8, -1.0, 1.0)
    B = BLOCK[fmt]
    j = np.arange(n) // B
    out = np.zeros((rows, n))
    first = 0
    for a, b in zip(bounds[:-1], bounds[1:]):
        r = np.arange(b - a)[:, None]
        byte = tiles[first + r // 128, j[None] // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + j[None] % 4].astype(np.int64)
        if fmt == "mxfp4":
            s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
        else:
            s = np.append(E4M3, np.nan)[byte]
        out[a:b] = v[a:b, :n] * s
        first += -(-(b - a) // 128)
    return out
