"""Plain 64-bit numpy implementation of the MX4 format, its layouts and products, written
from the format's definition (FP4 E2M1 elements, blocks of 32, E8M0 scales).  Test
infrastructure: shares no code with the library."""
import numpy as np

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])      # E2M1 magnitudes by code
BLOCK = 32


def bf16_values(bits):
    """float64 values of bf16 bit patterns."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def floor_log2(a):
    """floor(log2 a) of positive float64 values, exactly."""
    return np.frexp(a)[1] - 1


def quantize(x):
    """float64 [rows, K] -> codes uint8 [rows, K] (one per value) and scales [rows, K/32].
    Nearest magnitude by distance, ties to the code whose last bit is 0."""
    rows, K = x.shape
    b = x.reshape(rows, K // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    a = np.abs(np.where(bad[..., None], 0.0, b))
    big = a.max(axis=2)
    e = np.where(big > 0, floor_log2(np.where(big > 0, big, 1.0)) - 2, -127)
    e = np.clip(e, -127, 127)
    v = np.ldexp(a, -e[..., None])
    d = np.abs(v[..., None] - MAG)                              # distance to every magnitude
    near = d == d.min(axis=3, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(near.sum(axis=3) > 1, even.argmax(axis=3), near.argmax(axis=3))
    code = code + 8 * np.signbit(np.where(bad[..., None], 0.0, b))
    scale = np.where(bad, 255, e + 127)
    return code.reshape(rows, K).astype(np.uint8), scale.astype(np.uint8)


def values(codes, scales):
    """float64 values of one-per-value codes [..., K] and scales [..., K/32]."""
    m = np.where(codes & 8, -1.0, 1.0) * MAG[codes & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return m * np.repeat(s, BLOCK, axis=-1)


def pack_rows(codes):
    """Two codes a byte, even columns in the low nibble."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack_rows(packed):
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def to_tiles(codes, scales):
    """The tile layout of codes [rows, K] and scales [rows, K/32], entry by entry."""
    rows, K = codes.shape
    P, S = -(-rows // 16), -(-K // 128)
    Q = -(-S // 4)
    c = np.zeros((16 * P, 128 * S), np.uint8)
    c[:rows, :K] = codes
    s = np.zeros((16 * P, 16 * Q), np.uint8)
    s[:rows, :K // BLOCK] = scales
    tc = np.zeros((P, S, 64, 16), np.uint8)
    ts = np.zeros((P, Q, 64, 4), np.uint8)
    pk = pack_rows(c)
    for n in range(16):
        for g in range(4):
            for st in range(S):
                tc[:, st, n + 16 * g] = pk[n::16, 64 * st + 16 * g:64 * st + 16 * g + 16]
            for q in range(Q):
                for i in range(4):
                    ts[:, q, n + 16 * g, i] = s[n::16, 4 * (4 * q + i) + g]
    return tc.reshape(-1), ts.reshape(-1)


def product_bound(x, w):
    """Error bound of the products' fp32 sums.  Every product is exact (8 + 2 significant
    bits).  A value goes through at most 4 matrix instructions per 128 columns in a row, up
    to 16 partial sums, and inside an instruction a tree over its columns: each is taken as one
    fp32 step that rounds (or cuts off) less than 2^-23 of what has been summed in magnitude,
    of which |x| @ |w| is a bound."""
    n = 4 * -(-x.shape[1] // 128) + 16 + 2
    return n * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
