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


# ------------------------------------------------------------------------- MoE layer
class Layer:
    """A seeded MoE layer with MX4 experts: codes (one per value), scales, values (float64)."""

    def __init__(self, hidden, inter, n_experts, top_k, seed=0, shared=True, gated=False, bias=False, std=None):
        rng = np.random.default_rng(seed)
        self.hidden, self.inter, self.n_experts, self.top_k = hidden, inter, n_experts, top_k
        H, I, E = hidden, inter, n_experts

        def mat(rows, cols):
            w = rng.standard_normal((rows, cols)) * np.exp(0.5 * rng.standard_normal((rows, 1))) / np.sqrt(cols)
            c, s = quantize(w)
            return c, s, values(c, s)

        def bf16(v):
            f = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
            return ((f + 0x7FFF + ((f >> 16) & 1)) >> 16).astype(np.uint16)

        self.router_bits = bf16(rng.standard_normal((E, H)) / np.sqrt(H) * (std or 1.0))
        self.bias = (-1.1 * np.log(rng.permutation(E) + 1.0)).astype(np.float32) if bias else None
        self.gate_up, self.down = mat(E * 2 * I, H), mat(E * H, I)
        self.shared = (mat(2 * I, H), mat(H, I)) if shared else None
        self.gate_bits = bf16(rng.standard_normal(H) / np.sqrt(H)) if gated else None

    def logits(self, x):
        l = x @ bf16_values(self.router_bits).T
        return l if self.bias is None else l + self.bias.astype(np.float64)

    def route(self, x):
        """(idx ascending, gap between the k-th and the next logit) of float64 x [T, H]."""
        l = self.logits(x)
        order = np.argsort(-l, axis=1, kind="stable")
        k = self.top_k
        srt = np.take_along_axis(l, order, axis=1)
        gap = srt[:, k - 1] - srt[:, k] if k < l.shape[1] else np.full(len(l), np.inf)
        return np.sort(order[:, :k], axis=1), gap

    def weights(self, x, idx):
        part = np.take_along_axis(self.logits(x), idx, axis=1)
        w = np.exp(part - part.max(axis=1, keepdims=True))
        return w / w.sum(axis=1, keepdims=True)

    def forward(self, x, idx, prompt=False):
        """(y, error bound of the fp32 evaluation) for float64 x and a routing.

        The bound follows a value through the layer: g and u are sums as in product_bound;
        silu moves by at most 1.1 of its argument's error and is evaluated to 2^-16 of itself
        (the argument of its exponential, up to 2^6, is rounded once: 2^-18, and a few fp32
        roundings); h = w silu(g) u is kept to 2^-16 (a bf16 pair), w is off by twice the
        logits' error and 2^-20; the down sums as in product_bound, over all experts.  prompt: each
        expert's weighted output passes through fp16 (half a step, 2^-11 of it), flushed to zero
        below 2^-14 where the largest of its 64 columns is at least 2^-2, so by at most 2^-12 of
        that largest value (smaller ones are scaled up to 2^14 and lose less)."""
        H, I, T = self.hidden, self.inter, x.shape[0]
        w = self.weights(x, idx)
        dl = product_bound(x, bf16_values(self.router_bits)).max(axis=1)
        y, b, tot = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))

        def expert(t, gu, dn, wt, dw):
            xs = x[t]
            g, u = xs @ gu[:I].T, xs @ gu[I:].T
            dg, du = product_bound(xs, gu[:I]), product_bound(xs, gu[I:])
            s = g / (1 + np.exp(-g))
            h = wt[:, None] * s * u
            if prompt:
                o = np.abs(h @ dn.T)
                big = o.reshape(len(t), -1, 64).max(axis=2)
                b[t] += 2.0 ** -11 * o + np.repeat(2.0 ** -12 * big, 64, axis=1)
            dh = np.abs(wt)[:, None] * (1.1 * dg * np.abs(u) + np.abs(s) * du + 1.1 * dg * du)
            dh += np.abs(h) * (2.0 ** -15 + dw[:, None])
            y[t] += h @ dn.T
            b[t] += dh @ np.abs(dn).T
            tot[t] += np.abs(h) @ np.abs(dn).T

        for e in np.unique(idx):
            t, j = np.nonzero(idx == e)
            expert(t, self.gate_up[2][e * 2 * I:(e + 1) * 2 * I], self.down[2][e * H:(e + 1) * H], w[t, j],
                   2 * dl[t] + 2.0 ** -20)
        if self.shared:
            wt = np.ones(T)
            if self.gate_bits is not None:
                wt = 1 / (1 + np.exp(-(x @ bf16_values(self.gate_bits))))
            expert(np.arange(T), self.shared[0][2], self.shared[1][2], wt, 2 * dl + 2.0 ** -18)
        n = 4 * -(-I // 128) * (self.top_k + 1) + 16 + 2
        return y, b + n * 2.0 ** -23 * tot
