"""Plain 64-bit evaluation of moe_block_norm with an error bound of its fp32 evaluation, written from
its definition.  Test infrastructure: shares no code with the library.

Bound, with u = 2^-24 (half a step of fp32, what one operation rounds by, relative to its result):
a sum of n <= 16384 values is a chain of at most 18 additions in a thread and 26 more across threads,
so it is off by at most SUM u of the sum of magnitudes, SUM = 64."""
import numpy as np

U, SUM = 2.0 ** -24, 64
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}       # half a step, relative
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}    # (at least) the spacing of subnormals


def norm(v, bv, kind, eps, offset, weight, bias):
    """(norm of rows v, its error bound) for rows v known to within bv."""
    c, bc = v, bv
    if kind == "layer":
        m = v.mean(axis=1, keepdims=True)
        dm = (SUM + 2) * U * np.abs(v).mean(axis=1, keepdims=True) * 1.01 + bv.mean(axis=1, keepdims=True)
        c = v - m
        bc = bv + dm + U * np.abs(c) * 1.01
    q = (c * c).mean(axis=1, keepdims=True) + eps
    dq = (2 * np.abs(c) * bc + bc * bc).mean(axis=1, keepdims=True) + (SUM + 4) * U * ((np.abs(c) + bc) ** 2).mean(
        axis=1, keepdims=True) + 2 * U * q
    rel = dq / (2 * np.maximum(q - dq, 1e-300)) + 3 * U                  # of 1 / sqrt
    s = np.sqrt(q)
    gain = np.ones_like(v[:1]) if weight is None else offset + weight[None]
    out = c / s * gain
    b = np.abs(gain) / s * (bc * (1 + rel) + np.abs(c) * rel) + 4 * U * np.abs(out)
    if bias is not None:
        out = out + bias[None]
        b = b + U * (np.abs(out) + b)
    return out, b


def block(y, r, post, gate, act, scale, pre):
    """((r', bound), (x, bound)); post and pre are dicts of norm's arguments or None."""
    scale = float(np.float32(scale))
    if y is None:
        t, b = r, np.zeros_like(r)
    else:
        z, b = y, np.zeros_like(y)
        if post:
            z, b = norm(z, b, **post)
        if gate is not None:
            with np.errstate(over="ignore"):
                s = 1 / (1 + np.exp(-gate))
            # exp within 2 steps (4 u, and its argument is exact), a sum, a quotient, a product; below
            # fp32's range it is 0
            g, dg = {"none": (gate, 0 * gate), "sigmoid": (s, 10 * U * s + 2.0 ** -125),
                     "silu": (gate * s, 12 * U * np.abs(gate * s) + 2.0 ** -125 * (1 + np.abs(gate)))}[act]
            b = b * (np.abs(g) + dg) + np.abs(z) * dg + 2 * U * np.abs(z * g)
            z = z * g
        z, b = z * scale, np.abs(scale) * b + 2 * U * np.abs(z * scale)
        t = z if r is None else r + z
        b = b + U * (np.abs(t) + b)
    return (t, b), (norm(t, b, **pre) if pre else (None, None))


def rounded(v, b, dtype):
    """The bound of v stored in dtype."""
    return b + HALF[dtype] * (np.abs(v) + b) + TINY[dtype]
