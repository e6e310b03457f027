"""Plain 64-bit evaluation of lora_gemm with an error bound, written from its definition.  Test
infrastructure: shares no code with the library.

Bound: a product of two bf16 values is exact; a value of A x goes through at most one matrix
instruction per 32 columns and 16 partial sums, with a tree over 32 columns inside, each taken as an
fp32 step that rounds (or cuts off) less than 2^-23 of the magnitudes summed so far.  It is scaled
(half a step, 2^-24), and kept as bf16 parts, each leaving at most 2^-8 of what was left: two for a bf16
y, three for an fp32 one; a part below 2^-126 may be flushed.  The second product likewise, then the
addition of base (2^-24), and y's own rounding (2^-8 or 2^-24)."""
import numpy as np


def forward(a, b, ids, x, base, scales=None, ranks=None, f32=False):
    """(y, bound): float64 a [n, R, K], b [n, N, R], x [T, K], base [T, N] or None."""
    n, R, K = a.shape
    T, N = x.shape[0], b.shape[1]
    parts = 3 if f32 else 2
    y = np.zeros((T, N)) if base is None else base.copy()
    bound = np.zeros((T, N))
    for t in range(T):
        i = int(ids[t])
        if not 0 <= i < n:
            continue
        r = R if ranks is None else min(max(int(ranks[i]), 0), R)
        s = 1.0 if scales is None else float(scales[i])
        A, B = a[i, :r], b[i, :, :r]
        v, mag = A @ x[t], np.abs(A) @ np.abs(x[t])
        dv = (-(-K // 32) + 16 + 32) * 2.0 ** -23 * mag * abs(s)
        v = v * s
        dv = dv + (2.0 ** -24 + 2.0 ** (-8 * parts)) * (np.abs(v) + dv) + parts * 2.0 ** -126
        y[t] += B @ v
        aB = np.abs(B)
        bound[t] = aB @ dv + (-(-parts * R // 32) + 32) * 2.0 ** -23 * (aB @ (np.abs(v) + dv))
        bound[t] += 2.0 ** -24 * (np.abs(y[t]) + bound[t])
    return y, bound


def check(got, y, bound, bf16, what=None):
    half = 2.0 ** -8 if bf16 else 0.0            # (an fp32 y: the addition's own rounding)
    err, lim = np.abs(got - y), bound + half * (np.abs(y) + bound) + 2.0 ** -133
    assert (err <= lim).all(), (what, float((err / lim).max()))
