"""Plain 64-bit implementation of the routing rules, one token at a time, written from their
definition (moe_router_rule).  Test infrastructure: shares no code with the library."""
import numpy as np

import mx4_ref


def select(logits, k, score="softmax", renorm=True, n_groups=1, group_top_k=1, group_score="max", scale=1.0,
           select_bias=None):
    """(idx [T, k] ascending, w [T, k], gap [T]) for float64 logits [T, E].

    gap: how far the selection is from another one -- the smaller of the distances between the
    last expert (group) taken and the first one left, in selection values (0 for ties)."""
    T, E = logits.shape
    idx, w, gap = np.zeros((T, k), np.int64), np.zeros((T, k)), np.full(T, np.inf)
    for t in range(T):
        l = logits[t]
        with np.errstate(all="ignore"):
            live = l > -np.inf
            s = np.zeros(E)
            if score == "sigmoid":
                s[live] = 1.0 / (1.0 + np.exp(-l[live]))
            elif live.any():
                top = l[live].max()
                s[live] = np.where(l[live] == top, 1.0, np.exp(l[live] - top))
                s /= s.sum()
            c, g = l.copy(), s.copy()
            if select_bias is not None:
                c = g = s + select_bias
                live = live & (c > -np.inf)
            if group_score == "max":
                g = c
        c = np.where(live, c, -np.inf)
        g = np.where(live, g, -np.inf)
        groups = list(range(n_groups))
        size = E // n_groups
        if group_top_k < n_groups:
            worth = []
            for j in groups:
                two = sorted(g[j * size:(j + 1) * size], reverse=True)[:2]
                worth.append(two[0] + two[1] if group_score == "top2" and size > 1 and two[1] > -np.inf else two[0])
            order = sorted(groups, key=lambda j: -worth[j])          # (stable: ties to the lower group)
            a, b = worth[order[group_top_k - 1]], worth[order[group_top_k]]
            gap[t] = a - b if b > -np.inf else gap[t]
            groups = order[:group_top_k]
        cand = [e for e in range(E) if e // size in groups]
        order = sorted(cand, key=lambda e: -c[e])
        if len(order) > k and c[order[k]] > -np.inf:
            gap[t] = min(gap[t], c[order[k - 1]] - c[order[k]])
        idx[t] = np.sort(order[:k])
        v = np.where(live, s, 0.0)[idx[t]]
        if renorm:
            v = v / v.sum() if v.sum() > 0 else np.zeros(k)
        w[t] = v * np.float64(np.float32(scale))
    return idx.astype(np.int32), w, gap


class RuledLayer:
    """mx4_ref.Layer under a routing rule."""

    def __new__(cls, rule, **kw):
        class Ruled(mx4_ref.Layer):
            def route(self, x):
                i, _, gap = select(self.logits(x), self.top_k, **rule)
                return i, gap

            def weights(self, x, idx):
                return weights_of(self.logits(x), idx, **rule)

        return Ruled(**kw)


def weights_of(logits, idx, score="softmax", renorm=True, scale=1.0, **_):
    """The weights of a given selection (all experts live)."""
    if score == "sigmoid":
        s = 1.0 / (1.0 + np.exp(-logits))
    else:
        e = np.exp(logits - logits.max(axis=1, keepdims=True))
        s = e / e.sum(axis=1, keepdims=True)
    w = np.take_along_axis(s, idx.astype(np.int64), axis=1)
    return (w / w.sum(axis=1, keepdims=True) if renorm else w) * np.float64(np.float32(scale))
