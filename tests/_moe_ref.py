"""Plain 64-bit references of the mixture-of-experts operators (numpy, one definition each)."""
import numpy as np

SUM_FLOOR = 2.0 ** -126


def scores(z, score):
    """softmax of each row, or the sigmoid; -inf logits give 0."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        top = z.max(axis=1, keepdims=True)
        x = np.where(np.isneginf(z), 0.0, np.exp(z - np.where(np.isfinite(top), top, 0.0)))
        total = x.sum(axis=1, keepdims=True)
        return x / np.where(total > 0, total, 1.0)


def route(z, k, score="softmax", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """weights [T, k] float64 and ids [T, k] int32, token by token."""
    z = np.asarray(z, dtype=np.float64)
    T, E = z.shape
    size = E // groups
    p_all = scores(z, score)
    weights, ids = np.zeros((T, k)), np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        if np.isnan(z[t]).any() or (score == "softmax" and np.isposinf(z[t]).any()):
            weights[t] = np.nan
            continue
        key = z[t].copy() if bias is None else p_all[t] + np.asarray(bias, dtype=np.float64)
        key[np.isneginf(z[t]) | np.isnan(key)] = -np.inf
        if groups > 1:
            value = []
            for g in range(groups):
                best = sorted(key[g * size:(g + 1) * size], reverse=True)
                two = bias is not None and size > 1 and best[1] != -np.inf
                value.append(best[0] + best[1] if two else best[0])
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            for g in range(groups):
                if g not in kept:
                    key[g * size:(g + 1) * size] = -np.inf
        order = [e for e in np.argsort(-key, kind="stable") if key[e] != -np.inf][:k]
        n = len(order)
        ids[t, :n] = order
        if n == 0:
            continue
        if score == "softmax" and renormalize:
            x = np.exp(z[t, order] - z[t, order].max())
            weights[t, :n] = scale * x / x.sum()
        else:
            p = p_all[t, order]
            weights[t, :n] = scale * p / (max(p.sum(), SUM_FLOOR) if renormalize else 1.0)
    return weights, ids


def route_backward(z, ids, dw, score="softmax", renormalize=True, scale=1.0):
    """dlogits [T, E] float64, and for each row the sum of the magnitudes that enter it (for error
    bounds)."""
    z, dw = np.asarray(z, dtype=np.float64), np.asarray(dw, dtype=np.float64)
    T, E = z.shape
    p_all = scores(z, score)
    dz, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        at = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not at:
            continue
        e, d = ids[t, at], dw[t, at]
        if score == "softmax" and renormalize:
            x = np.exp(z[t, e] - z[t, e].max())
            q = x / x.sum()
            np.add.at(dz[t], e, scale * q * (d - (q * d).sum()))
            np.add.at(size[t], e, abs(scale) * q * (abs(d) + (q * abs(d)).sum()))
        elif score == "softmax":
            p = p_all[t]
            dp = np.zeros(E)
            np.add.at(dp, e, scale * d)
            dz[t] = p * (dp - (dp * p).sum())
            size[t] = p * (abs(dp) + (abs(dp) * p).sum())
        else:
            p = p_all[t, e]
            g, a = scale * d, abs(scale * d)
            if renormalize:
                D = max(p.sum(), SUM_FLOOR)
                live = p.sum() >= SUM_FLOOR
                g = scale * (d - (d * p).sum() / D * live) / D
                a = abs(scale) * (abs(d) + (abs(d) * p).sum() / D) / D
            np.add.at(dz[t], e, g * p * (1 / (1 + np.exp(z[t, e]))))
            np.add.at(size[t], e, a * p)
    return dz, size


def plan(ids, E):
    """offsets, slots, rows of the stable sort by expert."""
    flat = ids.reshape(-1).astype(np.int64)
    bins = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(bins, kind="stable")
    offsets = np.searchsorted(bins[order], np.arange(E + 1)).astype(np.int64)
    place = np.arange(flat.size)
    slots = np.empty(flat.size, dtype=np.int32)
    slots[order] = np.where(place < offsets[E], place, -1 - place)
    rows = np.where(place < offsets[E], order, -1).astype(np.int32)
    return offsets, slots.reshape(ids.shape), rows


def combine(rows, slots, weights):
    """y [T, H] float64 and the sums of magnitudes; rows as float64."""
    T, k = slots.shape
    y, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            w = 1.0 if weights is None else float(weights[t, j])
            if 0 <= slots[t, j] < rows.shape[0]:
                y[t] += w * rows[slots[t, j]]
                size[t] += abs(w * rows[slots[t, j]])
            else:
                y[t] += w * 0.0
    return y, size


def choose(g, T, k, E, dropped=0.0):
    """[T, k] int32 distinct experts of each token, some replaced by ids that name no expert."""
    ids = np.argsort(g.standard_normal((T, E)) + 0.7 * g.standard_normal(E), axis=1)[:, :k].astype(np.int32)
    if dropped:
        bad = np.array([-1, E, -2 ** 31, 2 ** 31 - 1, E + 5], dtype=np.int64).astype(np.int32)
        hit = g.random((T, k)) < dropped
        ids = np.where(hit, bad[g.integers(0, len(bad), (T, k))], ids)
    return np.ascontiguousarray(ids)
