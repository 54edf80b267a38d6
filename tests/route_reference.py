"""A router's choice and its gradient from the definition, in 64 bits (numpy)."""
import numpy as np


def scores(l, sigmoid):
    with np.errstate(all="ignore"):
        if sigmoid:
            e = np.exp(-np.abs(l))
            return np.where(l >= 0, 1.0, e) / (1 + e)
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
        return e / np.maximum(e.sum(1, keepdims=True), np.finfo(float).tiny)


def _rank(row):
    """Indices, largest first, NaN above all, ties to the lowest index; -inf left out."""
    order = sorted(range(len(row)), key=lambda i: (not np.isnan(row[i]), 0.0 if np.isnan(row[i]) else -row[i], i))
    return [i for i in order if not row[i] == -np.inf]


def route(l, topk, sigmoid, renorm, scale, bias=None, groups=1, topk_groups=1, group_best=2):
    tokens, experts = l.shape
    s = scores(l, sigmoid)
    with np.errstate(all="ignore"):
        c = l.copy() if bias is None else np.where(np.isneginf(l), -np.inf, s + bias)
    size = experts // groups
    expert = np.full((tokens, topk), -1, np.int64)
    weight = np.zeros((tokens, topk))
    for t in range(tokens):
        row = c[t].copy()
        if groups > 1:
            by = row if bias is not None or group_best == 1 else np.where(np.isneginf(l[t]), -np.inf, s[t])
            total = np.full(groups, -np.inf)
            for g in range(groups):
                part = by[g * size:(g + 1) * size]
                best = _rank(part)[:group_best]
                if best:
                    total[g] = sum(part[i] for i in best)
            stay = _rank(total)[:topk_groups]
            for g in range(groups):
                if g not in stay:
                    row[g * size:(g + 1) * size] = -np.inf
        best = _rank(row)[:topk]
        expert[t, :len(best)] = best
        chosen = s[t, best]
        total = chosen.sum() if renorm else 1.0
        with np.errstate(all="ignore"):
            weight[t, :len(best)] = scale * chosen / (total if total != 0 else 1.0)
    return expert, weight


def route_grad(l, expert, d_weight, sigmoid, renorm, scale):
    """(gradient of the logits, a bound of the size of what is summed for it)."""
    tokens, experts = l.shape
    s = scores(l, sigmoid)
    d, size = np.zeros_like(l), np.zeros_like(l)
    for t in range(tokens):
        slots = [j for j in range(expert.shape[1]) if 0 <= expert[t, j] < experts]
        e = expert[t, slots]
        p, g = s[t, e], d_weight[t, slots]
        total = p.sum() if renorm else 1.0
        total = total if total != 0 else 1.0
        ds, big = np.zeros(experts), np.zeros(experts)
        mean, most = ((g * p).sum() / total, (np.abs(g) * p).sum() / total) if renorm else (0.0, 0.0)
        np.add.at(ds, e, scale / total * (g - mean))
        np.add.at(big, e, abs(scale) / total * (np.abs(g) + most))
        if sigmoid:
            slope = s[t] * scores(-l[t:t + 1], True)[0]
            d[t], size[t] = ds * slope, big * slope
        else:
            # renormalised, sum s ds = scale / S (sum s g - mean sum s) = 0, of which 64 bits would leave a rounding error
            d[t] = s[t] * (ds - (0.0 if renorm else (s[t] * ds).sum()))
            size[t] = s[t] * (big + (0.0 if renorm else (s[t] * big).sum()))
    return d, size
