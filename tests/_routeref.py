"""The routing's definitions in 64 bits, a token at a time (numpy; no code of the package)."""
import math

import numpy as np


def rank(values, n):
    """Indices of the n largest, ties to the lowest index; -inf is never among them."""
    live = [i for i, v in enumerate(values) if not v == -math.inf]
    return sorted(live, key=lambda i: (not math.isnan(values[i]), -values[i] if not math.isnan(values[i]) else 0.0, i))[:n]


def sigmoid(x):
    if math.isnan(x):
        return x
    return 1 / (1 + math.exp(-x)) if x >= 0 else math.exp(x) / (1 + math.exp(x)) if x > -700 else 0.0


def softmax(v):
    m = max(v)
    if any(math.isnan(x) for x in v) or m == math.inf:
        return [math.nan] * len(v)
    e = [math.exp(x - m) for x in v]
    t = math.fsum(e)
    return [x / t for x in e]


def select(l, k, score, bias=None, groups=1, top_groups=None, group_score="top2"):
    """The experts of one token with logits l (floats)."""
    E = len(l)
    scores = [float(x) for x in l]
    if score == "sigmoid":
        scores = [sigmoid(x) for x in scores]
    elif score == "softmax_all":
        live = [x for x in scores if x != -math.inf]
        p = softmax(live) if live else []
        it = iter(p)
        scores = [next(it) if x != -math.inf else 0.0 for x in scores]
    # without a bias, and with one that is the same for all, the order is the logits'
    same = bias is None or (len(set(float(b) for b in bias)) == 1 and math.isfinite(float(bias[0])))
    key = [float(x) for x in l] if same else [x + float(b) for x, b in zip(scores, bias)]
    key = [-math.inf if x == -math.inf else v for x, v in zip(l, key)]
    value = [float(x) for x in (scores if same else key)]  # what a group's sum is of
    if groups > 1:
        n = E // groups
        worth = []
        for g in range(groups):
            part = key[g * n:(g + 1) * n]
            if group_score == "max":
                best = [part[i] for i in rank(part, 1)]
            else:
                best = [value[g * n + i] for i in rank(part, 2)]
            worth.append(sum(best) if best else -math.inf)
        stay = rank(worth, top_groups)
        key = [v if i // n in stay else -math.inf for i, v in enumerate(key)]
    return rank(key, k)


def weights(l, chosen, score, renormalize=False, scale=1.0):
    l = [float(x) for x in l]
    if not chosen:
        return []
    if score == "softmax" or (score == "softmax_all" and renormalize):
        w = softmax([l[e] for e in chosen])
    elif score == "softmax_all":
        live = [x for x in l if x != -math.inf]
        p = dict(zip([i for i, x in enumerate(l) if x != -math.inf], softmax(live)))
        w = [p[e] for e in chosen]
    else:
        w = [sigmoid(l[e]) for e in chosen]
        if renormalize:  # by logarithms, so that tiny scores keep their quotients
            a = [-math.log1p(math.exp(-l[e])) if l[e] > 0 else l[e] - math.log1p(math.exp(l[e])) for e in chosen]
            w = softmax(a)
    return [x * scale for x in w]


def gradient(l, chosen, dw, score, renormalize=False, scale=1.0):
    """dlogits of one token, by the formulas' Jacobian written out."""
    E = len(l)
    l = [float(x) for x in l]
    out = np.zeros(E)
    w = weights(l, chosen, score, renormalize, 1.0)
    d = [x * scale for x in dw[:len(chosen)]]
    if score == "softmax_all" and not renormalize:
        if not chosen:
            return out
        p = [w_ for w_ in weights(l, list(range(E)), score)] if all(x != -math.inf for x in l) else None
        if p is None:
            live = [i for i in range(E) if l[i] != -math.inf]
            q = weights(l, live, score)
            p = [0.0] * E
            for i, v in zip(live, q):
                p[i] = v
        for j, e in enumerate(chosen):
            for i in range(E):
                out[i] += d[j] * p[e] * ((1.0 if i == e else 0.0) - p[i])
        return out
    if score == "sigmoid" and not renormalize:
        for j, e in enumerate(chosen):
            out[e] += d[j] * w[j] * sigmoid(-l[e])
        return out
    for j in range(len(chosen)):
        for i, e in enumerate(chosen):
            slope = sigmoid(-l[e]) if score == "sigmoid" else 1.0
            out[e] += d[j] * w[j] * ((1.0 if i == j else 0.0) - w[i]) * slope
    return out


def plan(experts, E, multiple):
    """offs, counts, rows by group (lists of choices) of experts [T, k]."""
    flat = [int(e) for e in np.asarray(experts).reshape(-1)]
    groups = [[i for i, e in enumerate(flat) if e == g] for g in range(E)]
    ends, at = [], 0
    place = [-1] * len(flat)
    slot = []
    for rows in groups:
        for n, i in enumerate(rows):
            place[i] = at + n
        padded = -(-len(rows) // multiple) * multiple
        slot += rows + [-1] * (padded - len(rows))
        at += padded
        ends.append(at)
    if E == 1:  # one group is all rows there can be
        n = len(flat)
        ends = [(n + min(1, n) * (multiple - 1)) // multiple * multiple]
        slot += [-1] * (ends[0] - len(slot))
    return ends, [len(r) for r in groups], slot, np.array(place).reshape(np.asarray(experts).shape)
