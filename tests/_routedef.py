"""The selection by its definition, with sums of keys in exact arithmetic (no code of the package).  Logits finite or -inf,
biases finite or -inf."""
import math
from fractions import Fraction


def scores(l, score):
    """In 64 bits; 0 (unused) where the logit is -inf."""
    if score == "softmax":
        return [0.0 if x == -math.inf else x for x in l]
    if score == "sigmoid":
        return [1 / (1 + math.exp(-x)) if x >= 0 else math.exp(max(x, -745.0)) / (1 + math.exp(x)) for x in l]
    top = max(l)
    e = [math.exp(x - top) if x != -math.inf else 0.0 for x in l]
    total = math.fsum(e)
    return [x / total if total else 0.0 for x in e]


def select(l, k, score, bias=None, groups=1, top_groups=None, group_score="top2"):
    """The experts of one token: key = score + bias, -inf as a logit or a bias takes an expert out; a group is worth the sum
    of the two largest keys of the experts left in it (of the one, where there is one), or the largest."""
    E = len(l)
    b = [0.0] * E if bias is None else [float(x) for x in bias]
    live = [x != -math.inf and y != -math.inf for x, y in zip(l, b)]
    same = len(set(b)) == 1
    s = scores(l, score) if any(live) else [0.0] * E
    key = [Fraction(x) + Fraction(y) if n else None for x, y, n in zip(s, b, live)]
    # where all have the same bias, experts rank by their logits, which order as their scores do
    order = [Fraction(x) if n else None for x, n in zip(l, live)] if same else key
    left = [e for e in range(E) if live[e]]
    if groups > 1:
        n = E // groups
        worth = {}
        for g in range(groups):
            mine = [e for e in left if e // n == g]
            if not mine:
                continue
            if group_score == "max":
                worth[g] = max(order[e] for e in mine)
            else:
                best = sorted(mine, key=lambda e: order[e], reverse=True)[:2]
                worth[g] = sum(key[e] for e in best)
        stay = sorted(worth, key=lambda g: (-worth[g], g))[:top_groups]
        left = [e for e in left if e // n in stay]
    return sorted(left, key=lambda e: (-order[e], e))[:k]
