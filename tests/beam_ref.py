"""Beam search's selection and reordering from their definitions, in 64 bits (numpy)."""
import numpy as np


def log_probs(x, allowed=None):
    """x [R, V] float64 -> log-softmax over the allowed tokens, -inf elsewhere."""
    x = np.array(x, np.float64)
    if allowed is not None:
        x[~allowed] = -np.inf
    out = np.full_like(x, -np.inf)
    for r in range(x.shape[0]):
        top = x[r].max(initial=-np.inf)
        if top > -np.inf:
            keep = x[r] > -np.inf
            out[r, keep] = (x[r, keep] - top) - np.log(np.exp(x[r, keep] - top).sum())
    return out


def candidate_scores(x, scores, allowed=None, ended=None, end_token=0):
    """[R, V] float64 scores of all continuations, -inf where there is none."""
    s = log_probs(x, allowed)
    for r in range(s.shape[0]):
        if ended is not None and ended[r]:
            s[r] = -np.inf
            s[r, end_token] = scores[r]
        elif scores[r] == -np.inf:
            s[r] = -np.inf
        else:
            s[r] = np.where(s[r] > -np.inf, np.float64(scores[r]) + s[r], -np.inf)
    return s


def select(s, cu, k):
    """The k best of each request's rows: (scores, rows, tokens)."""
    out = np.full((len(cu) - 1, k), -np.inf), np.full((len(cu) - 1, k), -1), np.full((len(cu) - 1, k), -1)
    for b in range(len(cu) - 1):
        rows = s[cu[b]:cu[b + 1]]
        r, t = np.nonzero(rows > -np.inf)
        v = rows[r, t]
        order = np.lexsort((t, r, -v))[:k]
        n = len(order)
        out[0][b, :n], out[1][b, :n], out[2][b, :n] = v[order], r[order] + cu[b], t[order]
    return out


def reorder(parents, table, lens, spare, bs):
    """(table, lens, slots, used, copies [(from, to, rows)])."""
    n, width = len(parents), table.shape[1]
    out, ln = np.full((n, width), -1, np.int32), np.zeros(n, np.int32)
    slots, used, copies, met = np.full(n, -1, np.int64), np.zeros(n, np.int32), [], set()
    for i, p in enumerate(parents):
        if p < 0:
            continue
        full, rest = divmod(int(lens[p]), bs)
        out[i, :full] = table[p, :full]
        if rest == 0 or p in met:
            out[i, full], used[i] = spare[i], 1
            if rest:
                copies.append((int(table[p, full]), int(spare[i]), rest))
        else:
            out[i, full] = table[p, full]
        met.add(p)
        ln[i] = lens[p] + 1
        slots[i] = int(out[i, full]) * bs + rest
    return out, ln, slots, used, copies
