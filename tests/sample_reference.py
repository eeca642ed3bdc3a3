"""Plain reference of drawing tokens and of judging drafts: one row at a time in 64 bits, written from the definitions in
include/dspark.h; CPU only."""
import math

import numpy as np


def distribution(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """p of one row's tokens, float64 [vocab]; zeros where the row has no token."""
    l = np.asarray(logits, dtype=np.float64)
    p = np.zeros(l.size)
    order = [v for v in np.lexsort((np.arange(l.size), -np.where(np.isnan(l), -np.inf, l))) if l[v] > -np.inf]
    if not order:
        return p
    top = l[order[0]]
    if not temperature > 0:
        p[order[0]] = 1.0
        return p
    order = np.array(order)
    if top == np.inf:
        order = order[l[order] == np.inf]
        w = np.ones(order.size)
    else:
        w = np.exp((l[order] - top) / temperature)
    if 0 < top_k < l.size:
        order, w = order[:top_k], w[:top_k]
    if top_p < 1:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1]))
        stay = before < top_p * w.sum()
        stay[0] = True
        order, w = order[stay], w[stay]
    if min_p > 0:
        order, w = order[w >= min(min_p, 1.0)], w[w >= min(min_p, 1.0)]
    p[order] = w
    return p / p.sum()


def pick(p, u):
    """The lowest token whose p, added up to it, exceeds u of the sum; -1 if nothing weighs anything."""
    upto = np.cumsum(p)
    if not upto[-1] > 0:
        return -1
    u = 0.0 if not u > 0 else u
    at = int(np.searchsorted(upto, u * upto[-1], side="right"))
    return at if at < p.size else int(np.nonzero(p)[0][-1])


def margin(p, u):
    """How far u is from where pick's answer changes."""
    upto = np.concatenate(([0.0], np.cumsum(p)))
    upto /= upto[-1]
    return float(np.abs(upto[1:-1] - u).min()) if p.size > 1 else math.inf


def verify(rows, drafts, uniforms, draft_probs=None, vocab=None):
    """One sequence: rows: p of each of its len(drafts) + 1 rows; uniforms [rows, 2].  Returns (ids, accepted)."""
    ids, taken = [], 0
    for i, p in enumerate(rows):
        if i < len(drafts):
            x = int(drafts[i])
            if 0 <= x < p.size:
                q = np.zeros(p.size) if draft_probs is None else draft_probs[i].astype(np.float64)
                if draft_probs is None:
                    q[x] = 1.0
                if float(uniforms[i][0]) * q[x] < p[x]:
                    ids.append(x)
                    taken += 1
                    continue
                rest = np.maximum(p - q, 0.0)
                p = rest if rest.sum() > 0 else p
        ids.append(pick(p, float(uniforms[i][1])))
        break
    return ids + [-1] * (len(rows) - len(ids)), taken
