"""Float64 definitions of the operators that check drafted trees of several requests.

Plain numpy and Python on the host, one request, row or token at a time; nothing is
shared with the GPU path.
"""
from __future__ import annotations

import numpy as np


def ancestors(parents, n):
    """Rows that each of n rows attends to ([n][n] bool) and its depth; None for a row that hangs below no earlier one.
    parents None: a chain."""
    out = []
    for i in range(n):
        p = i - 1 if parents is None else int(parents[i])
        if i > 0 and (not 0 <= p < i or out[p] is None):
            out.append(None)
            continue
        see, depth = (np.zeros(n, bool), 0) if i == 0 else (out[p][0].copy(), out[p][1] + 1)
        see[i] = True
        out.append((see, depth))
    return out


def step_slots(held, fresh, owned, table, ring, state, page, rows, parents=None, base=0, words=0, limit=None, in_place=False):
    """A dict of the call's outputs. limit: rows that a request may bring."""
    n, width, pages = len(held), table.shape[1], len(ring)
    first, free = int(state[0]), int(state[1])
    o = {"new_table": np.array(table) if in_place else np.full_like(table, -1), "new_owned": np.zeros(n, int),
         "ctx_len": np.full(n, -1), "row_start": np.zeros(n + 1, int), "ring": np.array(ring),
         "seq": np.full(rows, -1), "positions": np.full(rows, -1), "slots": np.full(rows, -1),
         "mask": np.zeros((rows, 32 * words), bool)}
    at = asked = given = 0
    back = []
    for s in range(n):
        mine = max(0, int(fresh[s])) if held[s] >= 0 else 0
        lo, at = at, at + mine
        o["row_start"][s + 1] = min(at, rows)
        if held[s] < 0:
            back += [int(e) for e in table[s, : owned[s]]]
            continue
        o["new_table"][s, : owned[s]] = table[s, : owned[s]]
        o["new_owned"][s] = owned[s]
        need = -(-(int(held[s]) + mine) // page)
        if need > width or at > rows or (limit is not None and mine > limit):
            continue
        lack = max(0, need - int(owned[s]))
        asked += lack
        if lack and asked > free:
            continue
        got = [int(ring[(first + given + j) % pages]) for j in range(lack)]
        o["new_table"][s, owned[s]: owned[s] + lack] = got
        o["new_owned"][s] += lack
        given += lack
        o["ctx_len"][s] = held[s]
        rel = ancestors(None if parents is None else parents[lo:at], mine) if words or parents is not None else None
        for i in range(mine):
            if rel is not None and rel[i] is None:
                continue
            t = int(held[s]) + i
            o["seq"][lo + i] = s
            o["positions"][lo + i] = base + int(held[s]) + (i if rel is None else rel[i][1])
            o["slots"][lo + i] = int(o["new_table"][s, t // page]) * page + t % page
            if words:
                o["mask"][lo + i, :mine] = rel[i][0]
    for k, e in enumerate(back[: pages - free]):
        o["ring"][(first + free + k) % pages] = e
    o["new_free_state"] = np.array([(first + given) % pages if pages else 0, free - given + min(len(back), pages - free)])
    return o


def adjust(x, text, prompt, drafted, rep, freq, pres, biases, allowed):
    """One row of logits. text, drafted: its tokens, one behind the other, the first `prompt` of them all the prompt; biases:
    pairs (token, value), the last of a token counts; allowed: bool [vocab] or None. Also the greedy token, or -1."""
    x = np.array(x, dtype=np.float64)
    v = len(x)
    whole = [int(t) for t in list(text) + list(drafted)]
    said = [t for t in whole[prompt:] if 0 <= t < v]
    for t in {t for t in whole if 0 <= t < v}:
        x[t] = x[t] / rep if x[t] > 0 else x[t] * rep
        n = said.count(t)
        if n:
            x[t] = x[t] - freq * n - pres
    for t, b in {int(t): b for t, b in biases}.items():
        if 0 <= t < v:
            x[t] += b
    if allowed is not None:
        x[~allowed] = -np.inf
    y = np.where(np.isnan(x), -np.inf, x)
    return x, int(np.argmax(y)) if np.max(y) > -np.inf else -1


def accept(parents, draft, after, most):
    """The accepted rows of one request's tree (parents None: a chain)."""
    n, path = len(draft), [0]
    while len(path) < most:
        r = path[-1]
        child = [c for c in range(r + 1, n) if after[r] >= 0 and draft[c] == after[r]
                 and (c - 1 if parents is None else parents[c]) == r]
        if not child:
            break
        path.append(child[0])
    return path


def attend(q, k, v, seen, scale):
    """q [rows, group, d] over k, v [n, d], row i over the keys seen[i]: (outputs, log-sums, sum of p |v|)."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    out, lse, size = np.zeros_like(q), np.full(q.shape[:2], -np.inf), np.zeros_like(q)
    for i in range(q.shape[0]):
        kk, vv = k[seen[i]], v[seen[i]]
        if not len(kk):
            continue
        s = q[i] @ kk.T * scale
        m = np.max(s, axis=1, keepdims=True)
        p = np.exp(s - m)
        z = np.sum(p, axis=1, keepdims=True)
        out[i], lse[i], size[i] = p @ vv / z, (m + np.log(z))[:, 0], p @ np.abs(vv) / z
    return out, lse, size
