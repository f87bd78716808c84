"""Plain implementations, in 64 bits or whole numbers, of sampling, rotary
positions and the cache's forks and moves, for their tests.  They loop over rows,
requests and blocks as the definitions in include/specdec_step.h read, and share no
code with the CUDA path."""
import math

import numpy as np


def sample_row(row, T=1.0, k=0, p=1.0, m=0.0, u=None):
    """One row of floats: the ids kept (a set) and the token (-1: none)."""
    row = np.array(row, dtype=np.float64) + 0.0
    row[np.isnan(row)] = -math.inf
    if (row == math.inf).any():  # the others are nothing beside it
        row = np.where(row == math.inf, 0.0, -math.inf)
    V = row.size
    order = np.lexsort((np.arange(V), -row))
    order = order[row[order] > -math.inf]
    if order.size == 0:
        return set(), -1
    T, p, m = float(np.float32(T)), float(np.float32(p)), float(np.float32(m))
    if not float(np.float32(1e-6)) <= T <= float(np.float32(3e38)):
        return {int(order[0])}, int(order[0])
    top = row[order[0]]
    w = np.exp((row[order].astype(np.longdouble) - top) / np.longdouble(T))
    n = order.size
    if 0 < k < V:
        n = min(n, k)
    total = w[:n].sum()
    if not p >= 0:
        p = 1.0
    if p < 1.0:
        before = np.concatenate([[0.0], np.cumsum(w[:n])[:-1]])
        n = max(1, int((before < p * total).sum()))
    m = 0.0 if not m >= 0 else min(m, 1.0)
    n = min(n, int((w >= m).sum())) if m > 0 else n
    kept = {int(i) for i in order[:n]}
    if u is None:
        return kept, None
    u = float(np.float32(u))
    u = 1.0 - 2.0 ** -24 if u >= 1 else (u if u >= 0 else 0.0)
    run = np.cumsum(w[:n])
    return kept, int(order[int((run > u * run[-1]).argmax())])


def rotate(x, positions, freq, pairs_layout, factor, before):
    """x [T, H, D] in float64 turned; rows of negative positions as in `before`."""
    x = np.array(x, dtype=np.float64)
    out = np.array(before, dtype=np.float64)
    half = len(freq)
    for t, p in enumerate(positions):
        if p < 0:
            continue
        out[t] = x[t]
        for i, f in enumerate(freq):
            a, b = (2 * i, 2 * i + 1) if pairs_layout else (i, i + half)
            angle = float(p) * f
            c, s = factor * math.cos(angle), factor * math.sin(angle)
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
    return out


def fork(table, kv_len, accepted, held, parent, keep, shares, ring, state, bs):
    """As kv_fork; `bad`: whether it sets the error bit."""
    P, W = table.shape
    B, N = len(parent), len(ring)
    ring, bad = ring.copy(), False
    head, free = int(state[0]), int(state[1])
    if not (0 <= head < N and 0 <= free <= N):
        bad, head, free = True, head if 0 <= head < N else 0, max(0, min(free, N))
    held = [int(h) for h in held]
    bad |= any(h < 0 or h > W for h in held)
    held = [max(0, min(h, W)) for h in held]
    holders = {x: int(shares[x]) + 1 for x in range(N)}
    named = set()
    for p in range(P):
        for x in table[p, :held[p]]:
            if 0 <= x < N:
                holders[int(x)] -= 1
                named.add(int(x))
            else:
                bad = True
    rows, tokens = [], []
    for b in range(B):
        p = int(parent[b])
        if p < -1 or p >= P:
            bad, p = True, -1
        if p < 0:
            rows.append([])
            tokens.append(0)
            continue
        n = int(kv_len[p]) + (max(int(accepted[p]), -1) + 1 if accepted is not None else 0)
        if n < 0 or n > held[p] * bs:
            bad, n = True, max(0, min(n, held[p] * bs))
        if keep is not None:
            n = max(0, min(n, int(keep[b])))
        rows.append([int(x) for x in table[p, :(n + bs - 1) // bs]])
        tokens.append(n)
        for x in rows[b]:
            if 0 <= x < N:
                holders[x] += 1
            else:
                bad = True
    back = sorted(x for x in named if holders[x] <= 0)
    copies, asked = [], 0
    for b in range(B):
        if tokens[b] % bs == 0:
            continue
        x = rows[b][-1]
        if not 0 <= x < N or holders[x] <= 1:
            continue
        holders[x] -= 1
        asked += 1
        if asked > free:
            bad = True
            rows[b].pop()
            tokens[b] = tokens[b] // bs * bs
            continue
        fresh = int(ring[(head + len(copies)) % N])
        bad |= not 0 <= fresh < N
        copies.append((x, fresh))
        rows[b][-1] = fresh
    for i, x in enumerate(back):
        ring[(head + free + i) % N] = x
    out = np.full((B, W), -1, dtype=np.int64)
    for b in range(B):
        out[b, :len(rows[b])] = rows[b]
    new_shares = np.array([max(0, holders[x] - 1) if x in named else int(shares[x]) for x in range(N)])
    return dict(block_table=out, kv_len=np.array(tokens), held=np.array([len(r) for r in rows]), shares=new_shares, ring=ring,
                ring_state=np.array([(head + len(copies)) % N, min(N, free - len(copies) + len(back))]), copies=copies, bad=bad)


def compact(table, held, shares, ring, state):
    """As kv_compact."""
    B, W = table.shape
    N, bad = len(ring), False
    head, free = int(state[0]), int(state[1])
    if not (0 <= head < N and 0 <= free <= N):
        bad, head, free = True, head if 0 <= head < N else 0, max(0, min(free, N))
    listed = [int(ring[(head + i) % N]) for i in range(free)]
    bad |= any(x < 0 or x >= N for x in listed)
    empty = {x for x in listed if 0 <= x < N}
    n = N - len(empty)
    moves = list(zip((x for x in range(n, N) if x not in empty), sorted(x for x in empty if x < n)))
    name = {x: x for x in range(N) if x not in empty}
    name.update(moves)
    out = np.full((B, W), -1, dtype=np.int64)
    for b in range(B):
        h = int(held[b])
        if h < 0 or h > W:
            bad, h = True, max(0, min(h, W))
        for j in range(h):
            out[b, j] = name.get(int(table[b, j]), -1)
            bad |= out[b, j] < 0
    new_shares = np.zeros(N, dtype=np.int64)
    for x, y in name.items():
        new_shares[y] = shares[x]
    return dict(block_table=out, shares=new_shares, free=list(range(n, N)), renamed=np.array([name.get(x, -1) for x in range(N)]),
                copies=moves, bad=bad)
