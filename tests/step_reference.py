"""Plain implementations, in 64 bits or whole numbers, of the operators around
the verify step, for their tests.  They loop over requests, rows and tokens as
the definitions in include/specdec_step.h read, and share no code with the
CUDA path."""
import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_values():
    """The 256 values of the 8-bit type (sign, 4 exponent bits, 3 mantissa bits, no infinities)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return out


VALUES = e4m3_values()


def to_e4m3(x):
    """Codes of the nearest values, ties to the even code, saturating; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    grid = VALUES[:127]  # 0 .. 448
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf)), E4M3_MAX)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = grid[hi] - a, a - grid[lo]
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def pow2_scale(amax):
    if not amax > 0:
        return 0.0
    s = 2.0 ** (math.ceil(math.log2(amax / E4M3_MAX)) - 1)
    while amax > E4M3_MAX * s:
        s *= 2
    return max(s, 2.0 ** -126)


def append(x, slots, cache, scale):
    """One of keys and values: codes `cache` [N, H, bs, D] and `scale` [N, H] after the call."""
    cache, scale = cache.copy(), scale.astype(np.float64).copy()
    N, H, bs, D = cache.shape
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if s < 0 or s >= N * bs:
            t += 1
            continue
        block, off = divmod(s, bs)
        n = 1
        while t + n < len(slots) and off + n < bs and slots[t + n] == s + n:
            n += 1
        for h in range(H):
            new = x[t:t + n, h].astype(np.float64)
            fin = np.abs(new[np.isfinite(new)])
            now = pow2_scale(fin.max() if fin.size else 0.0)
            if off:
                old = scale[block, h]
                now = max(now, old)
                if now > old:
                    cache[block, h, :off] = to_e4m3(VALUES[cache[block, h, :off]] * old / now)
            scale[block, h] = now
            cache[block, h, off:off + n] = to_e4m3(new / now) if now else to_e4m3(new * 0.0)
        t += n
    return cache, scale


def block_step(table, kv_len, held, new, ring, state, bs, capacity, accepted=None):
    """Returns a dict of what kv_block_step leaves, as lists and arrays, and its error bit."""
    table, ring = table.copy(), ring.copy()
    B, width = table.shape
    N = len(ring)
    head, count = int(state[0]), int(state[1])
    bad = False
    if not 0 <= head < N:
        bad, head = True, 0
    if not 0 <= count <= N:
        bad, count = True, min(max(count, 0), N)
    asked = took = gave = tokens = 0
    kv_out, held_out, cu, cub, slots, pos = [], [], [0], [0], [], []
    back = []
    for b in range(B):
        h = int(held[b])
        if not 0 <= h <= width:
            bad, h = True, min(max(h, 0), width)
        w = max(int(new[b]), 0)
        kept = 0
        if new[b] >= 0:
            kept = int(kv_len[b]) + (max(int(accepted[b]), -1) + 1 if accepted is not None else 0)
            if not 0 <= kept <= h * bs:
                bad, kept = True, min(max(kept, 0), h * bs)
        need = -(-(kept + w) // bs)
        fits = need <= width
        grow = max(need - h, 0) if fits else 0
        asked += grow
        ok = fits and (grow == 0 or asked <= count)
        if not ok:
            bad, grow, give, w = True, 0, 0, 0
        else:
            give = max(h - need, 0)
        for i in range(give):
            back.append(int(table[b, h - give + i]))
        for i in range(grow):
            table[b, h + i] = ring[(head + took + i) % N]
        took += grow
        gave += give
        for i in range(w):
            p = kept + i
            if tokens < capacity:
                slots.append(int(table[b, p // bs]) * bs + p % bs)
                pos.append(p)
            else:
                bad = True
            tokens += 1
        kv_out.append(kept)
        held_out.append(h + grow - give)
        cu.append(min(tokens, capacity))
        cub.append(took)
    for i, blk in enumerate(back):
        ring[(head + count + i) % N] = blk
    slots += [-1] * (capacity - len(slots))
    pos += [-1] * (capacity - len(pos))
    return dict(table=table, ring=ring, kv_len=kv_out, held=held_out, ring_state=[(head + took) % N, min(N, count - took + gave)],
                cu_tokens=cu, cu_blocks=cub, slot_map=slots, positions=pos, bad=bad)


def attention(q, cu, kv_len, table, k_cache, v_cache, k_scale, v_scale, scale):
    """Returns (out, sum of p |v|, largest sum of |q k| scale of a row) [T, Hq, D] / [T, Hq]; rows of no request are NaN."""
    T, Hq, D = q.shape
    N, H, bs, _ = k_cache.shape
    out = np.full((T, Hq, D), np.nan)
    mag = np.zeros((T, Hq, D))
    big = np.zeros((T, Hq))
    for b in range(len(kv_len)):
        lo, hi = max(0, int(cu[b])), min(T, int(cu[b + 1]))
        if hi <= lo:
            continue
        L = min(int(kv_len[b]) + hi - lo, table.shape[1] * bs)
        ids = table[b, :-(-L // bs)] if L > 0 else table[b, :0]
        there = (ids >= 0) & (ids < N)
        at = np.where(there, ids, 0)
        live = there[:, None, None, None]
        k = np.where(live, VALUES[k_cache[at]] * k_scale[at][:, :, None, None].astype(np.float64), 0.0)
        v = np.where(live, VALUES[v_cache[at]] * v_scale[at][:, :, None, None].astype(np.float64), 0.0)
        k = k.transpose(1, 0, 2, 3).reshape(H, -1, D)
        v = v.transpose(1, 0, 2, 3).reshape(H, -1, D)
        for i in range(hi - lo):
            n = min(int(kv_len[b]) + i + 1, L)
            for hq in range(Hq):
                h = hq // (Hq // H)
                if n <= 0:
                    out[lo + i, hq] = 0.0
                    continue
                prod = k[h, :n] * q[lo + i, hq].astype(np.float64)
                s = prod.sum(1) * scale
                big[lo + i, hq] = np.abs(prod).sum(1).max() * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[lo + i, hq] = w @ v[h, :n]
                mag[lo + i, hq] = w @ np.abs(v[h, :n])
    return out, mag, big


def process_logits(x, history=None, prompt_len=None, history_len=None, draft_tokens=None, draft_len=None, repetition=None,
                   presence=None, frequency=None, bias_offsets=None, bias_ids=None, bias_values=None, mask=None, mask_rows=None):
    """Returns (out, sum of the magnitudes that met in each value); rows past a request's drafts keep x."""
    x = x.astype(np.float64)
    out, mag = x.copy(), np.abs(x)
    B, rows, V = x.shape
    for b in range(B):
        n = rows - 1 if draft_len is None else int(draft_len[b])
        rep = 1.0 if repetition is None else float(repetition[b])
        pres = 0.0 if presence is None else float(presence[b])
        freq = 0.0 if frequency is None else float(frequency[b])
        S = 0 if history is None else int(history_len[b])
        P = 0 if history is None else int(prompt_len[b])
        prompt = {int(v) for v in (history[b, :P] if P else [])}
        made = [int(v) for v in (history[b, P:S] if S > P else [])]
        bias = {}
        if bias_offsets is not None:
            for i in range(int(bias_offsets[b]), int(bias_offsets[b + 1])):
                bias[int(bias_ids[i])] = bias.get(int(bias_ids[i]), 0.0) + float(bias_values[i])
        for j in range(n + 1):
            tokens = made + [int(v) for v in (draft_tokens[b, :j] if j else [])]
            count = np.zeros(V)
            for v in tokens:
                if 0 <= v < V:
                    count[v] += 1
            seen = count > 0
            for v in prompt:
                if 0 <= v < V:
                    seen[v] = True
            y = x[b, j]
            y = np.where(seen, np.where(y > 0, y / rep, y * rep), y)
            m = np.abs(y) + abs(freq) * count + abs(pres) * (count > 0)
            y = y - freq * count - pres * (count > 0)
            for v, a in bias.items():
                if 0 <= v < V:
                    y[v] += a
                    m[v] += abs(a)
            if mask is not None and 0 <= mask_rows[b, j] < mask.shape[0]:
                words = mask[mask_rows[b, j]].astype(np.int64) & 0xFFFFFFFF
                allow = (words[np.arange(V) // 32] >> (np.arange(V) % 32)) & 1
                y = np.where(allow == 1, y, -np.inf)
            out[b, j], mag[b, j] = y, m
    return out, mag
