"""Plain fp64 restatement of a step of new tokens over the paged cache (numpy, on
the host): pages assigned, queries and keys turned and stored, attention of
chunks.

Test infrastructure only; every function loops over sequences, tokens and heads
and goes by the definition.  Arrays are laid out as in paged_oracle.
"""

import math

import numpy as np

from .paged_oracle import _rows


def assign(have, want, pos, table, free, count, max_tokens, page):
    """table and free (numpy) change in place.  Returns lens, cu_new, token_map, count."""
    B, max_pages = table.shape
    cap, n_pages = max_pages * page, len(free)
    have = [min(max(int(x), 0), cap) for x in have]
    want = [min(max(int(x), 0), cap) for x in want]
    stack = [int(x) for x in free[:min(max(int(count), 0), n_pages)]]
    for b in range(B):
        for e in range(-(-want[b] // page), -(-have[b] // page)):
            if len(stack) < n_pages:
                stack.append(int(table[b, e]))
    free[:len(stack)] = stack  # what came back stays written, though it may be taken again
    lens, cu, rows, served = [], [0], [], True
    for b in range(B):
        h, w = have[b], want[b]
        need = -(-w // page) - -(-h // page)
        if w > h:
            served = served and need <= len(stack) and len(rows) + w - h <= max_tokens
            if not served:
                w = h
            else:
                for e in range(-(-h // page), -(-w // page)):
                    table[b, e] = stack.pop()
                rows += [(b, t, int(table[b, t // page]), (h if pos is None else int(pos[b])) + t - h)
                         for t in range(h, w)]
        lens.append(w)
        cu.append(len(rows))
    rows += [(-1,) * 4] * (max_tokens - len(rows))
    return lens, cu, rows, len(stack)


def frequencies(rope):
    """Angle per position of every pair, by the layouts' common definition."""
    r = rope.rotary_dim
    t = [rope.rope_theta ** (-2.0 * i / r) for i in range(r // 2)]
    if rope.scaling == 0:
        return np.array(t)
    if rope.scaling == 1:
        return np.array(t) / rope.factor
    if rope.scaling == 2:
        out = []
        for x in t:
            turns = rope.original * x / (2 * math.pi)
            if turns >= rope.high:
                out.append(x)
            elif turns <= rope.low:
                out.append(x / rope.factor)
            else:
                s = (turns - rope.low) / (rope.high - rope.low)
                out.append((1 - s) * x / rope.factor + s * x)
        return np.array(out)
    index = [r * math.log(rope.original / (x * 2 * math.pi)) / (2 * math.log(rope.rope_theta))
             for x in (rope.high, rope.low)]
    i0, i1 = max(math.floor(index[0]), 0), min(math.ceil(index[1]), r - 1)
    if i0 >= i1:
        i1 = i0 + 0.001
    s = np.clip((np.arange(r // 2) - i0) / (i1 - i0), 0.0, 1.0)
    return np.array(t) * (1 - s) + np.array(t) / rope.factor * s


def turn(x, m, rope):
    """x [H, d] at position m."""
    r = rope.rotary_dim
    a = m * frequencies(rope)
    c, s = np.cos(a) * rope.magnitude, np.sin(a) * rope.magnitude
    i = np.arange(r // 2) if rope.layout == 1 else 2 * np.arange(r // 2)
    j = i + r // 2 if rope.layout == 1 else i + 1
    y = np.array(x, dtype=np.float64)
    y[:, i], y[:, j] = x[:, i] * c - x[:, j] * s, x[:, i] * s + x[:, j] * c
    return y


def rope_append(q, k, v, token_map, q_out, kp, vp, weight, token_pos, rope):
    """In place for q_out (or None), kp, vp (or None) and the statistics (or None)."""
    for x, (b, t, page, m) in enumerate(token_map):
        if b < 0:
            continue
        if q is not None:
            q_out[x] = turn(q[x], m, rope)
        if k is not None:
            kp[page, :, t % kp.shape[2]] = turn(k[x], m, rope)
            vp[page, :, t % kp.shape[2]] = v[x]
            if weight is not None:
                weight[b, :, t] = 0.0
            if token_pos is not None:
                token_pos[b, :, t] = m


def chunk_attention(q, cu, kp, vp, table, lens):
    """q [n_tokens, Hq, d] turned.  Returns out (zeros in rows of no sequence), the
    weights that each slot receives [B, Hkv, T_cap], the logits' scale A [n_tokens, Hq] =
    max sum |q| |k| / sqrt(d) and sum p |V| [n_tokens, Hq, d] (for error bounds)."""
    n_pages, Hkv, page, d = kp.shape
    B, cap = table.shape[0], table.shape[1] * page
    Hq = q.shape[1]
    G = Hq // Hkv
    out, received = np.zeros(q.shape), np.zeros((B, Hkv, cap))
    scale, p_abs_v = np.zeros(q.shape[:2]), np.zeros(q.shape)
    for b in range(B):
        n, length = cu[b + 1] - cu[b], min(max(int(lens[b]), 0), cap)
        if n <= 0:
            continue
        slots = np.arange(length)
        pg, r = _rows(table[b], n_pages, page, slots)
        slots, r, pg = slots[pg >= 0], r[pg >= 0], pg[pg >= 0]
        for h in range(Hkv):
            K, V = kp[pg, h, r], vp[pg, h, r]
            for j in range(n):
                see = int(np.searchsorted(slots, length - n + j, side="right"))
                if see == 0:
                    continue
                x, heads = cu[b] + j, slice(h * G, (h + 1) * G)
                z = q[x, heads] @ K[:see].T / np.sqrt(d)
                w = np.exp(z - z.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                out[x, heads] = w @ V[:see]
                received[b, h, slots[:see]] += w.sum(axis=0)
                scale[x, heads] = (np.abs(q[x, heads]) @ np.abs(K[:see]).T).max(axis=1) / np.sqrt(d)
                p_abs_v[x, heads] = w @ np.abs(V[:see])
    return out, received, scale, p_abs_v
