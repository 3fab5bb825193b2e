"""Plain fp64 restatement of the paged-cache operators (numpy, on the host).

Test infrastructure only.  The cache is a pool of pages [n_pages, Hkv, page, d]
(fp64 arrays holding exactly the stored values), a page table [B, max_pages],
and the statistics weight and token_pos [B, Hkv, T_cap].  Every function loops
over sequences and heads and goes by the definition; an entry of the page table
outside the pool is a page that holds nothing.
"""

import numpy as np

from .fasa_oracle import apply_rope_q


def _rows(table, n_pages, page, slots):
    """(page index, row in the page) of each slot; page index -1 outside the pool."""
    pg = table[slots // page]
    pg = np.where((pg >= 0) & (pg < n_pages), pg, -1)
    return pg, slots % page


def rotate(x, pos, theta):
    """x [H, d] turned by the position pos (interleaved pairs)."""
    return apply_rope_q(np.asarray(x, dtype=np.float64)[None], np.array([pos]), theta)[0]


def paged_append(k_new, v_new, cu_new, pos, table, lens, kp, vp, weight, token_pos, theta):
    """In place; keys are left unrounded.  Tokens without a slot or a page are left out."""
    n_pages, _, page, _ = kp.shape
    cap = table.shape[1] * page
    for b in range(table.shape[0]):
        for j, x in enumerate(range(cu_new[b], cu_new[b + 1])):
            t = lens[b] + j
            if lens[b] < 0 or t >= cap:
                continue
            pg, r = _rows(table[b], n_pages, page, np.array([t]))
            if pg[0] < 0:
                continue
            m = int(pos[b]) + j
            kp[pg[0], :, r[0]] = rotate(k_new[x], m, theta)
            vp[pg[0], :, r[0]] = v_new[x]
            if weight is not None:
                weight[b, :, t] = 0.0
            if token_pos is not None:
                token_pos[b, :, t] = m


def paged_attention(q, pos, kp, vp, table, lens, theta):
    """out [B, Hq, d], the weights each slot receives [B, Hkv, T_cap], the
    logits' scale A [B, Hq, T_cap] = sum |q| |k| / sqrt(d) (for error bounds)
    and sum_t p |V| [B, Hq, d]."""
    n_pages, Hkv, page, d = kp.shape
    B, Hq, _ = q.shape
    G, cap = Hq // Hkv, table.shape[1] * page
    out, received = np.zeros((B, Hq, d)), np.zeros((B, Hkv, cap))
    scale, p_abs_v = np.zeros((B, Hq, cap)), np.zeros((B, Hq, d))
    for b in range(B):
        slots = np.arange(min(max(int(lens[b]), 0), cap))
        pg, r = _rows(table[b], n_pages, page, slots)
        slots, r, pg = slots[pg >= 0], r[pg >= 0], pg[pg >= 0]
        if slots.size == 0:
            continue
        qr = rotate(q[b], pos[b], theta)
        for h in range(Hkv):
            K, V = kp[pg, h, r], vp[pg, h, r]
            for g in range(h * G, (h + 1) * G):
                z = K @ qr[g] / np.sqrt(d)
                w = np.exp(z - z.max())
                w /= w.sum()
                out[b, g] = w @ V
                received[b, h, slots] += w
                scale[b, g, slots] = np.abs(K) @ np.abs(qr[g]) / np.sqrt(d)
                p_abs_v[b, g] = w @ np.abs(V)
    return out, received, scale, p_abs_v


def evict_choice(weight, token_pos, pos, keep, sinks, recent):
    """Slots of one (sequence, head) that stay, ascending: held ones first,
    then the heaviest; equal ones by slot; NaN last."""
    n = len(weight)
    held = (token_pos < sinks) | (token_pos.astype(np.int64) > int(pos) - recent)
    nan = np.isnan(weight)
    rank = [(0, 0.0, t) if held[t] else (2, 0.0, t) if nan[t] else (1, -float(weight[t]), t) for t in range(n)]
    order = [t for _, _, t in sorted(rank)]
    return np.array(sorted(order[:keep]), dtype=np.int64)


def paged_evict(weight, token_pos, pos, table, lens, keep, sinks, recent, kp, vp, weight_out, token_pos_out):
    """In place for kp, vp and the outputs (which may be the inputs); returns new_lens."""
    n_pages, Hkv, page, _ = kp.shape
    B, cap = table.shape[0], table.shape[1] * page
    new = np.zeros(B, dtype=np.int32)
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        new[b] = min(n, keep)
        for h in range(Hkv):
            w, tp = weight[b, h, :n].copy(), token_pos[b, h, :n].copy()
            if n > keep:
                stay = evict_choice(w, tp, pos[b], keep, sinks, recent)
                dst = np.setdiff1d(np.arange(keep), stay)
                src = stay[stay >= keep]
                pd, rd = _rows(table[b], n_pages, page, dst)
                ps, rs = _rows(table[b], n_pages, page, src)
                ok = (pd >= 0) & (ps >= 0)
                k_rows, v_rows = kp[ps[ok], h, rs[ok]].copy(), vp[ps[ok], h, rs[ok]].copy()
                kp[pd[ok], h, rd[ok]], vp[pd[ok], h, rd[ok]] = k_rows, v_rows
                w[dst], tp[dst] = w[src], tp[src]
            weight_out[b, h, :new[b]], token_pos_out[b, h, :new[b]] = w[:new[b]], tp[:new[b]]
    return new
