"""Plain 64-bit references of the paged-cache operators (numpy, one row at a time)."""
from __future__ import annotations

import numpy as np


def tree_masks(offsets, parents, lens, words):
    t = len(parents)
    mask = np.zeros((t, words), np.uint64)
    pos = np.zeros(t, np.int32)
    for b in range(len(offsets) - 1):
        for i in range(offsets[b + 1] - offsets[b]):
            row, j, depth = offsets[b] + i, int(i), 0
            while j >= 0:
                mask[row, j // 64] |= np.uint64(1 << (j % 64))
                j = int(parents[offsets[b] + j])
                depth += j >= 0
            pos[row] = (0 if lens is None else lens[b]) + depth
    return mask, pos


def attention(q, k_new, v_new, k, v, offsets, lens, table, mask, pos, window, scale):
    """q [T, hq, d], k_new/v_new [T, hk, d], k/v [blocks, hk, bs, d] in float64; returns out, lse and, for the
    error bounds, sum_j p_j |v_j| and max_j scale * sum_d |q_d k_jd|."""
    T, hq, d = q.shape
    offsets, lens = [int(x) for x in offsets], [int(x) for x in lens]
    hk, bs = k.shape[1], k.shape[2]
    out, lse = np.zeros((T, hq, d)), np.full((T, hq), -np.inf)
    mass, dot = np.zeros((T, hq, d)), np.zeros((T, hq))
    for b in range(len(lens)):
        t0, t1, ln = offsets[b], offsets[b + 1], lens[b]
        at = np.arange(ln)
        blk = table[b][at // bs] if ln else np.zeros(0, int)
        pk, pv = k[blk, :, at % bs], v[blk, :, at % bs]
        dpos = np.array([min(max(pos[t], ln), ln + t1 - t0 - 1) if pos is not None else ln + t - t0
                         for t in range(t0, t1)])
        for t in range(t0, t1):
            p = dpos[t - t0]
            see = np.ones(ln, bool) if not window else p - at < window
            dr = [j for j in range(t0, t1)
                  if (int(mask[t, (j - t0) // 64]) >> ((j - t0) % 64) & 1 if mask is not None else j <= t)
                  and (not window or p - dpos[j - t0] < window)]
            for h in range(hq):
                g = h // (hq // hk)
                kk = np.concatenate([pk[see, g], k_new[dr, g]])
                vv = np.concatenate([pv[see, g], v_new[dr, g]])
                if not len(kk):
                    continue
                s = scale * (kk @ q[t, h])
                m = s.max()
                e = np.exp(s - m)
                lse[t, h] = m + np.log(e.sum())
                w = e / e.sum()
                out[t, h] = w @ vv
                mass[t, h] = w @ np.abs(vv)
                dot[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, mass, dot


def plan(bs, max_blocks, n_slots, lens, new, owned, table, ring, state):
    """The block plan request by request; returns every output (table and ring as copies)."""
    table, ring = table.copy(), ring.copy()
    size = len(ring)
    head, count = int(state[0]), int(state[1])
    lens_out, owned_out = lens.copy(), owned.copy()
    offsets, slots = [0], np.full(n_slots, -1, np.int32)
    asked = taken = pushed = 0
    for b in range(len(lens)):
        t0 = offsets[-1]
        add = max(int(new[b]), 0)
        offsets.append(t0 + add)
        if new[b] < 0:
            for j in range(owned[b]):
                if pushed + j < size - count:
                    ring[(head + count + pushed + j) % size] = table[b, j]
            pushed += int(owned[b])
            lens_out[b] = owned_out[b] = 0
            continue
        after = -(-(int(lens[b]) + add) // bs)
        if after > max_blocks or t0 + add > n_slots:
            continue
        need = max(after - int(owned[b]), 0)
        first, asked = asked, asked + need
        if need and asked > count:
            continue
        for j in range(need):
            table[b, owned[b] + j] = ring[(head + first + j) % size]
        taken = max(taken, asked if need else 0)
        lens_out[b] += add
        owned_out[b] += need
        for i in range(add):
            p = int(lens[b]) + i
            slots[t0 + i] = table[b, p // bs] * bs + p % bs
    return dict(block_table=table, ring=ring, lens=lens_out, owned=owned_out, slots=slots,
                offsets=np.array(offsets, np.int32),
                state=np.array([(head + taken) % size, count - taken + min(pushed, size - count)], np.int32))
