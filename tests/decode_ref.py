"""Plain 64-bit (and integer) definitions of the decode-step operators, in numpy, for the tests."""
from __future__ import annotations

import numpy as np


def rotary(x, pos, freq, amplitude=1.0, interleaved=False, inverse=False):
    """x [n, heads, dh] float64 -> (rotated, |u| + |v| of every element's pair)."""
    x = np.asarray(x, dtype=np.float64)
    rd = 2 * len(freq)
    ang = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(freq)[None, None, :]
    turn = amplitude * np.exp(1j * (-ang if inverse else ang))
    iu = np.arange(0, rd, 2) if interleaved else np.arange(rd // 2)
    iv = iu + 1 if interleaved else iu + rd // 2
    z = (x[..., iu] + 1j * x[..., iv]) * turn
    y, size = x.copy(), np.zeros_like(x)
    y[..., iu], y[..., iv] = z.real, z.imag
    size[..., iu] = size[..., iv] = abs(amplitude) * (np.abs(x[..., iu]) + np.abs(x[..., iv]))
    return y, size


def decode(q, k_pool, v_pool, table, lens, window=0, scale=0.0):
    """(out, lse, sum p|v|, error bound of a score) of one new token per sequence, float64."""
    n, hq, dh = q.shape
    ps, hkv = k_pool.shape[1], k_pool.shape[2]
    g = hq // hkv
    sc = scale if scale > 0 else dh ** -0.5
    out, lse = np.zeros((n, hq, dh)), np.full((n, hq), -np.inf)
    mass, ds = np.zeros((n, hq, dh)), np.zeros((n, hq))
    for r in range(n):
        j = np.arange(max(0, lens[r] - window) if window else 0, lens[r])
        if not len(j):
            continue
        rows = (table[r, j // ps], j % ps)
        k, v = k_pool[rows].astype(np.float64), v_pool[rows].astype(np.float64)
        for h in range(hq):
            s = sc * (k[:, h // g] @ q[r, h])
            m = s.max()
            p = np.exp(s - m)
            out[r, h] = (p / p.sum()) @ v[:, h // g]
            mass[r, h] = (p / p.sum()) @ np.abs(v[:, h // g])
            lse[r, h] = m + np.log(p.sum())
            ds[r, h] = dh * 2.0 ** -23 * sc * (np.abs(k[:, h // g]) @ np.abs(q[r, h])).max()
    return out, lse, mass, ds


def beams(logits, scores, k, finished=None, eos=-1):
    """(scores, tokens, parents, finished) by sorting every candidate in 64 bits."""
    n, w, vocab = logits.shape
    out = (np.full((n, k), -np.inf), np.full((n, k), -1), np.full((n, k), -1), np.zeros((n, k), bool))
    for r in range(n):
        cand = []
        for b in range(w):
            if finished is not None and finished[r, b]:
                cand.append((-float(scores[r, b]), b, eos))
                continue
            x = logits[r, b].astype(np.float64)
            m = x.max()
            with np.errstate(all="ignore"):
                c = float(scores[r, b]) + ((x - m) - np.log(np.exp(x - m).sum()))  # m + log would lose it at 3e38
            c[np.isnan(c)] = -np.inf
            # the K best of a beam are enough; a stable sort keeps ties in token order
            for t in np.argsort(-c, kind="stable")[:k]:
                cand.append((-c[t], b, int(t)))
        cand = sorted(x for x in cand if x[0] < np.inf)[:k]
        for i, (c, b, t) in enumerate(cand):
            out[0][r, i], out[1][r, i], out[2][r, i] = -c, t, r * w + b
            out[3][r, i] = t == eos or (finished is not None and bool(finished[r, b]))
    return out


def fork(parent, lens, table, refs):
    lens, table, refs = np.array(lens), np.array(table), np.array(refs)
    par = [p if -1 <= p < len(parent) else i for i, p in enumerate(parent)]
    nt = np.array([table[p] if p >= 0 else np.full(table.shape[1], -1) for p in par], dtype=np.int32).reshape(table.shape)
    nl = np.array([lens[p] if p >= 0 else 0 for p in par], dtype=np.int32)
    for e in table[table >= 0]:
        refs[e] -= 1
    for e in nt[nt >= 0]:
        refs[e] += 1
    return nl, nt, refs


def reserve(starts, lens, table, refs, pools, page, n, advance):
    """One sequence after the other, by the definition. Returns lens, table, refs, pools, slots, positions, bad."""
    lens, table, refs = np.array(lens), np.array(table), np.array(refs)
    pools = [np.array(p) for p in pools]
    before = refs.copy()  # free and shared are as at the start
    slots, pos = np.full(n, -1, np.int32), np.zeros(n, np.int32)
    rows, width = table.shape
    if any(starts[r] < 0 or starts[r + 1] < starts[r] or starts[r + 1] > n for r in range(rows)):
        return lens, table, refs, pools, slots, pos, True
    free = [i for i in range(len(refs)) if before[i] == 0]
    taken, bad = 0, False
    for r in range(rows):
        count, L = int(starts[r + 1] - starts[r]), int(lens[r])
        if count == 0:
            continue
        if L < 0 or L + count > width * page:
            bad = True
            continue
        touched = range(L // page, -(-(L + count) // page))
        e = {p: int(table[r, p]) for p in touched}
        if any(x >= len(refs) or x < -1 or (x >= 0 and before[x] <= 0) or (x < 0 and p == L // page and L % page)
               for p, x in e.items()):
            bad = True
            continue
        need = [p for p in touched if e[p] < 0 or before[e[p]] > 1]
        if need and taken + len(need) > len(free):
            taken += len(need)
            bad = True
            continue
        for p in need:
            new = free[taken]
            taken += 1
            if e[p] >= 0:
                refs[e[p]] -= 1
                if p == L // page:
                    for x in pools:
                        x[new, :L % page] = x[e[p], :L % page]
            refs[new] = 1
            table[r, p] = new
        for i in range(count):
            p = L + i
            slots[starts[r] + i], pos[starts[r] + i] = table[r, p // page] * page + p % page, p
        if advance:
            lens[r] += count
    return lens, table, refs, pools, slots, pos, bad


def compact(table, refs, pools):
    table, refs = np.array(table), np.array(refs)
    pools = [np.array(p) for p in pools]
    used = int((refs > 0).sum())
    src = [i for i in range(used, len(refs)) if refs[i] > 0]
    dst = [i for i in range(used) if refs[i] == 0]
    to = dict(zip(src, dst))
    for a, b in to.items():
        for x in pools:
            x[b] = x[a]
        refs[b], refs[a] = refs[a], 0
    for i in np.ndindex(table.shape):
        table[i] = to.get(int(table[i]), table[i])
    return table, refs, pools, used
