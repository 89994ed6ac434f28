"""Plain 64-bit implementations of the decode-side operators, on the CPU, for
the tests: loops over sequences, heads and entries, no shared code with the
library."""
from __future__ import annotations

import math

import numpy as np
import torch


def slot_place(table, page_size, b, slot):
    return int(table[b, slot // page_size]), slot % page_size


def gather(pool, table, page_size, b, h, n):
    """Rows 0..n-1 of sequence b, head h: float64 [n][dim]."""
    rows = [pool[pg, h, off].double() for pg, off in (slot_place(table, page_size, b, s) for s in range(n))]
    return torch.stack(rows) if rows else torch.zeros((0, pool.shape[3]), dtype=torch.float64)


def rope(x, pos, inv, magnitude, rot, interleaved):
    """x [rows][heads][dim] -> rotated float64."""
    x = x.double().clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ang = torch.tensor([math.fmod(float(p) * inv[i], 2 * math.pi) for p in pos.tolist()], dtype=torch.float64)
        c, s = (torch.cos(ang) * magnitude)[:, None], (torch.sin(ang) * magnitude)[:, None]
        u, v = x[:, :, a].clone(), x[:, :, b].clone()
        x[:, :, a], x[:, :, b] = u * c - v * s, u * s + v * c
    return x


def attention(q, kpool, vpool, table, lens, new, page_size, scale):
    """(out [seqs*n][q_heads][dim], weights {(b, h): [len]}, largest scale*sum|q||k|)."""
    B, H, D = len(lens), kpool.shape[1], kpool.shape[3]
    n = q.shape[0] // B
    G = q.shape[1] // H
    out = torch.zeros(q.shape, dtype=torch.float64)
    weights, reach = {}, 0.0
    for b in range(B):
        for h in range(H):
            k, v = gather(kpool, table, page_size, b, h, lens[b]), gather(vpool, table, page_size, b, h, lens[b])
            w = torch.zeros(lens[b], dtype=torch.float64)
            for t in range(new[b]):
                m = lens[b] - new[b] + t + 1
                if m < 1:
                    continue
                rows = q[b * n + t, h * G:(h + 1) * G].double()
                p = torch.softmax(rows @ k[:m].T * scale, -1)
                reach = max(reach, float((rows.abs() @ k[:m].abs().T).max()) * abs(scale))
                out[b * n + t, h * G:(h + 1) * G] = p @ v[:m]
                w[:m] += p.sum(0)
            weights[b, h] = w
    return out, weights, reach


def evict_row(weight, pos, keep_from, budget):
    """For one row of n > budget entries: source slot of every slot below the budget."""
    n = len(weight)
    first = sorted(range(n), key=lambda j: (pos[j] < keep_from, -weight[j] if pos[j] < keep_from else 0.0, j))[:budget]
    stay = set(first)
    src = list(range(budget))
    holes = [j for j in range(budget) if j not in stay]
    for d, s in zip(holes, [j for j in sorted(stay) if j >= budget]):
        src[d] = s
    return src


def verify(target, draft, tokens, uniform, count):
    """tokens [seqs][n+1], accepted [seqs], in whole numbers throughout."""
    B, n1, V = target.shape
    out, acc = np.full((B, n1), -1, np.int64), np.zeros(B, np.int64)
    for b in range(B):
        n, a, bad = int(count[b]), 0, False
        while a < n:
            x = int(tokens[b, a])
            if not 0 <= x < V:
                bad = True
                break
            q = np.float32(draft[b, a, x]) if draft is not None else np.float32(1)
            if not np.float32(uniform[b, a]) * q < np.float32(target[b, a, x]):
                break
            a += 1
        p = target[b, a].astype(np.float32)
        d = p
        if a < n and not bad:
            if draft is not None:
                d = p - draft[b, a].astype(np.float32)
            else:
                d = p.copy()
                d[int(tokens[b, a])] -= np.float32(1)
        fixed = lambda z: [int(round(float(np.clip(y, 0, 1)) * 2 ** 40)) for y in z]  # noqa: E731  (half to even)
        w = fixed(d)
        if sum(w) == 0:
            w = fixed(p)
        r = sum(w) * int(float(uniform[b, n1 - 1]) * 2 ** 24) >> 24
        tok, c = 0, 0
        for j, x in enumerate(w):
            c += x
            if c > r:
                tok = j
                break
        out[b, :a] = tokens[b, :a]
        out[b, a], acc[b] = tok, a
    return out, acc
