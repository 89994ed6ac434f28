"""Plain 64-bit implementations of the operators for prompts and trees of drafts, on the CPU, for the tests: no shared code
with the library."""
from __future__ import annotations

import math

import torch

from tests.serve_ref import gather, slot_place

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def visible(i, t, b, n, ln, case):
    """Slots that row t (at slot i) of sequence b sees: bool [ln]."""
    j = torch.arange(ln)
    lo = 0 if not case.get("first") else int(case["first"][b][t])
    if case.get("tree"):
        node = j - (ln - n)
        word = case["tree"][b][t]
        bits = torch.tensor([1 if s < ln - n or (word >> (s - (ln - n))) & 1 else 0 for s in range(ln)], dtype=torch.bool)
        return bits & (j >= lo) & ((node < 0) | (node < n))
    hi = i + 1
    if case.get("prefix"):
        hi = max(hi, min(int(case["prefix"][b]), ln))
    if case.get("window"):
        lo = max(lo, i - case["window"] + 1)
    return (j >= lo) & (j < hi)


def attention(q, kpool, vpool, table, lens, new, page_size, scale, cap=0.0, slopes=None, skip_bad_v=False, **case):
    """(out, bound) [seqs*n][q_heads][dim] float64: the bound is how far an implementation may be off that rounds p to the
    cache's type, keeps f32 otherwise, and does not round the output.

    A score's f32 sums are off by at most 2^-20 scale sum|q||k|, the capped score besides by cap 2^-20 (an exponential, an
    addition, a reciprocal and the product: below 8 half steps of values up to 2 cap), the bias by 2^-21 of itself; a
    probability is off by twice that relatively, by 2^-18 for exponential, maximum and sums, by half a step of the type for
    its rounding, and (f16) by 2^-31 of the row's largest absolutely."""
    B, H, D = len(lens), kpool.shape[1], kpool.shape[3]
    n_all = q.shape[0] // B
    G = q.shape[1] // H
    u = HALF[kpool.dtype]
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for b in range(B):
        n, ln = new[b], lens[b]
        if n == 0:
            continue
        i = torch.arange(ln - n, ln)
        seen = torch.stack([visible(int(x), t, b, n, ln, case) for t, x in enumerate(i)])
        for h in range(H):
            k, v = gather(kpool, table, page_size, b, h, ln), gather(vpool, table, page_size, b, h, ln)
            if skip_bad_v:
                v = torch.where(torch.isfinite(v), v, torch.zeros((), dtype=torch.float64))
            for gq in range(G):
                head = h * G + gq
                rows = q[b * n_all:b * n_all + n, head].double()
                s = rows @ k.T * scale
                off = 2.0 ** -20 * abs(scale) * (rows.abs() @ k.abs().T)
                if cap:
                    s = cap * torch.tanh(s / cap)
                    off = off + cap * 2.0 ** -20
                if slopes is not None:
                    bias = float(slopes[head]) * (torch.arange(ln)[None] - i[:, None]).double()
                    s = s + bias
                    off = off + bias.abs() * 2.0 ** -21
                s = s.masked_fill(~seen, -math.inf)
                empty = ~seen.any(1)
                p = torch.softmax(s, -1)
                p[empty] = 0.0
                ds = torch.where(seen, off, torch.zeros((), dtype=torch.float64)).amax(1, keepdim=True)
                av = v.abs()
                out[b * n_all:b * n_all + n, head] = p @ v
                floor = 2.0 ** -31 * (seen.double() @ av) if kpool.dtype == torch.float16 else 0.0
                tol[b * n_all:b * n_all + n, head] = (u * 1.01 + 2 * ds + 2.0 ** -18) * (p @ av) + floor
    return out, tol


def norm_rope(x, w, eps, pos, axis, fixed, rot, magnitude, interleaved):
    """x [rows][heads][dim] f32 -> (rotated float64, bound for an f32 computation of it).

    Off by: the mean of squares (dim additions: dim/2 half steps, halved by the root), the root's 2 ulp, two products; then
    the rotation's 8 half steps of |a| + |b|."""
    x = x.double()
    D = x.shape[-1]
    rel = 0.0
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
        rel = (D / 2 + 8) * 2.0 ** -24
    y, tol = x.clone(), x.abs() * (rel + 2.0 ** -24)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        where = pos[axis[i] if axis is not None else 0]
        ang = torch.tensor([2 * math.pi * (((int(p) * fixed[i]) % (1 << 64)) / 2.0 ** 64) for p in where], dtype=torch.float64)
        c, s = (torch.cos(ang) * magnitude)[:, None], (torch.sin(ang) * magnitude)[:, None]
        u, v = x[:, :, a], x[:, :, b]
        y[:, :, a], y[:, :, b] = u * c - v * s, u * s + v * c
        tol[:, :, a] = tol[:, :, b] = (u.abs() + v.abs()) * magnitude * (rel + 8 * 2.0 ** -24)
    return y, tol


def keep(pools, table, lens, new, page_size, path, count):
    """Moves entries of CPU tensors [pages][heads][page_size](...) in place, one after the other."""
    for b in range(len(lens)):
        for i in range(count[b]):
            s, d = (slot_place(table, page_size, b, lens[b] - new[b] + x) for x in (int(path[b][i]), i))
            for x in pools:
                x[d[0], :, d[1]] = x[s[0], :, s[1]].clone()
