"""Plain forms of the step operators (plans, rotary positions), one sequence or one pair at a time."""
from __future__ import annotations

import math

import torch

BAD_INDEX, NO_PAGES = 1, 4


def plan(new, kv, held, shared, nxt, table, free, count, *, page, pool, total):
    """Everything a plan leaves behind, and its error bits; lists in, lists out. free[count:] holds what was there before."""
    B, width, cap = len(kv), len(table[0]) if table else 1, len(free)
    table, free = [list(r) for r in table], list(free)
    err = 0

    def cut(x, lo, hi):
        nonlocal err
        if not lo <= x <= hi:
            err |= BAD_INDEX
        return min(max(x, lo), hi)
    new = [cut(x, 0, 1 << 40) for x in (new or [0] * B)]
    kv = [cut(x, 0, width * page) for x in kv]
    held = [cut(x, 0, width) for x in held]
    shared = [min(cut(x, 0, 1 << 40), h) for x, h in zip(shared or [0] * B, held)]
    count = cut(count, 0, cap)
    ends, fits = 0, []
    for n, L in zip(new, kv):
        ends += n
        ok = (n == 0 or ends <= total) and -(-(L + n) // page) <= width
        fits.append(ok)
        if not ok:
            err |= BAD_INDEX
    top, keep = count, []
    for s in range(B):
        k = max(-(-(kv[s] + new[s]) // page), shared[s]) if fits[s] else held[s]
        keep.append(min(k, held[s]))
        for j in range(keep[s], held[s]):
            if top == cap:
                err |= BAD_INDEX
                break
            free[top] = table[s][j]
            top += 1
    cu, slots, pos, seq = [0], [], [], []
    kv_out, held_out, nxt_out = [], [], []
    asked, stack = 0, top
    for s in range(B):
        need = max(0, -(-(kv[s] + new[s]) // page) - held[s]) if fits[s] else 0
        asked += need
        ok = fits[s]
        if need and asked > stack:
            ok = False
            err |= NO_PAGES
        if ok:
            for j in range(need):
                top -= 1
                table[s][held[s] + j] = free[top]
        kv_out.append(kv[s] + new[s] if ok else kv[s])
        held_out.append(keep[s] + need if ok else (keep[s] if fits[s] else held[s]))
        first = kv[s] if nxt is None else nxt[s]
        if nxt is not None:
            nxt_out.append(first + (new[s] if ok else 0))
        for i in range(min(new[s], total - len(slots))):
            slot = -1
            if ok:
                p = table[s][(kv[s] + i) // page]
                if 0 <= p < pool:
                    slot = p * page + (kv[s] + i) % page
                else:
                    err |= BAD_INDEX
            slots.append(slot)
            pos.append(first + i)
            seq.append(s)
        cu.append(len(slots))
    pad = total - len(slots)
    return dict(cu_q=cu, slots=slots + [-1] * pad, pos=pos + [0] * pad, seq=seq + [-1] * pad, table=table, free=free,
                kv_len=kv_out, held=held_out, next_pos=nxt_out, count=top), err


def frequencies(dim, theta, scaling, factor=1.0, original=0, fast=32.0, slow=1.0):
    out = []
    for j in range(dim // 2):
        f = theta ** (-2.0 * j / dim)
        w = {"none": 1.0, "linear": 0.0}.get(scaling)
        if scaling == "turns":
            w = (original * f / (2 * math.pi) - slow) / (fast - slow)
        if scaling == "index":
            a, b = (dim * math.log(original / (2 * math.pi * x)) / (2 * math.log(theta)) for x in (fast, slow))
            a, b = max(0, math.floor(a)), min(dim - 1, math.ceil(b))
            w = 1 - (j - a) / (b - a if b > a else 0.001)
        w = min(1.0, max(0.0, w))
        out.append(f if w == 1.0 else w * f + (1 - w) * f / factor)
    return out


def rope(x, pos, freqs, first, layout, inverse=False, magnitude=1.0):
    """x [T, heads, D] turned, in 64 bits, and the error that the fp32 arithmetic and the rounding to x's type allow."""
    y, size = x.double(), x.double().abs()
    out, tol = y.clone(), torch.zeros_like(y)
    h = len(freqs)
    for j, f in enumerate(freqs):
        a, b = (first + j, first + j + h) if layout == "half" else (first + 2 * j, first + 2 * j + 1)
        t = pos.double() * (-f if inverse else f)
        c, s = (torch.cos(t) * magnitude)[:, None], (torch.sin(t) * magnitude)[:, None]
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
        # The reduced angle (below pi) rounded to fp32 is off by 2^-22.3, sine and cosine by 2 units in the last place (2^-23
        # below 1), their product with the magnitude, the two products and their sum by 2^-24 each: below 2^-21 of |a| + |b|.
        # The angle before the reduction is off by 2^-52 relative on either side.
        tol[..., a] = tol[..., b] = (size[..., a] + size[..., b]) * abs(magnitude) * (2.0 ** -21 + pos.double().abs() * f * 2.0 ** -51)[:, None]
    fi = torch.finfo(x.dtype)
    turned = tol > 0
    return out, torch.where(turned, tol + (out.abs() + tol) * fi.eps / 2 + fi.tiny * fi.eps / 2, tol)
