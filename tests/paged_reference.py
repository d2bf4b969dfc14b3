"""Plain 64-bit forms of the paged-cache operators, one sequence and one head at a time."""
from __future__ import annotations

import math

import torch

F32_STEP = 2.0 ** -24                    # half a step of fp32, relative
BF16_STEP = 2.0 ** -8                    # half a step of bf16, relative


def rotate(x, pos, rope, theta, sign):
    """x [T, H, D] in 64 bits: the pairs of the last `rope` channels turned by sign * pos * theta^(-2j/rope)."""
    y = x.clone()
    D = x.shape[-1]
    for j in range(rope // 2):
        a = sign * pos.double() * theta ** (-2.0 * j / rope)
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        e, o = x[..., D - rope + 2 * j], x[..., D - rope + 2 * j + 1]
        y[..., D - rope + 2 * j] = e * c - o * s
        y[..., D - rope + 2 * j + 1] = e * s + o * c
    return y


def norm_rope(x, gamma, pos, rope, theta, eps):
    x = x.double()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    if gamma is not None:
        y = y * gamma.double()
    return rotate(y, pos, rope, theta, 1)


def rows_of(pages, table, s, n):
    """Rows 0 .. n - 1 of sequence s: [n, kv_heads, dim]; only the pages in use are looked up."""
    ps = pages.shape[1]
    j = torch.arange(n, device=pages.device)
    page = table[s, : -(-n // ps)].long() if n else table[s, :0].long()
    return pages[page[j // ps], j % ps]


def bounds(L, n, window):
    """[lo, hi) of each of a sequence's n newest tokens."""
    out = []
    for t in range(n):
        hi = max(L - n + t + 1, 0)
        out.append((max(hi - window, 0) if window else 0, hi))
    return out


def attention(q, k_pages, v_pages, table, cu, lens, scale, window=0, sink=None, rope=0, pos=None, theta=1e4):
    """(out, lse, spread, score error): spread is sum p |v| per output, the score error the bound of the fp32 products."""
    T, H, D = q.shape
    KV = k_pages.shape[2]
    dev = q.device
    out = torch.zeros(T, H, D, dtype=torch.float64, device=dev)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    spread = torch.zeros_like(out)
    serr = torch.zeros(T, H, dtype=torch.float64, device=dev)
    for s, L in enumerate(lens):
        t0, n = cu[s], cu[s + 1] - cu[s]
        if n == 0:
            continue
        first = min((lo for lo, hi in bounds(L, n, window) if hi > lo), default=0)
        kk = rows_from(k_pages, table, s, first, L)
        vv = kk if v_pages is None else rows_from(v_pages, table, s, first, L)
        for t, (lo, hi) in enumerate(bounds(L, n, window)):
            for h in range(KV):
                hs = slice(h * (H // KV), (h + 1) * (H // KV))
                x = q[t0 + t, hs].double()
                k = kk[lo - first:hi - first, h].double() if hi > lo else kk[:0, h].double()
                v = vv[lo - first:hi - first, h].double() if hi > lo else vv[:0, h].double()
                z = x @ k.t() * scale
                zs = z if sink is None else torch.cat([z, sink[hs].double()[:, None]], 1)
                if zs.shape[1] == 0:
                    continue
                m = torch.logsumexp(zs, 1)
                lse[t0 + t, hs] = m
                p = torch.exp(z - m[:, None])
                out[t0 + t, hs] = p @ v
                spread[t0 + t, hs] = p @ v.abs()
                if hi > lo:
                    # D products summed in fp32 in some order, and the products with the scale and log2(e)
                    serr[t0 + t, hs] = ((x.abs() @ k.abs().t()) * abs(scale)).amax(1) * (D + 8) * 2 * F32_STEP
    if rope:
        out = rotate(out, pos, rope, theta, -1)
        spread[..., -rope:] = (spread[..., -rope::2] + spread[..., -rope + 1::2]).repeat_interleave(2, -1)
    return out, lse, spread, serr


def rows_from(pages, table, s, first, n):
    """Rows first .. n - 1 of sequence s; the pages before and after are not looked up."""
    ps = pages.shape[1]
    j = torch.arange(first, max(n, first), device=pages.device)
    return pages[table[s].long()[j // ps], j % ps]


def check_attention(got, lse, ref):
    out, rl, spread, serr = ref
    assert torch.isfinite(got.float()).all()
    # each P and the output are rounded to bf16, a score is off by serr (its exponential by as much, relative), and
    # the fp32 sums, exponentials and the rotation by a few steps
    tol = BF16_STEP * out.abs() + (BF16_STEP + 3 * serr[..., None] + 2.0 ** -16) * spread * (1 + BF16_STEP) + 1e-30
    err = (got.double() - out).abs()
    bad = err > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs off; worst {(err / tol).max():.2f} times the tolerance"
    if lse is not None:
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse), empty)
        e = (lse.double() - rl).abs()[~empty]
        t = (serr + 2.0 ** -18 * (1 + rl.abs()))[~empty]
        assert (e <= t).all(), f"lse off by {(e / t).max():.2f} times the tolerance"


def weights(q, lse, k_pages, table, cu, lens, scale, acc, acc_in, window=0):
    """acc in 64 bits, and the error the fp32 scores allow."""
    T, H, D = q.shape
    KV = k_pages.shape[2]
    out = acc.double().clone()
    tol = torch.zeros_like(out)
    for s, L in enumerate(lens):
        t0, n = cu[s], cu[s + 1] - cu[s]
        w = torch.zeros(L, dtype=torch.float64, device=q.device)
        e = torch.zeros_like(w)
        b = bounds(L, n, window)
        first = min((lo for lo, hi in b if hi > lo), default=L)
        kk = rows_from(k_pages, table, s, first, L)
        for t, (lo, hi) in enumerate(b):
            if hi <= lo:
                continue
            for h in range(KV):
                hs = slice(h * (H // KV), (h + 1) * (H // KV))
                x, k = q[t0 + t, hs].double(), kk[lo - first:hi - first, h].double()
                z = x @ k.t() * scale
                l = lse[t0 + t, hs].double()[:, None]
                p = torch.exp(z - l)
                err = (x.abs() @ k.abs().t()) * abs(scale) * (D + 8) * 2 * F32_STEP + (l.abs() + z.abs()) * 4 * F32_STEP
                w[lo:hi] += p.sum(0)
                e[lo:hi] += (p * (2 * err + 2.0 ** -20)).sum(0)
        base = acc_in[s, :L].double() if acc_in is not None else 0.0
        out[s, :L] = base + w
        tol[s, :L] = e + (out[s, :L].abs()) * (n * H + 2) * F32_STEP + 1e-30
    return out, tol


def evict(lens, acc, budget, recent):
    """Kept rows of each sequence."""
    kept = []
    for s, n in enumerate(lens):
        rows = list(range(n))
        if n > budget:
            a = acc[s].tolist()
            old = sorted(range(max(0, n - recent)), key=lambda i: (-a[i], i))[:budget - recent]
            rows = sorted(old) + list(range(max(0, n - recent), n))
        kept.append(rows)
    return kept
