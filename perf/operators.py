"""Cases of the paged-cache operators: what is run, on which inputs, and what it cannot do without.

The four operators of a paged KV cache as a serving loop runs them:
  norm_rope   RMSNorm of queries and keys per head, RoPE in the same pass, K (and V) rows appended to the pages
  attn        attention of each sequence's new tokens (one, or a chunk) over its paged rows
  weights     the attention weight each cached row received, accumulated
  evict       the cache cut to a budget of rows by that weight, the most recent rows kept, rows compacted in order
"""
import math
import random

import torch

own = False

NEG = float("-inf")


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the queries and the shared KV row of one decode step of 16 sequences
        dict(name="norm_rope_step", op="norm_rope", tokens=16, heads=64, kv_heads=1, dim=512, shared=True, page=64, rope=64),
        # a prefill chunk of odd length, read out of a fused QKV projection, K and V kept apart
        dict(name="norm_rope_chunk", op="norm_rope", tokens=2039, heads=64, kv_heads=8, dim=128, shared=False, page=16, rope=128),
        # one sequence's single token over a short context: latency
        dict(name="attn_one", op="attn", batch=1, q=1, ctx=1000, heads=8, kv_heads=1, dim=128, shared=True, page=16, window=0,
             sink=True, rope=0),
        # a decode step of 16 sequences at 8K
        dict(name="attn_step", op="attn", batch=16, q=1, ctx=8192, heads=64, kv_heads=1, dim=512, shared=True, page=64, window=0,
             sink=True, rope=64),
        # a decode step over long caches: 1 GB of rows
        dict(name="attn_long", op="attn", batch=4, q=1, ctx=262144, heads=64, kv_heads=1, dim=512, shared=True, page=64, window=0,
             sink=True, rope=0),
        # a prefill chunk of 2048 tokens behind 14K cached ones
        dict(name="attn_chunk", op="attn", batch=1, q=2048, ctx=16384, heads=64, kv_heads=1, dim=512, shared=True, page=64, window=0,
             sink=True, rope=64),
        # a sliding-window layer over a ragged batch of chunks
        dict(name="attn_window", op="attn", batch=7, q=509, ctx=4099, heads=64, kv_heads=1, dim=512, shared=True, page=64, window=128,
             sink=True, rope=0),
        # single tokens and chunks in one batch, grouped heads, K and V kept apart
        dict(name="attn_mixed", op="attn", batch=24, q=257, ctx=5003, heads=32, kv_heads=8, dim=128, shared=False, page=16, window=0,
             sink=False, rope=0),
        # the weights of a decode step of 16 sequences
        dict(name="weights_step", op="weights", batch=16, q=1, ctx=8192, heads=64, kv_heads=1, dim=512, shared=True, page=64, window=0),
        # the weights of a prefill chunk
        dict(name="weights_chunk", op="weights", batch=2, q=1023, ctx=8191, heads=64, kv_heads=1, dim=512, shared=True, page=64,
             window=0),
        # a few short caches cut to 512 rows
        dict(name="evict_short", op="evict", batch=3, ctx=1537, budget=512, recent=64, kv_heads=4, dim=128, shared=False, page=16),
        # long caches cut by half
        dict(name="evict_long", op="evict", batch=4, ctx=65536, budget=32768, recent=128, kv_heads=1, dim=512, shared=True, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    """(heads, kv_heads, dim, shared): any grouping, K and V in one row or apart (apart up to 256 channels)."""
    dim = rng.choice([128, 256, 512])
    shared = dim == 512 or rng.random() < 0.4
    kv = 1 if shared and rng.random() < 0.6 else rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 64])
    while kv * group > 64:
        group = max(1, group // 2)
    return kv * group, kv, dim, shared


def draw(rng):
    op = rng.choice(["norm_rope", "attn", "attn", "attn", "weights", "evict"])
    heads, kv, dim, shared = _heads(rng)
    page = rng.choice([8, 16, 32, 48, 64, 128, 256])
    if op == "norm_rope":
        return dict(op=op, tokens=_log(rng, 1, 4096), heads=heads, kv_heads=kv, dim=dim, shared=shared, page=page,
                    rope=rng.choice([2, 64, 128, dim if dim <= 128 else 64]))
    if op == "evict":
        batch = _log(rng, 1, 32)
        ctx = _log(rng, 100, max(200, 262144 // batch))
        budget = max(2, int(ctx * rng.uniform(0.2, 0.9)))
        return dict(op=op, batch=batch, ctx=ctx, budget=budget, recent=rng.randrange(0, min(budget, 512)), kv_heads=kv, dim=dim,
                    shared=shared, page=page)
    batch = _log(rng, 1, 64)
    q = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
    ctx = max(q, _log(rng, 64, 131072))
    while batch * ctx * kv * dim > 4 * 262144 * 512:
        ctx = max(q, ctx // 2)
        batch = max(1, batch - batch // 4) if ctx == q else batch
    while batch * q * heads * ctx > 2048 * 64 * 16384 or batch * q * heads * ctx * dim > 2048 * 64 * 14336 * 512:
        q = max(1, q // 2)
        batch = max(1, batch - 1) if q == 1 else batch
    c = dict(op=op, batch=batch, q=q, ctx=max(q, ctx), heads=heads, kv_heads=kv, dim=dim, shared=shared, page=page,
             window=rng.choice([0, 0, rng.randrange(1, 2048)]))
    if op == "attn":
        c.update(sink=rng.random() < 0.5, rope=rng.choice([0, 64]))
    return c


def _lengths(case):
    """The batch's (new tokens, cached rows with them) per sequence: the first as long as the case says, the others shorter."""
    r = random.Random(case["batch"] * 1000003 + case["ctx"])
    kv = [case["ctx"]] + [r.randint(max(1, case["ctx"] // 2), case["ctx"]) for _ in range(case["batch"] - 1)]
    most = case.get("q", 1)
    q = [most] + [1 if r.random() < 0.4 else r.randint(1, most) for _ in range(case["batch"] - 1)]
    return [min(a, b) for a, b in zip(q, kv)], kv


# ------------------------------------------------------------------------------------------ inputs
def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    x = torch.empty(*shape, device="cuda", dtype=dtype)
    return x.normal_(0.0, std, generator=g)


def _cache(case, g, rows, tables=1):
    """Pages and `tables` block tables of [batch, pages for `rows` rows], over pages in a random order, none shared."""
    per = -(-rows // case["page"])
    n = tables * case["batch"] * per + 3
    order = torch.randperm(n, generator=g, device="cuda")[:n - 3].to(torch.int32)
    shape = (n, case["page"], case["kv_heads"], case["dim"])
    k = _normal(g, *shape)
    v = None if case["shared"] else _normal(g, *shape)
    return k, v, [t.contiguous() for t in order.view(tables, case["batch"], per)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=case)
    D, KV = case["dim"], case["kv_heads"]
    if case["op"] == "norm_rope":
        T, H = case["tokens"], case["heads"]
        parts = H + KV * (1 if case["shared"] else 2)
        x = _normal(g, T, parts, D, std=1.5)                         # the projection's output, heads side by side
        s["q"], s["k"] = x[:, :H], x[:, H:H + KV]
        s["v"] = None if case["shared"] else x[:, H + KV:]
        s["gamma_q"] = _normal(g, D, std=0.1, dtype=torch.float32) + 1
        s["gamma_k"] = _normal(g, D, std=0.1, dtype=torch.float32) + 1
        n = -(-(T + 3 * case["page"]) // case["page"])
        s["k_pages"] = _normal(g, n, case["page"], KV, D)
        s["v_pages"] = None if case["shared"] else _normal(g, n, case["page"], KV, D)
        s["slots"] = torch.randperm(n * case["page"], generator=g, device="cuda")[:T].contiguous()
        s["slots"][::37] = -1                                        # padding: nothing is appended
        s["pos"] = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
        s["q_out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "evict":
        _, kv = _lengths(case)
        s["k_pages"], s["v_pages"], (s["table"], s["out_table"]) = _cache(case, g, case["ctx"], 2)
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        w = torch.empty(case["batch"], case["ctx"], device="cuda").exponential_(1.0, generator=g).pow_(3)
        s["acc"] = (w * 64).round_() / 64                            # long-tailed, with ties and zeros
        s["acc_out"] = torch.zeros(case["batch"], case["ctx"], device="cuda")
        s["kv_len_out"] = torch.zeros_like(s["kv_len"])
        s["keep"] = torch.empty(case["batch"], case["budget"], dtype=torch.int32, device="cuda")
    else:
        ql, kv = _lengths(case)
        T, H = sum(ql), case["heads"]
        s["q_len"], s["kv_host"] = ql, kv
        s["q"] = _normal(g, T, H, D, std=2.0)
        s["k_pages"], s["v_pages"], (s["table"],) = _cache(case, g, case["ctx"])
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["cu_q"] = torch.tensor([0] + ql, device="cuda").cumsum(0).to(torch.int32)
        if case["op"] == "attn":
            s["sink"] = _normal(g, H, dtype=torch.float32) if case["sink"] else None
            first = torch.randint(0, 1 << 20, (case["batch"],), generator=g, device="cuda")
            seq = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"), torch.tensor(ql, device="cuda"))
            s["pos"] = first[seq] + torch.arange(T, device="cuda") if case["rope"] else None
            s["out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty(T, H, device="cuda")
        else:
            s["lse"] = _statistics(s)
            s["acc_in"] = torch.empty(case["batch"], case["ctx"], device="cuda").exponential_(1.0, generator=g)
            s["acc"] = torch.zeros(case["batch"], case["ctx"], device="cuda")
    if own:
        s["call"] = _plan(s)
    return s


def _statistics(s):
    """log(sum(exp)) of every query's scores, as the attention before would have left it."""
    case = s["case"]
    sc, vis, valid = _scores(s)
    sc = torch.logsumexp(torch.where(vis, sc, NEG), -1)
    B, KV, G, Lq = sc.shape
    return sc.permute(0, 3, 1, 2).reshape(B, Lq, KV * G)[valid].contiguous()


def _plan(s):
    """The prepared calls and workspaces a serving loop keeps."""
    import compressed_sparse_attention_08_gb300 as m
    case = s["case"]
    ws = lambda n: torch.empty(max(256, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    if case["op"] == "norm_rope":
        a = m.norm_rope_args(s["q"], s["q_out"], s["pos"], k=s["k"], k_pages=s["k_pages"], v=s["v"], v_pages=s["v_pages"],
                             slots=s["slots"], gamma_q=s["gamma_q"], gamma_k=s["gamma_k"], rope_dim=case["rope"])
        return lambda: m.dsv4_norm_rope_append(a)
    if case["op"] == "attn":
        a = m.paged_attn_args(s["q"], s["out"], s["k_pages"], s["table"], s["cu_q"], s["kv_len"], v_pages=s["v_pages"],
                              max_q=case["q"], sink=s["sink"], lse=s["lse"], window=case["window"], out_rope_pos=s["pos"],
                              out_rope_dim=case["rope"])
        w = ws(m.dsv4_paged_attn_workspace_size(a))
        return lambda: m.dsv4_paged_attn(a, w)
    if case["op"] == "weights":
        a = m.paged_weights_args(s["q"], s["lse"], s["k_pages"], s["table"], s["cu_q"], s["kv_len"], s["acc"], acc_in=s["acc_in"],
                                 max_q=case["q"], window=case["window"])
        w = ws(m.dsv4_paged_attn_weights_workspace_size(a))
        return lambda: m.dsv4_paged_attn_weights(a, w)
    a = m.paged_evict_args(s["k_pages"], s["table"], s["kv_len"], s["acc"], s["keep"], budget=case["budget"], recent=case["recent"],
                           v_pages=s["v_pages"], out_table=s["out_table"], kv_len_out=s["kv_len_out"], acc_out=s["acc_out"])
    w = ws(m.dsv4_paged_evict_workspace_size(a))
    return lambda: m.dsv4_paged_evict(a, w)


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
    else:
        {"norm_rope": _norm_rope, "attn": _attn, "weights": _weights, "evict": _evict}[op](s)
    if op == "norm_rope":
        return dict(q=s["q_out"], k=s["k_pages"], v=s["v_pages"])
    if op == "attn":
        return dict(out=s["out"], lse=s["lse"])
    if op == "weights":
        return dict(acc=s["acc"])
    return dict(keep=s["keep"], kv_len=s["kv_len_out"], acc=s["acc_out"], k=s["k_pages"], v=s["v_pages"])


def _rotated(x, pos, rope, sign):
    """x [T, H, D] with the pairs (2j, 2j+1) of its last `rope` channels turned by sign * pos * 10000^(-2j/rope)."""
    D = x.shape[-1]
    f = 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64, device=x.device) / rope)
    a = sign * pos.double()[:, None] * f
    c, n = a.cos().float()[:, None], a.sin().float()[:, None]
    e, o = x[..., D - rope::2], x[..., D - rope + 1::2]
    return torch.cat([x[..., :D - rope], torch.stack([e * c - o * n, e * n + o * c], -1).flatten(-2)], -1)


def _normed(x, gamma, pos, rope):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma
    return _rotated(x, pos, rope, 1.0).to(torch.bfloat16)


def _norm_rope(s):
    rope = s["case"]["rope"]
    s["q_out"].copy_(_normed(s["q"], s["gamma_q"], s["pos"], rope))
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    s["k_pages"].flatten(0, 1)[at] = _normed(s["k"], s["gamma_k"], s["pos"], rope)[kept]
    if s["v"] is not None:
        s["v_pages"].flatten(0, 1)[at] = s["v"][kept]


def _rows(pages, table):
    """The paged rows in order: [batch, rows, kv_heads, dim] in 32 bits."""
    return pages[table.long()].flatten(1, 2).float()


def _scores(s):
    """Scores [batch, kv_heads, group, new tokens, rows], where they are visible, and which padded tokens are real."""
    case = s["case"]
    B, KV, D = case["batch"], case["kv_heads"], case["dim"]
    dev = s["q"].device
    n = torch.tensor(s["q_len"], device=dev)
    i = torch.arange(case["q"], device=dev)
    valid = i < n[:, None]
    tok = torch.where(valid, s["cu_q"][:-1, None].long() + i, 0)
    q = s["q"][tok].float().view(B, case["q"], KV, -1, D).permute(0, 2, 3, 1, 4)
    k = _rows(s["k_pages"], s["table"]).permute(0, 2, 3, 1)
    G = q.shape[2]
    sc = torch.matmul(q.reshape(B, KV, -1, D), k).mul_(1.0 / math.sqrt(D)).view(B, KV, G, case["q"], -1)
    at = s["kv_len"].long()[:, None] - n[:, None] + i                # each new token's own row
    j = torch.arange(sc.shape[-1], device=dev)
    vis = (j <= at[..., None]) & valid[..., None]
    if case["window"]:
        vis = vis & (j > at[..., None] - case["window"])
    return sc, vis[:, None, None], valid


def _attn(s):
    case = s["case"]
    B, KV, D, H = case["batch"], case["kv_heads"], case["dim"], case["heads"]
    sc, vis, valid = _scores(s)
    sc = torch.where(vis, sc, NEG)
    m = sc.amax(-1, keepdim=True)
    sink = None if s["sink"] is None else s["sink"].view(1, KV, -1, 1, 1)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = m.masked_fill(m == NEG, 0.0)
    p = sc.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - m)
    v = _rows(s["k_pages"] if s["v_pages"] is None else s["v_pages"], s["table"]).permute(0, 2, 1, 3)
    G = p.shape[2]
    o = torch.matmul(p.view(B, KV, -1, p.shape[-1]), v).view(B, KV, G, case["q"], D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B, case["q"], H, D)[valid]
    lse = (m + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, case["q"], H)[valid]
    if case["rope"]:
        o = _rotated(o, s["pos"], case["rope"], -1.0)
    s["out"].copy_(o)
    s["lse"].copy_(lse)


def _weights(s):
    case = s["case"]
    sc, vis, valid = _scores(s)
    B, KV, G, Lq, _ = sc.shape
    lse = torch.zeros(B, Lq, KV * G, device=sc.device)
    lse[valid] = s["lse"]
    p = torch.where(vis, sc.sub_(lse.view(B, Lq, KV, G).permute(0, 2, 3, 1)[..., None]), NEG).exp_()
    w = p.sum((1, 2, 3))[:, :case["ctx"]]
    own_row = torch.arange(case["ctx"], device=sc.device) < s["kv_len"][:, None]
    s["acc"].copy_(torch.where(own_row, s["acc_in"] + w, s["acc"]))


def _evict(s):
    case = s["case"]
    n, recent, budget, page = s["kv_len"].long()[:, None], case["recent"], case["budget"], case["page"]
    j = torch.arange(case["ctx"], device=n.device)
    old = j < n - recent
    order = torch.sort(torch.where(old, s["acc"], NEG), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order))
    kept = ((old & (rank < budget - recent)) | ~old | (n <= budget)) & (j < n)
    b, src = kept.nonzero(as_tuple=True)
    dst = (kept.cumsum(1) - 1)[b, src]
    s["keep"].fill_(-1)
    s["keep"][b, dst] = src.to(torch.int32)
    s["kv_len_out"].copy_(kept.sum(1))
    s["acc_out"][b, dst] = s["acc"][b, src]
    frm = s["table"][b, src // page].long() * page + src % page
    to = s["out_table"][b, dst // page].long() * page + dst % page
    for pages in (s["k_pages"], s["v_pages"]):
        if pages is not None:
            pages.flatten(0, 1)[to] = pages.flatten(0, 1)[frm]


# ------------------------------------------------------------------------------------------ floors
def _visible(case):
    """(query, row) pairs that are visible, and rows that some query sees."""
    pairs = rows = 0
    for q, n in zip(*_lengths(case)):
        w = case["window"] or n
        ends = range(n - q + 1, n + 1)
        pairs += sum(min(e, w) for e in ends)
        rows += min(n, w + q - 1)
    return pairs, rows


def work(case):
    D, KV = case["dim"], case["kv_heads"]
    both = 1 if case["shared"] else 2
    if case["op"] == "norm_rope":
        T = case["tokens"]
        stored = T - len(range(0, T, 37))
        return dict(bytes=T * case["heads"] * D * 4 + T * 16 + stored * KV * D * 4 * both + D * 8, flops=T * (case["heads"] + KV) * D * 8)
    if case["op"] == "evict":
        _, kv = _lengths(case)
        kept = sum(min(n, case["budget"]) for n in kv)
        return dict(bytes=sum(kv) * 4 + kept * (KV * D * 4 * both + 12), flops=0)
    ql, kv = _lengths(case)
    pairs, rows = _visible(case)
    q = sum(ql) * case["heads"]
    if case["op"] == "attn":
        return dict(bytes=q * (D * 4 + 4) + rows * KV * D * 2 * both, flops=4 * D * case["heads"] * pairs)
    return dict(bytes=q * (D * 2 + 4) + rows * KV * D * 2 + sum(kv) * 8, flops=2 * D * case["heads"] * pairs)


# ------------------------------------------------------------------------------------------ in 64 bits
def _turn64(x, pos, rope, sign):
    D = x.shape[-1]
    y = x.clone()
    for j in range(rope // 2):
        a = sign * pos.double() * 10000.0 ** (-2.0 * j / rope)
        c, n = torch.cos(a)[:, None], torch.sin(a)[:, None]
        e, o = x[..., D - rope + 2 * j], x[..., D - rope + 2 * j + 1]
        y[..., D - rope + 2 * j] = e * c - o * n
        y[..., D - rope + 2 * j + 1] = e * n + o * c
    return y


def exact(case, seed):
    s = prepare(case, seed)
    D, KV, page = case["dim"], case["kv_heads"], case["page"]
    if case["op"] == "norm_rope":
        def one(x, gamma):
            x = x.double()
            return _turn64(x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma.double(), s["pos"], case["rope"], 1)
        k_pages, v_pages = s["k_pages"].double(), None if case["shared"] else s["v_pages"].double()
        k = one(s["k"], s["gamma_k"])
        at = s["slots"].tolist()
        here = [t for t, a in enumerate(at) if a >= 0]
        to = torch.tensor([at[t] for t in here], dtype=torch.long, device="cuda")
        k_pages.view(-1, KV, D)[to] = k[here]
        if v_pages is not None:
            v_pages.view(-1, KV, D)[to] = s["v"].double()[here]
        return dict(q=one(s["q"], s["gamma_q"]), k=k_pages, v=v_pages)
    if case["op"] == "evict":
        out = dict(keep=None, kv_len=None, acc=s["acc_out"].double(), k=s["k_pages"].clone(), v=None if case["shared"] else s["v_pages"].clone())
        acc = s["acc"].cpu()
        for b, n in enumerate(s["kv_len"].tolist()):
            old = max(0, n - case["recent"])
            rows = list(range(n))
            if n > case["budget"]:
                best = sorted(range(old), key=lambda i, a=acc[b].tolist(): (-a[i], i))[:case["budget"] - case["recent"]]
                rows = sorted(best) + list(range(old, n))
            src = torch.tensor(rows, device="cuda")
            dst = torch.arange(len(rows), device="cuda")
            out["acc"][b, :len(rows)] = s["acc"][b, src].double()
            frm = s["table"][b].long()[src // page] * page + src % page
            to = s["out_table"][b].long()[dst // page] * page + dst % page
            for name, pages in (("k", s["k_pages"]), ("v", s["v_pages"])):
                if pages is not None:
                    out[name].view(-1, KV, D)[to] = pages.view(-1, KV, D)[frm]
        return {n: x if x is None else x.double() for n, x in out.items()}
    pairs, _ = _visible(case)
    if 4 * D * case["heads"] * pairs > 6e12:
        return None
    H, G = case["heads"], case["heads"] // KV
    T = s["q"].shape[0]
    out = torch.zeros(T, H, D, dtype=torch.float64, device="cuda") if case["op"] == "attn" else None
    lse = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    acc = None if out is not None else s["acc"].double()
    t0 = 0
    for b, (q, n) in enumerate(zip(s["q_len"], s["kv_host"])):
        row = torch.arange(n, device="cuda")
        at = s["table"][b].long()[row // page] * page + row % page
        if acc is not None:
            acc[b, :n] = s["acc_in"][b, :n].double()
        step = max(1, (1 << 28) // (n * G))
        for h in range(KV):
            k = s["k_pages"].view(-1, KV, D)[at, h].double()
            v = k if s["v_pages"] is None else s["v_pages"].view(-1, KV, D)[at, h].double()
            hs = slice(h * G, (h + 1) * G)
            for i in range(0, q, step):
                i1 = min(q, i + step)
                end = n - q + torch.arange(i, i1, device="cuda")
                hide = row > end[:, None]
                if case["window"]:
                    hide |= row <= end[:, None] - case["window"]
                z = torch.einsum("tgd,nd->gtn", s["q"][t0 + i:t0 + i1, hs].double(), k) / math.sqrt(D)
                z.masked_fill_(hide, NEG)
                if out is None:
                    acc[b, :n] += torch.exp(z - s["lse"][t0 + i:t0 + i1, hs].double().t()[..., None]).sum((0, 1))
                    continue
                if s["sink"] is not None:
                    z = torch.cat([z, s["sink"][hs].double()[:, None, None].expand(G, i1 - i, 1)], -1)
                l = torch.logsumexp(z, -1)
                lse[t0 + i:t0 + i1, hs] = l.t()
                out[t0 + i:t0 + i1, hs] = torch.einsum("gtn,nd->tgd", torch.exp(z[..., :n] - l[..., None]), v)
        t0 += q
    if out is None:
        return dict(acc=acc)
    return dict(out=_turn64(out, s["pos"], case["rope"], -1) if case["rope"] else out, lse=lse)
