"""Cases of a serving step around the paged cache: what is run, on which inputs, and what it cannot do without.

The three operators, in the order in which a step uses them:
  plan      block tables, slot maps, positions and offsets of a step from the requests' lengths, with a stack of free pages
  rope      rotary positions (pairs side by side or half a part apart, part of the head, scaled frequencies, either direction),
            the keys and values appended to the pages or left beside one another
  prefix    attention of each sequence's new tokens where groups of sequences share the first rows of their caches
"""
import math
import random

import torch

own = False

NEG = float("-inf")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the bookkeeping of one decode step of 16 sequences: latency
        dict(name="plan_step", op="plan", batch=16, q=1, ctx=8192, page=64),
        # 2,000 requests, chunks and single tokens mixed: the largest batch a scheduler forms
        dict(name="plan_mixed", op="plan", batch=2000, q=97, ctx=5003, page=16),
        # one decode step of 16 sequences, grouped heads, appended to the pages
        dict(name="rope_step", op="rope", tokens=16, heads=64, kv_heads=8, dim=128, rope=128, first=0, layout="half", inverse=False,
             scaling="index", dtype="bf16", append=True, page=64),
        # a prefill chunk of odd length, frequencies scaled for a long context, appended to the pages
        dict(name="rope_chunk", op="rope", tokens=2039, heads=64, kv_heads=8, dim=128, rope=128, first=0, layout="half",
             inverse=False, scaling="turns", dtype="bf16", append=True, page=16),
        # a chunk of wide heads, of which the last 64 channels turn
        dict(name="rope_part", op="rope", tokens=1023, heads=64, kv_heads=1, dim=512, rope=64, first=448, layout="interleaved",
             inverse=False, scaling="linear", dtype="fp16", append=False, page=64),
        # the gradients of queries and keys on their way back through the rotation
        dict(name="rope_back", op="rope", tokens=8192, heads=32, kv_heads=8, dim=128, rope=128, first=0, layout="interleaved",
             inverse=True, scaling="none", dtype="fp32", append=False, page=64),
        # two samples of one short prompt: latency
        dict(name="prefix_two", op="prefix", batch=2, groups=1, q=1, prefix=1000, ctx=1100, heads=8, kv_heads=1, dim=128,
             shared=True, page=16, sink=True, rope=0),
        # 64 requests behind one system prompt of 32K, grouped heads, K and V apart
        dict(name="prefix_step", op="prefix", batch=64, groups=1, q=1, prefix=32768, ctx=33792, heads=32, kv_heads=8, dim=128,
             shared=False, page=64, sink=False, rope=0),
        # a share of 16 heads of a wide shared-KV layer, 48 requests over a document of 64K
        dict(name="prefix_wide", op="prefix", batch=48, groups=1, q=1, prefix=65536, ctx=67001, heads=16, kv_heads=1, dim=512,
             shared=True, page=64, sink=True, rope=64),
        # three prompts of their own, ragged groups
        dict(name="prefix_groups", op="prefix", batch=45, groups=3, q=1, prefix=12345, ctx=14003, heads=16, kv_heads=2, dim=256,
             shared=True, page=16, sink=True, rope=64),
        # questions of up to 256 tokens about one text, prefilled together
        dict(name="prefix_chunks", op="prefix", batch=16, groups=1, q=256, prefix=32768, ctx=33205, heads=32, kv_heads=8, dim=128,
             shared=False, page=64, sink=False, rope=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope", "prefix", "prefix", "prefix"])
    page = rng.choice([8, 16, 32, 48, 64, 128, 256])
    if op == "plan":
        return dict(op=op, batch=_log(rng, 1, 2000), q=rng.choice([1, _log(rng, 2, 96)]), ctx=_log(rng, 100, 5000), page=max(16, page))
    if op == "rope":
        dim = rng.choice([64, 96, 128, 192, 256, 512])
        layout = rng.choice(["interleaved", "half"])
        rope = rng.choice([dim, 64, dim // 2, dim // 4 * 2 - 2 * rng.randrange(0, 3)])
        first = rng.choice([0, dim - rope])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 8])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 8192 * 40 * 128 * 4 // ((heads + 2 * kv) * dim * (4 if dtype == "fp32" else 2))
        inverse = rng.random() < 0.3
        return dict(op=op, tokens=_log(rng, 1, min(16384, most)), heads=heads, kv_heads=kv, dim=dim, rope=rope, first=first,
                    layout=layout, inverse=inverse, scaling=rng.choice(["none", "linear", "turns", "index"]), dtype=dtype,
                    append=not inverse and rng.random() < 0.6, page=page)
    dim = rng.choice([128, 128, 256, 512])
    shared = dim == 512 or rng.random() < 0.4
    kv = 1 if shared and rng.random() < 0.6 else rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    batch = _log(rng, 2, 64)
    groups = rng.choice([1, 1, 1, 2, 4])
    q = 1 if rng.random() < 0.6 else _log(rng, 2, 256)
    own_rows = _log(rng, max(q, 8), 2048)
    prefix = _log(rng, 100, 65536)
    pairs = 6e11 / (4 * dim * kv * group)                               # the largest listed case's products
    while batch * q * (prefix + own_rows) > pairs and (q > 1 or prefix > 100):
        q, prefix = max(1, q // 2), max(100, prefix * 3 // 4)
    while kv * dim * (groups * prefix + batch * own_rows) * (1 if shared else 2) > 8 * 128 * 2 * 65536:
        prefix, own_rows = max(100, prefix // 2), max(q, own_rows // 2)
    return dict(op=op, batch=batch, groups=min(groups, batch), q=q, prefix=prefix, ctx=prefix + own_rows, heads=kv * group,
                kv_heads=kv, dim=dim, shared=shared, page=page, sink=rng.random() < 0.5, rope=rng.choice([0, 64]))


def _lengths(case):
    """The batch's (new tokens, cached rows) per sequence. For prefix: the rows with the new tokens', the first sequence's
    as many as the case says, the others' own rows fewer; group of each sequence and prefix of each group."""
    r = random.Random(case["batch"] * 1000003 + case["ctx"])
    B, most, ctx = case["batch"], case["q"], case["ctx"]
    q = [most] + [1 if r.random() < 0.5 else r.randint(1, most) for _ in range(B - 1)]
    if case["op"] == "plan":
        kv = [ctx] + [r.randint(0, ctx) for _ in range(B - 1)]
        for i in range(1, B, 11):
            kv[i], q[i] = 0, 0                                           # requests that ended
        return q, kv
    G = case["groups"]
    start = [0] + sorted(r.sample(range(1, B), G - 1)) + [B]
    pre = [case["prefix"]] + [r.randint(max(1, case["prefix"] // 2), case["prefix"]) for _ in range(G - 1)]
    of = [max(g for g in range(G) if start[g] <= s) for s in range(B)]
    most_own = ctx - case["prefix"]
    rows = [ctx] + [0] * (B - 1)
    for s in range(1, B):
        rows[s] = pre[of[s]] + r.randint(q[s], max(q[s], most_own))
    return q, rows, start, pre, of


# ------------------------------------------------------------------------------------------ inputs
def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    x = torch.empty(*shape, device="cuda", dtype=dtype)
    return x.normal_(0.0, std, generator=g)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=case)
    {"plan": _prepare_plan, "rope": _prepare_rope, "prefix": _prepare_prefix}[case["op"]](case, g, s)
    if own:
        s["call"] = _plan(s)
    return s


def _prepare_plan(case, g, s):
    """Requests in the middle of their lives: pages held, a few too many where rows were evicted, the first shared by some."""
    page, B = case["page"], case["batch"]
    q, kv = _lengths(case)
    r = random.Random(int(torch.randint(1 << 30, (1,), generator=g, device="cuda")))
    held = [-(-n // page) + (r.randint(1, 5) if r.random() < 0.1 else 0) for n in kv]
    shared = [min(h, 2) if i % 3 == 0 else 0 for i, h in enumerate(held)]
    per = -(-(max(kv) + max(q)) // page) + 6
    pages = sum(-(-n // page) for n in kv) + sum(q) // page + 6 * B + 64
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    own_pages = torch.arange(per, device="cuda")[None] < _i32(held)[:, None]
    table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
    table[own_pages] = order[:sum(held)]
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    left = pages - sum(held)
    free[:left] = order[sum(held):]
    s.update(new_len=_i32(q), kv_len=_i32(kv), held=_i32(held), shared=_i32(shared), table=table, free=free,
             count=_i32([left]), pages=pages,
             next_pos=torch.randint(0, 1 << 20, (B,), generator=g, device="cuda"))
    T = -(-(sum(q) + 1) // 64) * 64                                      # the step's buffers are a little longer than the step
    for n in ("kv_len", "held", "next_pos", "count"):
        s[n + "_out"] = torch.zeros_like(s[n])
    s["cu_q"] = _i32([0] * (B + 1))
    s["slots"] = torch.zeros(T, dtype=torch.int64, device="cuda")
    s["pos"] = torch.zeros(T, dtype=torch.int64, device="cuda")
    s["seq"] = _i32([0] * T)


def _prepare_rope(case, g, s):
    T, H, KV, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    dt = TYPES[case["dtype"]]
    x = _normal(g, T, H + 2 * KV, D, std=1.5, dtype=dt)                  # a fused projection's output, heads side by side
    s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + KV], x[:, H + KV:] if case["append"] else None
    s["pos"] = torch.randint(0, 1 << 17, (T,), generator=g, device="cuda")
    s["q_out"] = torch.empty(T, H, D, dtype=dt, device="cuda")
    s["slots"] = s["v_out"] = None
    if case["append"]:
        n = -(-(T + 3 * case["page"]) // case["page"])
        s["k_out"], s["v_out"] = _normal(g, n, case["page"], KV, D, dtype=dt), _normal(g, n, case["page"], KV, D, dtype=dt)
        s["slots"] = torch.randperm(n * case["page"], generator=g, device="cuda")[:T].contiguous()
        s["slots"][::37] = -1                                            # padding: nothing is appended
    else:
        s["k_out"] = torch.empty(T, KV, D, dtype=dt, device="cuda")
    s["scaled"] = dict(scaling=case["scaling"], factor=8.0 if case["scaling"] != "none" else 1.0, original_len=4096,
                       beta_fast=32.0, beta_slow=1.0, magnitude=1.2079 if case["scaling"] == "index" else 1.0)


def _prepare_prefix(case, g, s):
    page, B, KV, D, H = case["page"], case["batch"], case["kv_heads"], case["dim"], case["heads"]
    q, rows, start, pre, of = _lengths(case)
    full = [p // page for p in pre]                                      # whole pages are shared; a prefix may end inside one
    per = -(-max(rows) // page)
    n = sum(full) + sum(-(-rows[i] // page) - full[of[i]] for i in range(B)) + 3
    shape = (n, page, KV, D)
    s["k_pages"] = _normal(g, *shape)
    s["v_pages"] = None if case["shared"] else _normal(g, *shape)
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
    at = sum(full)
    for i in range(B):
        a = sum(full[:of[i]])
        f, c = full[of[i]], -(-rows[i] // page)
        table[i, :f] = order[a:a + f]
        table[i, f:c] = order[at:at + c - f]
        at += c - f
    for i in range(B):                                                   # the prefix's last rows, inside each one's own page
        f, p = full[of[i]], pre[of[i]] % page
        i0 = start[of[i]]
        if p and i != i0:
            for pages in (s["k_pages"], s["v_pages"]):
                if pages is not None:
                    pages[table[i, f].long(), :p] = pages[table[i0, f].long(), :p]
    s["table"], s["q_len"], s["rows"], s["start"], s["pre"] = table, q, rows, start, pre
    T = sum(q)
    s["q"] = _normal(g, T, H, D, std=2.0)
    s["kv_len"], s["cu_q"] = _i32(rows), _i32([0] + q).cumsum(0).to(torch.int32)
    s["prefix_len"], s["group_start"] = _i32(pre), _i32(start)
    s["sink"] = _normal(g, H, dtype=torch.float32) if case["sink"] else None
    s["pos"] = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda") if case["rope"] else None
    s["out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(T, H, device="cuda")


def _plan(s):
    """The prepared calls and workspaces a serving loop keeps."""
    import compressed_sparse_attention_08_gb300 as m
    case = s["case"]
    ws = lambda n: torch.empty(max(256, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    if case["op"] == "plan":
        a = m.paged_plan_args(s["new_len"], s["kv_len"], s["held"], s["table"], s["free"], s["count"], s["cu_q"], s["slots"],
                              page_size=case["page"], num_pages=s["pages"], shared=s["shared"], pos=s["pos"], seq=s["seq"],
                              next_pos=s["next_pos"], kv_len_out=s["kv_len_out"], held_out=s["held_out"],
                              free_count_out=s["count_out"], next_pos_out=s["next_pos_out"])
        w = ws(m.dsv4_paged_plan_workspace_size(a))
        return lambda: m.dsv4_paged_plan(a, w)
    if case["op"] == "rope":
        a = m.rope_args(s["q"], s["q_out"], s["pos"], k=s["k"], k_out=s["k_out"], v=s["v"], v_out=s["v_out"], slots=s["slots"],
                        rope_dim=case["rope"], first=case["first"], layout=case["layout"], inverse=case["inverse"],
                        rope_theta=10000.0, **s["scaled"])
        return lambda: m.dsv4_rope(a)
    a = m.paged_prefix_args(s["q"], s["out"], s["k_pages"], s["table"], s["cu_q"], s["kv_len"], s["prefix_len"],
                            group_start=s["group_start"], v_pages=s["v_pages"], sink=s["sink"], lse=s["lse"],
                            out_rope_pos=s["pos"], out_rope_dim=case["rope"])
    w = ws(m.dsv4_paged_prefix_attn_workspace_size(a))
    return lambda: m.dsv4_paged_prefix_attn(a, w)


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
    else:
        {"plan": _step, "rope": _rope, "prefix": _prefix}[op](s)
    if op == "plan":
        return {n: s[n] for n in ("cu_q", "slots", "pos", "seq", "table", "free", "kv_len_out", "held_out", "count_out", "next_pos_out")}
    if op == "rope":
        return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])
    return dict(out=s["out"], lse=s["lse"])


def _step(s):
    page = s["case"]["page"]
    n, L, held, shared = (s[k].long() for k in ("new_len", "kv_len", "held", "shared"))
    dev = n.device
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    s["cu_q"].copy_(cu)
    want = (L + n + page - 1) // page
    after = torch.maximum(torch.minimum(want, held), torch.minimum(shared, held))   # pages kept of those held
    j = torch.arange(s["table"].shape[1], device=dev)
    back = s["table"][(j >= after[:, None]) & (j < held[:, None])]                  # the others, in order
    count = s["count"].long()
    at = torch.arange(back.numel(), device=dev)
    s["free"][count + at] = back
    stack = count + back.numel()
    take = (want - held).clamp(min=0)
    ends = take.cumsum(0)
    served = (take == 0) | (ends <= stack)
    got = (j >= held[:, None]) & (j < want[:, None]) & served[:, None]
    k = (ends - take)[:, None] + j - held[:, None]                                  # the pages taken, counted from the top
    s["table"][got] = s["free"][stack - 1 - k[got]]
    s["count_out"].copy_(stack - torch.where(served, take, 0).sum())
    s["kv_len_out"].copy_(torch.where(served, L + n, L))
    s["held_out"].copy_(torch.where(served, torch.maximum(after, want), held))
    s["next_pos_out"].copy_(s["next_pos"] + torch.where(served, n, 0))
    t = torch.arange(s["slots"].numel(), device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    real = b < n.numel()
    b = torch.where(real, b, 0)
    i = t - cu[b]
    row = torch.where(real, L[b] + i, 0)
    s["slots"].copy_(torch.where(real & served[b], s["table"][b, row // page].long() * page + row % page, -1))
    s["pos"].copy_(torch.where(real, s["next_pos"][b] + i, 0))
    s["seq"].copy_(torch.where(real, b, -1))


def _frequencies(case, scaled, dev):
    d = case["rope"]
    j = torch.arange(d // 2, dtype=torch.float64, device=dev)
    f = 10000.0 ** (-2.0 * j / d)
    if scaled["scaling"] == "none":
        return f
    low = f / scaled["factor"]
    if scaled["scaling"] == "linear":
        return low
    turns = scaled["original_len"] * f / (2 * math.pi)                              # in the original context
    if scaled["scaling"] == "turns":
        keep = ((turns - scaled["beta_slow"]) / (scaled["beta_fast"] - scaled["beta_slow"])).clamp(0, 1)
    else:
        at = [d * math.log(scaled["original_len"] / (b * 2 * math.pi)) / (2 * math.log(10000.0))
              for b in (scaled["beta_fast"], scaled["beta_slow"])]
        a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
        keep = 1 - ((j - a) / (b - a if b > a else 0.001)).clamp(0, 1)
    return low * (1 - keep) + f * keep


def _turned(x, s):
    """x [T, heads, D] with the case's part turned, in 32 bits (angles in 64)."""
    case = s["case"]
    x = x.float()
    first, d = case["first"], case["rope"]
    a = s["pos"].double()[:, None] * _frequencies(case, s["scaled"], x.device) * (-1.0 if case["inverse"] else 1.0)
    m = s["scaled"]["magnitude"]
    c, n = (a.cos() * m).float()[:, None], (a.sin() * m).float()[:, None]
    part = x[..., first:first + d]
    if case["layout"] == "half":
        e, o = part[..., :d // 2], part[..., d // 2:]
        part = torch.cat([e * c - o * n, e * n + o * c], -1)
    else:
        e, o = part[..., 0::2], part[..., 1::2]
        part = torch.stack([e * c - o * n, e * n + o * c], -1).flatten(-2)
    return torch.cat([x[..., :first], part, x[..., first + d:]], -1)


def _rope(s):
    s["q_out"].copy_(_turned(s["q"], s))
    k = _turned(s["k"], s).to(s["k_out"].dtype)
    if s["slots"] is None:
        s["k_out"].copy_(k)
        return
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    s["k_out"].flatten(0, 1)[at] = k[kept]
    s["v_out"].flatten(0, 1)[at] = s["v"][kept]


def _rows(pages, table, row):
    """Rows `row` [.., n] of the tables [.., pages] in 32 bits: [.., n, kv_heads, dim]."""
    page = pages.shape[1]
    return pages[torch.gather(table, -1, row // page).long(), row % page].float()


def _prefix(s):
    """Scores of a group's tokens with the prefix's rows, of each sequence's with its own, one softmax over both."""
    case = s["case"]
    B, KV, D, H = case["batch"], case["kv_heads"], case["dim"], case["heads"]
    G, scale, dev = H // KV, 1.0 / math.sqrt(case["dim"]), s["q"].device
    sink = None if s["sink"] is None else s["sink"].view(1, KV, G, 1)
    out, lse = [], []
    v_pages = s["k_pages"] if s["v_pages"] is None else s["v_pages"]
    for g, P in enumerate(s["pre"]):
        b0, b1 = s["start"][g], s["start"][g + 1]
        t0, t1 = sum(s["q_len"][:b0]), sum(s["q_len"][:b1])
        q = s["q"][t0:t1].float().view(-1, KV, G, D)
        row = torch.arange(P, device=dev)
        kp, vp = (_rows(p, s["table"][b0], row) for p in (s["k_pages"], v_pages))
        a = torch.matmul(q.permute(1, 0, 2, 3).reshape(KV, -1, D), kp.permute(1, 2, 0)).mul_(scale).view(KV, -1, G, P)
        # each sequence's own rows: padded to the longest
        ql = torch.tensor(s["q_len"][b0:b1], device=dev)
        n = torch.tensor(s["rows"][b0:b1], device=dev) - P
        own_row = P + torch.arange(int(max(s["rows"][b0:b1])) - P, device=dev).expand(b1 - b0, -1)
        i = torch.arange(max(s["q_len"][b0:b1]), device=dev)
        valid = i < ql[:, None]
        tok = torch.where(valid, torch.cat([ql.new_zeros(1), ql.cumsum(0)])[:-1, None] + i, 0)
        ko, vo = (_rows(p, s["table"][b0:b1].clamp(min=0), own_row) for p in (s["k_pages"], v_pages))
        z = torch.matmul(q[tok].permute(0, 2, 1, 3, 4).reshape(b1 - b0, KV, -1, D), ko.permute(0, 2, 3, 1)).mul_(scale)
        z = z.view(b1 - b0, KV, i.numel(), G, -1)
        seen = torch.arange(z.shape[-1], device=dev) <= (n[:, None] - ql[:, None] + i)[..., None]
        z = torch.where(seen[:, None, :, None], z, NEG)
        own_tok = torch.where(valid, tok, -1)
        zt = z.permute(0, 2, 1, 3, 4)[own_tok >= 0]                                 # [tokens, KV, G, rows]
        m = torch.maximum(a.amax(-1).permute(1, 0, 2), zt.amax(-1))[..., None]
        if sink is not None:
            m = torch.maximum(m, sink)
        a = a.sub_(m[..., 0].permute(1, 0, 2)[..., None]).exp_()
        total = a.sum(-1).permute(1, 0, 2)[..., None]
        o = torch.matmul(a.view(KV, -1, P), vp.permute(1, 0, 2)).view(KV, -1, G, D).permute(1, 0, 2, 3)
        p = zt.sub_(m).exp_()
        total = total + p.sum(-1, keepdim=True)
        if sink is not None:
            total = total + torch.exp(sink - m)
        pz = torch.zeros_like(z).permute(0, 2, 1, 3, 4)
        pz[own_tok >= 0] = p
        oz = torch.matmul(pz.permute(0, 2, 1, 3, 4).reshape(b1 - b0, KV, -1, pz.shape[-1]), vo.permute(0, 2, 1, 3))
        o = o + oz.view(b1 - b0, KV, i.numel(), G, D).permute(0, 2, 1, 3, 4)[own_tok >= 0]
        out.append((o / total).reshape(-1, H, D))
        lse.append((m + total.log()).reshape(-1, H))
    o = torch.cat(out)
    if case["rope"]:
        d = case["rope"]
        f = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=dev) / d)
        a = -s["pos"].double()[:, None] * f
        c, n = a.cos().float()[:, None], a.sin().float()[:, None]
        e, b = o[..., D - d::2], o[..., D - d + 1::2]
        o = torch.cat([o[..., :D - d], torch.stack([e * c - b * n, e * n + b * c], -1).flatten(-2)], -1)
    s["out"].copy_(o)
    s["lse"].copy_(torch.cat(lse))


# ------------------------------------------------------------------------------------------ floors
def work(case):
    if case["op"] == "plan":
        q, kv = _lengths(case)
        pages = sum(-(-(a + b) // case["page"]) - -(-b // case["page"]) for a, b in zip(q, kv))
        return dict(bytes=sum(q) * 20 + case["batch"] * (4 * 5 + 8 * 2 + 4 * 2) + pages * 8, flops=0)
    D, KV, H = case["dim"], case["kv_heads"], case["heads"]
    if case["op"] == "rope":
        T, size = case["tokens"], 4 if case["dtype"] == "fp32" else 2
        stored = T - len(range(0, T, 37)) if case["append"] else T
        kv = stored * KV * (2 if case["append"] else 1)
        return dict(bytes=2 * (T * H + kv) * D * size + T * (16 if case["append"] else 8), flops=(T * H + stored * KV) * case["rope"] * 3)
    q, rows, start, pre, of = _lengths(case)
    both = 1 if case["shared"] else 2
    pairs = sum(sum(range(n - a + 1, n + 1)) for a, n in zip(q, rows))
    cached = sum(pre) + sum(n - pre[g] for n, g in zip(rows, of))
    return dict(bytes=sum(q) * H * (D * 4 + 4) + cached * KV * D * 2 * both, flops=4 * D * H * pairs)


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "prefix": _exact_prefix}[case["op"]](case, s)


def _exact_plan(case, s):
    """One request after another, on the host."""
    page = case["page"]
    new, kv, held, shared, nxt = (s[n].tolist() for n in ("new_len", "kv_len", "held", "shared", "next_pos"))
    table, free, count = s["table"].tolist(), s["free"].tolist(), s["count"].tolist()[0]
    for b in range(case["batch"]):
        keep = max(-(-(kv[b] + new[b]) // page), shared[b])
        for j in range(keep, held[b]):
            free[count] = table[b][j]
            count += 1
        held[b] = min(held[b], keep)
    top, dry = count, False
    cu, slots, pos, seq = [0], [], [], []
    for b in range(case["batch"]):
        need = max(0, -(-(kv[b] + new[b]) // page) - held[b])
        dry = dry or need > top
        ok = need == 0 or not dry
        for j in range(need if ok else 0):
            top -= 1
            table[b][held[b] + j] = free[top]
        for i in range(new[b]):
            row = kv[b] + i
            slots.append(table[b][row // page] * page + row % page if ok else -1)
            pos.append(nxt[b] + i)
            seq.append(b)
        cu.append(cu[-1] + new[b])
        if ok:
            held[b], kv[b], nxt[b] = held[b] + need, kv[b] + new[b], nxt[b] + new[b]
    pad = s["slots"].numel() - len(slots)
    dev = lambda x, like: torch.tensor(x, dtype=like.dtype, device="cuda")  # noqa: E731
    return dict(cu_q=dev(cu, s["cu_q"]), slots=dev(slots + [-1] * pad, s["slots"]), pos=dev(pos + [0] * pad, s["pos"]),
                seq=dev(seq + [-1] * pad, s["seq"]), table=dev(table, s["table"]), free=dev(free, s["free"]),
                kv_len_out=dev(kv, s["kv_len"]), held_out=dev(held, s["held"]), count_out=dev([top], s["count"]),
                next_pos_out=dev(nxt, s["next_pos"]))


def _exact_rope(case, s):
    d, first, sc = case["rope"], case["first"], s["scaled"]

    def one(x):
        y = x.double()
        for j in range(d // 2):
            f = 10000.0 ** (-2.0 * j / d)
            slow = f / sc["factor"]
            if sc["scaling"] == "linear":
                f = slow
            elif sc["scaling"] == "turns":
                t = sc["original_len"] * f / (2 * math.pi)
                w = min(1.0, max(0.0, (t - sc["beta_slow"]) / (sc["beta_fast"] - sc["beta_slow"])))
                f = w * f + (1 - w) * slow
            elif sc["scaling"] == "index":
                def at(turns):
                    return d * math.log(sc["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
                lo, hi = max(0, math.floor(at(sc["beta_fast"]))), min(d - 1, math.ceil(at(sc["beta_slow"])))
                w = min(1.0, max(0.0, (j - lo) / ((hi - lo) if hi > lo else 0.001)))
                f = f * (1 - w) + slow * w
            z = torch.polar(torch.full_like(s["pos"], 1).double() * sc["magnitude"], s["pos"].double() * (-f if case["inverse"] else f))
            a, b = (first + j, first + j + d // 2) if case["layout"] == "half" else (first + 2 * j, first + 2 * j + 1)
            w = torch.complex(x[..., a].double(), x[..., b].double()) * z[:, None]
            y[..., a], y[..., b] = w.real, w.imag
        return y
    q, k = one(s["q"]), one(s["k"])
    if s["slots"] is None:
        return dict(q=q, k=k, v=None)
    pages = [s["k_out"].double(), s["v_out"].double()]
    at = s["slots"].tolist()
    here = [t for t, a in enumerate(at) if a >= 0]
    to = torch.tensor([at[t] for t in here], dtype=torch.long, device="cuda")
    for p, x in zip(pages, (k, s["v"].double())):
        p.view(-1, case["kv_heads"], case["dim"])[to] = x[here]
    return dict(q=q, k=pages[0], v=pages[1])


def _exact_prefix(case, s):
    """Each sequence over its own table, as if nothing were shared."""
    D, KV, page, H = case["dim"], case["kv_heads"], case["page"], case["heads"]
    G, T = H // KV, s["q"].shape[0]
    if work(case)["flops"] > 6e12:
        return None
    out = torch.zeros(T, H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, rows) in enumerate(zip(s["q_len"], s["rows"])):
        row = torch.arange(rows, device="cuda")
        at = s["table"][b].long()[row // page] * page + row % page
        end = rows - n + torch.arange(n, device="cuda")
        for h in range(KV):
            k = s["k_pages"].view(-1, KV, D)[at, h].double()
            v = k if s["v_pages"] is None else s["v_pages"].view(-1, KV, D)[at, h].double()
            hs = slice(h * G, (h + 1) * G)
            z = torch.einsum("tgd,nd->gtn", s["q"][t0:t0 + n, hs].double(), k) / math.sqrt(D)
            z.masked_fill_(row > end[:, None], NEG)
            full = z
            if s["sink"] is not None:
                full = torch.cat([z, s["sink"][hs].double()[:, None, None].expand(G, n, 1)], -1)
            l = torch.logsumexp(full, -1)
            lse[t0:t0 + n, hs] = l.t()
            out[t0:t0 + n, hs] = torch.einsum("gtn,nd->tgd", torch.exp(z - l[..., None]), v)
        t0 += n
    for j in range(case["rope"] // 2):
        c = D - case["rope"] + 2 * j
        z = torch.polar(torch.ones(T, dtype=torch.float64, device="cuda"), -s["pos"].double() * 10000.0 ** (-2.0 * j / case["rope"]))
        w = torch.complex(out[..., c], out[..., c + 1]) * z[:, None]
        out[..., c], out[..., c + 1] = w.real, w.imag
    return dict(out=out, lse=lse)
