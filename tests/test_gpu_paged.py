"""The paged cache on the GPU: norm + rotation + append, attention, weights and eviction against
their plain 64-bit forms, at the sizes, layouts and masks where they can go wrong.

Tolerances are derived in paged_reference.py from the roundings the kernels make (bf16 of P and
of the output, fp32 sums); integers and moved rows are compared bit for bit.
"""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import paged_reference as ref  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_sparse_attention_08_gb300 import _build
    _build.build()


def lib():
    import compressed_sparse_attention_08_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=BF):
    return torch.empty(*shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)


def ws_for(n):
    return torch.full((max(n, 256),), 0xA5, dtype=torch.uint8, device="cuda")     # (needs no initialisation)


class Cache:
    """Pages in random order; table entries past a sequence's rows (and before its window) name no page."""

    def __init__(self, g, lens, page, kv, dim, shared=True, spare=3, first=None, poison=True):
        self.lens, self.page = lens, page
        per = max(1, max(-(-n // page) for n in lens))
        need = [-(-n // page) for n in lens]
        n = sum(need) + spare
        self.k = normal(g, n, page, kv, dim)
        self.v = None if shared else normal(g, n, page, kv, dim)
        order = torch.randperm(n, generator=g, device="cuda").tolist()
        table = [[(1 << 30) if i % 2 else -7 for i in range(per)] for _ in lens]
        used = torch.zeros(n, page, dtype=torch.bool, device="cuda")
        for s, c in enumerate(need):
            for i in range(c):
                table[s][i] = order.pop()
            for j in range(lens[s]):
                used[table[s][j // page], j % page] = True
            if first is not None:                                     # rows before `first` are freed pages
                for i in range(first[s] // page):
                    used[table[s][i]] = False
                    table[s][i] = -1
        if poison:                                                    # what nobody sees holds NaN
            for p in (self.k, self.v):
                if p is not None:
                    p[~used] = float("nan")
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")


def cu_of(ns):
    out = [0]
    for n in ns:
        out.append(out[-1] + n)
    return out


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attend(c, q, cu, *, window=0, sink=None, lse=True, max_q=None, pos=None, rope=64, scale=None, pad=0, ws=None):
    m = lib()
    T, H, D = q.shape
    out = torch.full((T, H, D), 7.0, dtype=BF, device="cuda")
    l = torch.full((T, H), 7.0, device="cuda") if lse else None
    a = m.paged_attn_args(q, out, c.k, c.table, i32(cu), c.kv_len, v_pages=c.v, max_q=max_q, sink=sink, lse=l,
                          window=window, scale=scale, out_rope_pos=pos, out_rope_dim=rope)
    ws = ws_for(m.dsv4_paged_attn_workspace_size(a)) if ws is None else ws
    m.dsv4_paged_attn(a, ws)
    assert m.dsv4_read_error_word(ws) == (0, 0)
    return out, l


# ------------------------------------------------------------------ attention
SHAPES = [(64, 1, 512, True), (8, 1, 128, True), (16, 1, 256, True), (32, 4, 128, False), (5, 5, 128, False),
          (12, 2, 256, False), (1, 1, 512, True), (128, 1, 512, True), (96, 1, 128, True), (200, 1, 256, True),
          (24, 3, 512, False)]


@pytest.mark.parametrize("H, KV, D, shared", SHAPES)
@pytest.mark.parametrize("page", [8, 48, 64])
def test_single_tokens(H, KV, D, shared, page):
    g = gen(H * 7 + D + page)
    lens = [1, 2, 127, 128, 129, 300, 1000]
    c = Cache(g, lens, page, KV, D, shared)
    q = normal(g, len(lens), H, D, std=2.0)
    sink = normal(g, H, dtype=torch.float32)
    cu = cu_of([1] * len(lens))
    out, lse = attend(c, q, cu, sink=sink, max_q=1)
    ref.check_attention(out, lse, ref.attention(q, c.k, c.v, c.table, cu, lens, 1 / math.sqrt(D), sink=sink))


@pytest.mark.parametrize("H, KV, D, shared", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 37, 128])
def test_chunks(H, KV, D, shared, window):
    """Ragged chunks: whole prompts, continued ones, empty ones, and chunks longer than a tile."""
    g = gen(H + D + window)
    ns, lens = [5, 0, 1, 33, 130, 7], [5, 0, 200, 140, 131, 500]
    first = [max(0, L - n + 1 - window) if window else 0 for n, L in zip(ns, lens)]
    c = Cache(g, lens, 16, KV, D, shared, first=first)
    cu = cu_of(ns)
    q = normal(g, cu[-1], H, D, std=2.0)
    out, lse = attend(c, q, cu, window=window, max_q=max(ns))
    ref.check_attention(out, lse, ref.attention(q, c.k, c.v, c.table, cu, lens, 1 / math.sqrt(D), window))


@pytest.mark.parametrize("D, max_q", [(512, 1), (512, 100), (128, 1), (128, 100), (256, 100)])
def test_tokens_that_see_nothing(D, max_q):
    """More tokens than rows: the first tokens stand before the cache. Output 0, lse the sink's or -inf."""
    g = gen(D)
    ns, lens = [9, 4, 3], [4, 0, 3]
    c = Cache(g, lens, 8, 1, D)
    cu = cu_of(ns)
    q = normal(g, cu[-1], 8, D)
    for sink in (None, normal(g, 8, dtype=torch.float32)):
        out, lse = attend(c, q, cu, sink=sink, max_q=max_q)
        r = ref.attention(q, c.k, None, c.table, cu, lens, 1 / math.sqrt(D), sink=sink)
        if sink is not None:
            for t in list(range(5)) + list(range(9, 13)):
                r[1][t] = sink.double()
        ref.check_attention(out, lse, r)
        assert (out[:5] == 0).all() and (out[9:13] == 0).all()


@pytest.mark.parametrize("H, D, shared", [(64, 512, True), (64, 128, False), (16, 256, True)])
def test_long_rows_are_split_and_merged(H, D, shared):
    """One sequence over every CTA, and one long beside short ones; the peak of the scores late, early and flat."""
    g = gen(3)
    lens = [20000, 1, 700]
    c = Cache(g, lens, 64, 1, D, shared)
    q = normal(g, 3, H, D, std=2.0)
    q[0, :8] *= 8                                   # scores of a few hundred: one row takes all
    q[0, 8:16] = 0                                  # flat
    pos = torch.tensor([5, 1 << 40, 123456], device="cuda")
    cu = [0, 1, 2, 3]
    sink = normal(g, H, dtype=torch.float32)
    out, lse = attend(c, q, cu, sink=sink, max_q=1, pos=pos)
    ref.check_attention(out, lse, ref.attention(q, c.k, c.v, c.table, cu, lens, 1 / math.sqrt(D), sink=sink, rope=64, pos=pos))


@pytest.mark.parametrize("rope", [2, 64, 128])
@pytest.mark.parametrize("H", [64, 6])
def test_output_rotation(rope, H):
    g = gen(rope)
    ns, lens = [40, 1], [40, 333]
    c = Cache(g, lens, 32, 1, 128)
    cu = cu_of(ns)
    q = normal(g, cu[-1], H, 128, std=2.0)
    pos = torch.randint(0, 1 << 20, (cu[-1],), generator=g, device="cuda")
    out, lse = attend(c, q, cu, pos=pos, rope=rope)
    ref.check_attention(out, lse, ref.attention(q, c.k, None, c.table, cu, lens, 1 / math.sqrt(128), rope=rope, pos=pos))


def test_scores_that_grow_along_the_cache():
    """Each unit outruns the reference maximum of the one before: the running output is rescaled every time."""
    g = gen(11)
    lens, D, H = [1500], 512, 64
    c = Cache(g, lens, 64, 1, D)
    base = torch.ones(D, device="cuda")
    for j in range(1500):
        c.k[c.table[0, j // 64], j % 64, 0] = (c.k[c.table[0, j // 64], j % 64, 0].float() * 0.1 + base * (j / 100)).to(BF)
    q = (normal(g, 3, H, D).float() * 0.1 + 1).to(BF)
    q[:, H // 2:] *= -1
    out, lse = attend(c, q, [0, 3])
    ref.check_attention(out, lse, ref.attention(q, c.k, None, c.table, [0, 3], lens, 1 / math.sqrt(D)))


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_scales(scale):
    g = gen(5)
    lens, ns = [300, 17], [2, 17]
    c = Cache(g, lens, 16, 2, 128, False)
    q = normal(g, 19, 8, 128)
    out, lse = attend(c, q, cu_of(ns), scale=scale)
    ref.check_attention(out, lse, ref.attention(q, c.k, c.v, c.table, cu_of(ns), lens, scale))


def test_strided_queries_and_rows_behind_the_last_sequence():
    """Queries inside a fused projection; tokens past cu_q[batch] keep what their outputs held."""
    g = gen(6)
    lens, ns = [100, 260], [3, 1]
    c = Cache(g, lens, 16, 1, 128)
    for extra in (0, 128, 8):
        x = torch.empty(9, 8 * 128 + extra, device="cuda", dtype=BF).normal_(generator=g)
        q = x[:, :1024].view(9, 8, 128) if extra == 0 else x.as_strided((9, 8, 128), (1024 + extra, 128, 1))
        out, lse = attend(c, q, cu_of(ns), max_q=3)
        r = ref.attention(q[:4], c.k, None, c.table, cu_of(ns), lens, 1 / math.sqrt(128))
        ref.check_attention(out[:4], lse[:4], r)
        assert (out[4:] == 7).all() and (lse[4:] == 7).all()


def test_pages_past_32_bit_offsets():
    """A pool of 6 GB: the rows of the sequence lie behind byte 2^32."""
    m = lib()
    g = gen(9)
    n, page, D = 96000, 64, 512
    k = torch.empty(n, page, 1, D, dtype=BF, device="cuda")
    k[-40:] = normal(g, 40, page, 1, D)
    table = torch.arange(n - 1, n - 33, -1, device="cuda").view(1, 32).to(torch.int32)
    c = Cache.__new__(Cache)
    c.k, c.v, c.table, c.kv_len, c.lens = k, None, table, i32([2000]), [2000]
    q = normal(g, 1, 64, D, std=2.0)
    out, lse = attend(c, q, [0, 1], max_q=1)
    ref.check_attention(out, lse, ref.attention(q, k, None, table, [0, 1], [2000], 1 / math.sqrt(D)))
    # and an append far behind
    x = normal(g, 2, 1, D)
    slots = torch.tensor([n * page - 1, (n - 36) * page + 5], device="cuda")
    pos = torch.tensor([3, 4], device="cuda")
    m.dsv4_norm_rope_append(m.norm_rope_args(None, None, pos, k=x, k_pages=k, slots=slots))
    want = ref.norm_rope(x, None, pos, 64, 1e4, 1e-6)
    got = k.view(-1, 1, D)[slots].double()
    assert (got - want).abs().max() <= BF_TOL * want.abs().max()


BF_TOL = 2.0 ** -8 + 2.0 ** -18


def test_a_graph_serves_every_step_and_results_repeat():
    """Captured once, replayed with other lengths and rows; two captures with a workspace of their own; bits repeat."""
    m = lib()
    g = gen(12)
    lens = [900, 64, 5, 2000]
    c = Cache(g, lens, 32, 1, 512, poison=False)
    q = normal(g, 4, 64, 512, std=2.0)
    out, lse = torch.empty_like(q), torch.empty(4, 64, device="cuda")
    acc = torch.zeros(4, 2048, device="cuda")
    cu = i32([0, 1, 2, 3, 4])
    a = m.paged_attn_args(q, out, c.k, c.table, cu, c.kv_len, max_q=1, lse=lse)
    b = m.paged_weights_args(q, lse, c.k, c.table, cu, c.kv_len, acc, max_q=1)
    wa, wb = ws_for(m.dsv4_paged_attn_workspace_size(a)), ws_for(m.dsv4_paged_attn_weights_workspace_size(b))
    m.dsv4_paged_attn(a, wa)
    m.dsv4_paged_attn_weights(b, wb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.dsv4_paged_attn(a, wa)
        m.dsv4_paged_attn_weights(b, wb)
    for step in range(3):
        now = [max(1, n - 31 * step) for n in lens]
        c.kv_len.copy_(i32(now))
        q.copy_(normal(g, 4, 64, 512, std=2.0))
        acc.fill_(-1)
        graph.replay()
        first = [x.clone() for x in (out, lse, acc)]
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(first, (out, lse, acc)))
        ref.check_attention(out, lse, ref.attention(q, c.k, None, c.table, [0, 1, 2, 3, 4], now, 1 / math.sqrt(512)))
        want, tol = ref.weights(q, lse, c.k, c.table, [0, 1, 2, 3, 4], now, 1 / math.sqrt(512), torch.full_like(acc, -1), None)
        assert ((acc.double() - want).abs() <= tol).all()
        assert all((acc[s, n:] == -1).all() for s, n in enumerate(now))


def test_streams():
    """Two calls at once on two streams, each with its workspace, as one after the other."""
    m = lib()
    g = gen(13)
    lens = [3000, 3000]
    c = Cache(g, lens, 64, 1, 512)
    qs = [normal(g, 2, 64, 512) for _ in range(2)]
    want = [attend(c, q, [0, 1, 2], max_q=1) for q in qs]
    side = [torch.cuda.Stream() for _ in qs]
    calls = []
    for q in qs:
        out, lse = torch.empty_like(q), torch.empty(2, 64, device="cuda")
        a = m.paged_attn_args(q, out, c.k, c.table, i32([0, 1, 2]), c.kv_len, max_q=1, lse=lse)
        calls.append((a, ws_for(m.dsv4_paged_attn_workspace_size(a)), out, lse))
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (a, w, _, _) in zip(side, calls):
            m.dsv4_paged_attn(a, w, stream=st)
    torch.cuda.synchronize()
    for (_, _, out, lse), (o, l) in zip(calls, want):
        assert torch.equal(out, o) and torch.equal(lse, l)


def test_many_sequences():
    """More sequences than CTAs, some without tokens, some without rows."""
    g = gen(14)
    lens = [(i * 37) % 260 for i in range(1200)]
    ns = [0 if i % 5 == 0 else (1 if lens[i] else 0) for i in range(1200)]
    c = Cache(g, lens, 16, 1, 128, poison=False)
    cu = cu_of(ns)
    q = normal(g, cu[-1], 8, 128, std=2.0)
    out, lse = attend(c, q, cu, max_q=1)
    ref.check_attention(out, lse, ref.attention(q, c.k, None, c.table, cu, lens, 1 / math.sqrt(128)))


def test_a_page_outside_the_pool_is_hidden_and_reported():
    m = lib()
    g = gen(15)
    lens, D = [200, 90], 128
    c = Cache(g, lens, 16, 1, D)
    q = normal(g, 2, 8, D)
    good = attend(c, q, [0, 1, 2], max_q=1)
    c.table[0, 3] = 1 << 20
    c.table[0, 12] = -1                              # the last page of the sequence
    out, lse, acc = torch.empty_like(q), torch.empty(2, 8, device="cuda"), torch.zeros(2, 256, device="cuda")
    a = m.paged_attn_args(q, out, c.k, c.table, i32([0, 1, 2]), c.kv_len, lse=lse)
    ws = ws_for(m.dsv4_paged_attn_workspace_size(a))
    m.dsv4_paged_attn(a, ws)
    assert m.dsv4_read_error_word(ws) == (m.DSV4_ERR_BAD_INDEX, m.DSV4_EWORD_BAD_INDEX)
    assert torch.equal(out[1], good[0][1])
    seen = torch.tensor([j for j in range(200) if j // 16 not in (3, 12)], device="cuda")
    k = c.k[c.table[0].long()[seen // 16], seen % 16, 0].double()
    p = torch.softmax(q[0].double() @ k.t() / math.sqrt(D), -1)
    assert ((out[0].double() - p @ k).abs() <= 2.0 ** -7 * (p @ k.abs()) + 2.0 ** -8 * (p @ k).abs()).all()
    b = m.paged_weights_args(q, lse, c.k, c.table, i32([0, 1, 2]), c.kv_len, acc, max_q=1)
    ws = ws_for(m.dsv4_paged_attn_weights_workspace_size(b))
    m.dsv4_paged_attn_weights(b, ws)
    assert m.dsv4_read_error_word(ws) == (m.DSV4_ERR_BAD_INDEX, m.DSV4_EWORD_BAD_INDEX)
    assert (acc[0, 48:64] == 0).all() and (acc[0, 192:] == 0).all()
    assert ((acc[0, seen].double() - p.sum(0)).abs() <= 1e-4 * p.sum(0)).all()
    for bad_cu, bad_len in (([0, 1, 3], lens), ([0, 1, 2], [200, 99999]), ([0, 1, 2], [-4, 90]), ([0, 2, 1], lens)):
        c.kv_len.copy_(i32(bad_len))
        a = m.paged_attn_args(q, out, c.k, c.table, i32(bad_cu), c.kv_len, lse=lse)
        ws = ws_for(m.dsv4_paged_attn_workspace_size(a))
        m.dsv4_paged_attn(a, ws)
        assert m.dsv4_read_error_word(ws)[1] == m.DSV4_EWORD_BAD_INDEX


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("H, KV, D, shared", SHAPES)
@pytest.mark.parametrize("kind", ["step", "chunk", "window"])
def test_weights(H, KV, D, shared, kind):
    m = lib()
    g = gen(H + D)
    lens = [1, 127, 128, 1000, 333, 0]
    ns = [1, 1, 1, 1, 1, 0] if kind == "step" else [1, 0, 130, 77, 333, 0]
    window = 50 if kind == "window" else 0
    first = [max(0, L - n + 1 - window) if window else 0 for n, L in zip(ns, lens)]
    c = Cache(g, lens, 16, KV, D, True, first=first)
    cu = cu_of(ns)
    q = normal(g, cu[-1], H, D, std=2.0)
    scale = 1 / math.sqrt(D)
    lse = ref.attention(q, c.k, None, c.table, cu, lens, scale, window)[1].float()
    acc_in = normal(g, len(lens), 1003, dtype=torch.float32).abs()
    for src in (None, acc_in, "self"):
        acc = acc_in.clone() if src == "self" else torch.full_like(acc_in, -3)
        a_in = acc if src == "self" else src
        a = m.paged_weights_args(q, lse, c.k, c.table, i32(cu), c.kv_len, acc, acc_in=a_in, max_q=max(ns), window=window)
        want, tol = ref.weights(q, lse, c.k, c.table, cu, lens, scale, acc, None if src is None else acc_in, window)
        ws = ws_for(m.dsv4_paged_attn_weights_workspace_size(a))
        m.dsv4_paged_attn_weights(a, ws)
        assert m.dsv4_read_error_word(ws) == (0, 0)
        err = (acc.double() - want).abs()
        assert (err <= tol).all(), (err / tol.clamp_min(1e-38)).max()


def test_weights_with_more_tokens_than_announced():
    """max_q chooses the tile and is not a limit: sequences with more tokens are answered alike."""
    m = lib()
    g = gen(21)
    lens, ns = [400, 300], [9, 2]
    c = Cache(g, lens, 16, 1, 512)
    q = normal(g, 11, 64, 512, std=2.0)
    lse = ref.attention(q, c.k, None, c.table, cu_of(ns), lens, 1 / math.sqrt(512))[1].float()
    out, l = attend(c, q, cu_of(ns), max_q=1)
    ref.check_attention(out, l, ref.attention(q, c.k, None, c.table, cu_of(ns), lens, 1 / math.sqrt(512)))
    acc = torch.zeros(2, 400, device="cuda")
    a = m.paged_weights_args(q, lse, c.k, c.table, i32(cu_of(ns)), c.kv_len, acc, max_q=1)
    m.dsv4_paged_attn_weights(a, ws_for(m.dsv4_paged_attn_weights_workspace_size(a)))
    want, tol = ref.weights(q, lse, c.k, c.table, cu_of(ns), lens, 1 / math.sqrt(512), torch.zeros_like(acc), None)
    assert ((acc.double() - want).abs() <= tol).all()


# ------------------------------------------------------------------ norm, rotation, append
@pytest.mark.parametrize("tokens", [1, 3, 700])
@pytest.mark.parametrize("H, KV, D, rope", [(64, 1, 512, 64), (5, 5, 128, 128), (32, 8, 256, 2), (0, 2, 128, 64), (7, 0, 256, 0)])
@pytest.mark.parametrize("v", [False, True])
def test_norm_rope_append(tokens, H, KV, D, rope, v):
    m = lib()
    g = gen(tokens + D)
    v = v and KV > 0
    x = normal(g, tokens, H + KV * (2 if v else 1) + 1, D, std=1.5)
    x[0] *= 1e-3                                     # (eps counts)
    q, k, vv = x[:, :H], x[:, H:H + KV], x[:, H + KV:H + 2 * KV]
    gq, gk = normal(g, D, dtype=torch.float32), normal(g, D, dtype=torch.float32)
    pos = torch.randint(0, 1 << 33, (tokens,), generator=g, device="cuda")
    pos[0] = 0
    n = tokens // 16 + 2
    pages = normal(g, n, 16, max(KV, 1), D)
    vpages = normal(g, n, 16, max(KV, 1), D)
    before, vbefore = pages.clone(), vpages.clone()
    slots = torch.randperm(n * 16, generator=g, device="cuda")[:tokens].contiguous()
    slots[2::5] = -1
    slots[3::50] = n * 16                            # past the pool: not stored
    out = torch.empty(tokens, H, D, dtype=BF, device="cuda")
    for gam in ((gq, gk), (None, None)):
        pages.copy_(before)
        vpages.copy_(vbefore)
        a = m.norm_rope_args(q if H else None, out if H else None, pos, k=k if KV else None, k_pages=pages if KV else None,
                             v=vv if v else None, v_pages=vpages if v else None, slots=slots if KV else None,
                             gamma_q=gam[0], gamma_k=gam[1], rope_dim=rope, eps=1e-6)
        m.dsv4_norm_rope_append(a)
        kept = (slots >= 0) & (slots < n * 16)
        pairs = [(out, q, gam[0])] if H else []
        if KV:
            pairs.append((pages.view(-1, KV, D)[slots[kept]], k, gam[1]))
            left = torch.ones(n * 16, dtype=torch.bool, device="cuda")
            left[slots[kept]] = False
            assert torch.equal(pages.view(-1, KV, D)[left], before.view(-1, KV, D)[left])
            if v:
                assert torch.equal(vpages.view(-1, KV, D)[slots[kept]], vv[kept])
                assert torch.equal(vpages.view(-1, KV, D)[left], vbefore.view(-1, KV, D)[left])
            else:
                assert torch.equal(vpages, vbefore)
        for got, src, gamma in pairs:
            want = ref.norm_rope(src, gamma, pos, rope, 1e4, 1e-6)
            if got is not out:
                want = want[kept]
            # one rounding to bf16, and a few fp32 steps of the pair's length (sum of squares, root, product, turn)
            size = want.abs()
            if rope:
                r = torch.hypot(want[..., -rope::2], want[..., -rope + 1::2]).repeat_interleave(2, -1)
                size = torch.cat([size[..., :D - rope], r], -1)
            tol = ref.BF16_STEP * want.abs() + (D / 8 + 16) * ref.F32_STEP * size + 1e-30
            assert ((got.double() - want).abs() <= tol).all()


def test_norm_rope_in_place():
    m = lib()
    g = gen(2)
    x = normal(g, 50, 9, 256)
    q = x[:, :8]
    pos = torch.arange(50, device="cuda")
    out = torch.empty(50, 8, 256, dtype=BF, device="cuda")
    m.dsv4_norm_rope_append(m.norm_rope_args(q, out, pos))
    keep = x[:, 8].clone()
    m.dsv4_norm_rope_append(m.norm_rope_args(q, q, pos))
    assert torch.equal(q, out) and torch.equal(x[:, 8], keep)


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("KV, D, shared, page", [(1, 512, True, 64), (3, 128, False, 16), (8, 256, False, 48), (5, 128, True, 8)])
@pytest.mark.parametrize("budget, recent", [(100, 20), (64, 64), (50, 0), (1, 0), (1, 1), (1500, 100)])
@pytest.mark.parametrize("place", ["in", "out", "acc"])
def test_evict(KV, D, shared, page, budget, recent, place):
    """In place, into other pages, and into other pages with the weights in place."""
    m = lib()
    g = gen(budget + recent + D)
    lens = [0, 1, budget, budget + 1, 1700, 333, max(1, budget - 1)]
    c = Cache(g, lens, page, KV, D, shared, spare=2 + len(lens) * (-(-budget // page)), poison=False)
    rows = 1801
    acc = normal(g, len(lens), rows, dtype=torch.float32).abs()
    acc = (acc * 4).round() / 4                      # ties, zeros
    kept = ref.evict(lens, acc, budget, recent)
    if place == "in":
        per = -(-max(budget, max(lens)) // page)
        table = torch.full((len(lens), per), 0, dtype=torch.int32, device="cuda")
        table[:, :c.table.shape[1]] = c.table
        c.table = table                              # (room for the budget; unused entries are not read)
        out_table, acc_out, len_out = table, acc, c.kv_len
    else:
        free = sorted(set(range(c.k.shape[0])) - set(c.table.flatten().tolist()))
        per = -(-budget // page)
        out_table = i32(free[:len(lens) * per]).view(len(lens), per)
        acc_out = acc if place == "acc" else torch.full_like(acc, -9)
        len_out = torch.full_like(c.kv_len, -9)
    old_acc, old_out = acc.clone(), acc_out.clone()
    want_k = c.k.clone()
    want_v = None if c.v is None else c.v.clone()
    for s, r in enumerate(kept):
        if not r:
            continue
        src = torch.tensor(r, device="cuda")
        dst = torch.arange(len(r), device="cuda")
        a, b = c.table[s].long()[src // page], out_table[s].long()[dst // page]
        want_k[b, dst % page] = c.k[a, src % page]
        if c.v is not None:
            want_v[b, dst % page] = c.v[a, src % page]
    keep = torch.full((len(lens), budget), -5, dtype=torch.int32, device="cuda")
    a = m.paged_evict_args(c.k, c.table, c.kv_len, acc, keep, budget=budget, recent=recent, v_pages=c.v, out_table=out_table,
                           kv_len_out=len_out, acc_out=acc_out)
    ws = ws_for(m.dsv4_paged_evict_workspace_size(a))
    m.dsv4_paged_evict(a, ws)
    assert m.dsv4_read_error_word(ws) == (0, 0)
    assert len_out.tolist() == [len(r) for r in kept]
    assert torch.equal(c.k, want_k) and (c.v is None or torch.equal(c.v, want_v))
    for s, r in enumerate(kept):
        assert keep[s].tolist() == r + [-1] * (budget - len(r))
        assert torch.equal(acc_out[s, :len(r)], old_acc[s, r])
        assert torch.equal(acc_out[s, len(r):], old_out[s, len(r):])


def test_evict_long_rows():
    """Rows long enough for the top-k over a cluster, in place, twice (the second cuts further)."""
    m = lib()
    g = gen(31)
    lens, page, D = [70000, 40000, 100], 64, 128
    c = Cache(g, lens, page, 1, D, poison=False)
    acc = (normal(g, 3, 70016, dtype=torch.float32).abs() * 64).round() / 64
    for budget, recent in ((33000, 128), (1000, 0)):
        now = c.kv_len.tolist()
        kept = ref.evict(now, acc.cpu(), budget, recent)
        flat = [c.k[c.table[s].long()[torch.tensor(r, device="cuda") // page], torch.tensor(r, device="cuda") % page] for s, r in enumerate(kept)]
        old = acc.clone()
        keep = torch.empty(3, budget, dtype=torch.int32, device="cuda")
        a = m.paged_evict_args(c.k, c.table, c.kv_len, acc, keep, budget=budget, recent=recent)
        ws = ws_for(m.dsv4_paged_evict_workspace_size(a))
        m.dsv4_paged_evict(a, ws)
        assert m.dsv4_read_error_word(ws) == (0, 0)
        assert c.kv_len.tolist() == [len(r) for r in kept]
        for s, r in enumerate(kept):
            assert keep[s, :len(r)].tolist() == r and (keep[s, len(r):] == -1).all()
            assert torch.equal(ref.rows_of(c.k, c.table, s, len(r)), flat[s])
            assert torch.equal(acc[s, :len(r)], old[s, r])


# ------------------------------------------------------------------ together
def test_a_serving_loop():
    """Prefill in chunks, then single tokens, with weights accumulated and the cache cut to a budget on the way: every
    step's attention equals the plain form over the rows that are then in the cache."""
    m = lib()
    g = gen(41)
    B, H, D, page, budget, recent = 3, 16, 128, 16, 200, 32
    pool = 80
    k = torch.full((pool, page, 1, D), float("nan"), dtype=BF, device="cuda")
    table = torch.randperm(pool, generator=g, device="cuda")[:B * 26].view(B, 26).to(torch.int32).contiguous()
    lens, seen = [0] * B, [0] * B
    acc = torch.zeros(B, 26 * page, device="cuda")
    keep = torch.empty(B, budget, dtype=torch.int32, device="cuda")
    kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    e = m.paged_evict_args(k, table, kv_len, acc, keep, budget=budget, recent=recent)
    we = ws_for(m.dsv4_paged_evict_workspace_size(e))
    for step in range(9):
        ns = [150, 7, 0] if step == 0 else [90, 140, 129] if step == 1 else [1, 1, 1]
        T = sum(ns)
        x = normal(g, T, H + 1, D, std=1.5)
        at = [(s, t) for s in range(B) for t in range(ns[s])]
        pos = torch.tensor([seen[s] + t for s, t in at], device="cuda")
        row = [lens[s] + t for s, t in at]
        slots = torch.tensor([int(table[s, r // page]) * page + r % page for (s, _), r in zip(at, row)], device="cuda")
        q = torch.empty(T, H, D, dtype=BF, device="cuda")
        m.dsv4_norm_rope_append(m.norm_rope_args(x[:, :H], q, pos, k=x[:, H:], k_pages=k, slots=slots))
        lens = [a + b for a, b in zip(lens, ns)]
        seen = [a + b for a, b in zip(seen, ns)]
        kv_len.copy_(i32(lens))
        cu = cu_of(ns)
        out, lse = torch.empty_like(q), torch.empty(T, H, device="cuda")
        a = m.paged_attn_args(q, out, k, table, i32(cu), kv_len, lse=lse, max_q=max(ns), out_rope_pos=pos)
        b = m.paged_weights_args(q, lse, k, table, i32(cu), kv_len, acc, acc_in=acc, max_q=max(ns))
        old = acc.clone()
        m.dsv4_paged_attn(a, ws_for(m.dsv4_paged_attn_workspace_size(a)))
        m.dsv4_paged_attn_weights(b, ws_for(m.dsv4_paged_attn_weights_workspace_size(b)))
        ref.check_attention(out, lse, ref.attention(q, k, None, table, cu, lens, 1 / math.sqrt(D), rope=64, pos=pos))
        want, tol = ref.weights(q, lse, k, table, cu, lens, 1 / math.sqrt(D), old, old)
        assert ((acc.double() - want).abs() <= tol).all()
        if step % 2:
            kept = ref.evict(lens, acc.cpu(), budget, recent)
            m.dsv4_paged_evict(e, we)
            lens = kv_len.tolist()
            assert lens == [len(r) for r in kept]
            assert all(keep[s, :len(r)].tolist() == r for s, r in enumerate(kept))
            for s in range(B):
                acc[s, lens[s]:] = 0                 # rows that the next tokens fill start without weight


# ------------------------------------------------------------------ empty calls, many sequences, bad pages
def test_calls_without_tokens_or_sequences():
    """No token: attention and append leave everything alone and the weights are acc_in; no sequence: nothing."""
    m = lib()
    g = gen(40)
    c = Cache(g, [70, 130], 16, 2, 128, False)
    q = torch.empty(0, 8, 128, dtype=BF, device="cuda")
    for table, cu, n in ((c.table, i32([0, 0, 0]), c.kv_len), (c.table[:0], i32([0]), c.kv_len[:0])):
        lse = torch.empty(0, 8, device="cuda")
        a = m.paged_attn_args(q, torch.empty_like(q), c.k, table, cu, n, v_pages=c.v, lse=lse)
        ws = ws_for(m.dsv4_paged_attn_workspace_size(a))
        m.dsv4_paged_attn(a, ws)
        assert m.dsv4_read_error_word(ws) == (0, 0)
        acc = torch.full((n.shape[0], 140), 7.0, device="cuda")
        acc_in = torch.arange(140, device="cuda", dtype=torch.float32).repeat(n.shape[0], 1)
        a = m.paged_weights_args(q, lse, c.k, table, cu, n, acc, acc_in=acc_in)
        ws = ws_for(m.dsv4_paged_attn_weights_workspace_size(a))
        m.dsv4_paged_attn_weights(a, ws)
        assert m.dsv4_read_error_word(ws) == (0, 0)
        for s, L in enumerate(c.lens[:n.shape[0]]):
            assert torch.equal(acc[s, :L], acc_in[s, :L]) and (acc[s, L:] == 7).all()
    before = c.k.clone()
    a = m.norm_rope_args(q, torch.empty_like(q), torch.empty(0, dtype=torch.int64, device="cuda"), k=q[:, :2], k_pages=c.k,
                         slots=torch.empty(0, dtype=torch.int64, device="cuda"))
    m.dsv4_norm_rope_append(a)
    torch.cuda.synchronize()
    assert torch.equal(before.view(torch.int16), c.k.view(torch.int16))


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("longest", [1, 5, 70])
def test_weights_of_many_sequences(window, longest):
    """More sequences than the block has warps, some without tokens or rows, some with more rows than acc."""
    m = lib()
    g = gen(41)
    r = torch.Generator().manual_seed(longest)
    B, rows = 300, 500
    lens = torch.randint(0, 700, (B,), generator=r).tolist()
    ns = [min(int(n), L) for n, L in zip(torch.randint(0, longest + 1, (B,), generator=r), lens)]
    c = Cache(g, lens, 8, 2, 128, True)
    cu = cu_of(ns)
    q = normal(g, cu[-1], 8, 128, std=2.0)
    scale = 1 / math.sqrt(128)
    lse = ref.attention(q, c.k, None, c.table, cu, lens, scale, window)[1].float()
    acc = torch.full((B, 700), -3.0, device="cuda")
    a = m.paged_weights_args(q, lse, c.k, c.table, i32(cu), c.kv_len, acc, max_q=longest, window=window)
    ws = ws_for(m.dsv4_paged_attn_weights_workspace_size(a))
    m.dsv4_paged_attn_weights(a, ws)
    assert m.dsv4_read_error_word(ws) == (0, 0)
    want, tol = ref.weights(q, lse, c.k, c.table, cu, lens, scale, torch.full_like(acc, -3.0), None, window)
    assert ((acc.double() - want).abs() <= tol).all()
    # an accumulator of fewer rows: the same, cut, and reported
    short = torch.full((B, rows), -3.0, device="cuda")
    a = m.paged_weights_args(q, lse, c.k, c.table, i32(cu), c.kv_len, short, max_q=longest, window=window)
    m.dsv4_paged_attn_weights(a, ws)
    assert m.dsv4_read_error_word(ws)[1] == m.DSV4_EWORD_BAD_INDEX
    assert ((short.double() - want[:, :rows]).abs() <= tol[:, :rows]).all()


def test_weights_hide_a_page_outside_the_pool():
    m = lib()
    g = gen(42)
    for ns in ([1, 1], [90, 200]):
        lens = [400, 300]
        c = Cache(g, lens, 16, 1, 256)
        cu = cu_of(ns)
        q = normal(g, cu[-1], 16, 256, std=2.0)
        lse = ref.attention(q, c.k, None, c.table, cu, lens, 1 / 16)[1].float()
        want, tol = ref.weights(q, lse, c.k, c.table, cu, lens, 1 / 16, torch.zeros(2, 400, device="cuda"), None)
        c.table[0, 3] = c.k.shape[0]                                 # rows 48 .. 63
        c.table[1, 10] = -1                                          # rows 160 .. 175
        want[0, 48:64] = 0
        want[1, 160:176] = 0
        acc = torch.zeros(2, 400, device="cuda")
        a = m.paged_weights_args(q, lse, c.k, c.table, i32(cu), c.kv_len, acc, max_q=max(ns))
        ws = ws_for(m.dsv4_paged_attn_weights_workspace_size(a))
        m.dsv4_paged_attn_weights(a, ws)
        assert m.dsv4_read_error_word(ws)[1] == m.DSV4_EWORD_BAD_INDEX
        assert ((acc.double() - want).abs() <= tol).all()


def test_tables_and_lengths_may_be_slices():
    """Lengths, tables and accumulators at addresses of their type's alignment only."""
    m = lib()
    g = gen(43)
    lens, ns = [333, 200, 45], [3, 1, 45]
    c = Cache(g, lens, 16, 1, 128)
    cu = cu_of(ns)

    def shifted(t):
        room = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        room[1:] = t.flatten()
        return room[1:].view(t.shape)

    q = normal(g, cu[-1], 8, 128, std=2.0)
    out = torch.empty_like(q)
    lse = shifted(torch.zeros(cu[-1], 8, device="cuda"))
    sink = shifted(normal(g, 8, dtype=torch.float32))
    table, cuq, n = shifted(c.table), shifted(i32(cu)), shifted(c.kv_len)
    a = m.paged_attn_args(q, out, c.k, table, cuq, n, lse=lse, sink=sink)
    ws = ws_for(m.dsv4_paged_attn_workspace_size(a))
    m.dsv4_paged_attn(a, ws)
    scale = 1 / math.sqrt(128)
    ref.check_attention(out, lse, ref.attention(q, c.k, None, c.table, cu, lens, scale, sink=sink))
    acc = shifted(torch.zeros(3, 333, device="cuda"))
    a = m.paged_weights_args(q, lse, c.k, table, cuq, n, acc)
    ws = ws_for(m.dsv4_paged_attn_weights_workspace_size(a))
    m.dsv4_paged_attn_weights(a, ws)
    want, tol = ref.weights(q, lse, c.k, c.table, cu, lens, scale, torch.zeros_like(acc), None)
    assert ((acc.double() - want).abs() <= tol).all()
    keep = shifted(torch.zeros(3, 50, dtype=torch.int32, device="cuda"))
    rows, old = c.k[c.table[0, :21].long()].flatten(0, 1).clone(), acc.clone()
    a = m.paged_evict_args(c.k, table, n, acc, keep, budget=50, recent=10)
    m.dsv4_paged_evict(a, ws_for(m.dsv4_paged_evict_workspace_size(a)))
    top = old[0, :323].topk(40).indices.sort().values
    assert torch.equal(keep[0].long(), torch.cat([top, torch.arange(323, 333, device="cuda")]))
    assert torch.equal(c.k[c.table[0, :4].long()].flatten(0, 1)[:50], rows[keep[0].long()])
    assert n.tolist() == [50, 50, 45]


# ------------------------------------------------------------------ values that are not finite
def _but(r, mask):
    """The reference's results of the queries in mask [T, H]."""
    return tuple(x[mask] for x in r)


@pytest.mark.parametrize("H, KV, D, shared", [(64, 1, 512, True), (8, 1, 128, True), (12, 2, 256, False), (32, 4, 128, False)])
@pytest.mark.parametrize("kind", ["split", "step", "chunk", "window"])
@pytest.mark.parametrize("with_sink", [False, True])
def test_a_nan_query_answers_nan(H, KV, D, shared, kind, with_sink):
    """Its output and lse are NaN, in one tile and over many CTAs, and so are the weights of the rows it sees; every other
    query's results are as without it."""
    m = lib()
    g = gen(H + D)
    lens = [20000, 300] if kind == "split" else [300, 77, 130, 1]
    ns = [1] * len(lens) if kind in ("split", "step") else [150, 2, 130, 1]
    window = 40 if kind == "window" else 0
    c = Cache(g, lens, 16, KV, D, shared)
    cu = cu_of(ns)
    q = normal(g, cu[-1], H, D, std=2.0)
    sink = normal(g, H, dtype=torch.float32) if with_sink else None
    scale = 1 / math.sqrt(D)
    r = ref.attention(q, c.k, c.v, c.table, cu, lens, scale, window, sink=sink)
    sick = torch.zeros(cu[-1], H, dtype=torch.bool, device="cuda")
    at = [(s, t, h) for s, t, h in ((0, 0, 3), (1, ns[1] - 1, H - 1), (0, ns[0] // 3, 0))]
    for s, t, h in at:
        sick[cu[s] + t, h] = True
        q[cu[s] + t, h, (7 * h + t) % D] = float("nan")
    out, lse = attend(c, q, cu, window=window, sink=sink, max_q=max(ns))
    ref.check_attention(out[~sick], lse[~sick], _but(r, ~sick))
    assert torch.isnan(out[sick].float()).all() and torch.isnan(lse[sick]).all()
    acc = torch.full((len(lens), max(lens)), -3.0, device="cuda")
    a = m.paged_weights_args(q, lse, c.k, c.table, i32(cu), c.kv_len, acc, max_q=max(ns), window=window)
    ws = ws_for(m.dsv4_paged_attn_weights_workspace_size(a))
    m.dsv4_paged_attn_weights(a, ws)
    assert m.dsv4_read_error_word(ws) == (0, 0)
    want = torch.full_like(acc, -3.0)
    for s, L in enumerate(lens):
        want[s, :L] = 0
    for s, t, h in at:
        lo, hi = ref.bounds(lens[s], ns[s], window)[t]
        want[s, lo:hi] = float("nan")
    assert torch.equal(torch.isnan(acc), torch.isnan(want))
    well = q.clone()
    well[sick] = 0                                   # (the weights of the others alone)
    weights, tol = ref.weights(well, torch.where(sick, 1e4, lse), c.k, c.table, cu, lens, scale, torch.full_like(acc, -3.0), None,
                               window)
    sound = ~torch.isnan(acc)
    assert ((acc.double() - weights).abs() <= tol)[sound].all()


@pytest.mark.parametrize("D, max_q", [(512, 1), (128, 1), (128, 100), (256, 100)])
@pytest.mark.parametrize("L", [300, 9000])
def test_scores_of_minus_infinity(D, max_q, L):
    """Scores that leave the range of fp32 downwards: rows that have them get no weight. A query with no other score has
    0/0 for an output and lse -inf; with a sink, output 0 and the sink's lse."""
    g = gen(D)
    c = Cache(g, [L, L], 16, 1, D, False)
    far = 256 if L == 300 else 8000
    row = torch.arange(L, device="cuda")
    for s in range(2):
        page, slot = c.table[s].long()[row // 16], row % 16
        c.k[page, slot, 0, 0] = torch.where(row < (far if s == 0 else L), -3e38, 0.0).to(BF)
    q = normal(g, 2, 8, D)
    q[..., 0] = 0
    tame = q.clone()
    q[:, ::2, 0] = 3e38                              # even heads: q . k past -3.4e38 where k's first channel is -3e38
    scale = 1 / math.sqrt(D)
    for sink in (None, normal(g, 8, dtype=torch.float32)):
        out, lse = attend(c, q, [0, 1, 2], sink=sink, max_q=max_q)
        # sequence 0, even heads: the rows from `far` on
        page, slot = c.table[0].long()[row[far:] // 16], row[far:] % 16
        k, v = c.k[page, slot, 0].double(), c.v[page, slot, 0].double()
        z = tame[0, ::2].double() @ k.t() * scale
        if sink is not None:
            z = torch.cat([z, sink[::2].double()[:, None]], 1)
        p = torch.softmax(z, 1)[:, :k.shape[0]]
        # (bf16 rounding of P and of the output; a score's fp32 sum has at most 32 steps, each off by 2^-23 of a partial
        # sum below 2^7, times the scale: below 2^-14, and 2^-12 with the exponentials and the sums)
        tol = ref.BF16_STEP * (p @ v).abs() + (ref.BF16_STEP + 2.0 ** -12) * (p @ v.abs())
        assert ((out[0, ::2].double() - p @ v).abs() <= tol).all()
        assert ((lse[0, ::2].double() - torch.logsumexp(z, 1)).abs() <= 2.0 ** -12).all()
        # sequence 1, even heads: nothing but -inf
        if sink is None:
            assert torch.isnan(out[1, ::2].float()).all() and (lse[1, ::2] == -math.inf).all()
        else:
            assert (out[1, ::2] == 0).all() and ((lse[1, ::2] - sink[::2]).abs() <= 2.0 ** -20 * (1 + sink[::2].abs())).all()
        assert torch.isfinite(out[:, 1::2].float()).all() and torch.isfinite(lse[:, 1::2]).all()


@pytest.mark.parametrize("D, max_q", [(512, 1), (128, 100)])
def test_the_lse_of_a_token_that_sees_nothing_is_its_sink(D, max_q):
    """Bit for bit, the type's lowest value included; such a sink adds nothing where rows are seen."""
    g = gen(D + 1)
    ns, lens = [9, 4, 3], [4, 0, 3]
    c = Cache(g, lens, 8, 1, D)
    cu = cu_of(ns)
    q = normal(g, cu[-1], 8, D)
    sink = normal(g, 8, dtype=torch.float32)
    sink[0], sink[1], sink[2] = torch.finfo(torch.float32).min, -3.0e38, -math.inf
    out, lse = attend(c, q, cu, sink=sink, max_q=max_q)
    blind = list(range(5)) + list(range(9, 13))
    assert torch.equal(lse[blind], sink.expand(len(blind), 8)) and (out[blind] == 0).all()
    seen = [t for t in range(cu[-1]) if t not in blind]
    r = ref.attention(q, c.k, None, c.table, cu, lens, 1 / math.sqrt(D), sink=sink)
    ref.check_attention(out[seen], lse[seen], tuple(x[seen] for x in r))


def test_sinks_of_a_sequence_without_a_page_over_many_ctas():
    """A long sequence none of whose pages lies in the pool, beside one that has rows: out 0, lse the sink, in the merge too."""
    m = lib()
    g = gen(77)
    lens, D, H = [30000, 200], 128, 8
    c = Cache(g, lens, 64, 1, D)
    c.table[0] = -1
    q = normal(g, 2, H, D)
    sink = normal(g, H, dtype=torch.float32)
    sink[1] = torch.finfo(torch.float32).min
    out, lse = torch.empty_like(q), torch.empty(2, H, device="cuda")
    a = m.paged_attn_args(q, out, c.k, c.table, i32([0, 1, 2]), c.kv_len, max_q=1, sink=sink, lse=lse)
    ws = ws_for(m.dsv4_paged_attn_workspace_size(a))
    m.dsv4_paged_attn(a, ws)
    assert m.dsv4_read_error_word(ws)[1] == m.DSV4_EWORD_BAD_INDEX
    assert (out[0] == 0).all() and torch.equal(lse[0], sink)
    one = ref.attention(q[1:], c.k, None, c.table[1:], [0, 1], lens[1:], 1 / math.sqrt(D), sink=sink)
    ref.check_attention(out[1:], lse[1:], one)


# ------------------------------------------------------------------ large pages, bad pages and lengths in the eviction
@pytest.mark.parametrize("page", [128, 256, 384, 2048])
@pytest.mark.parametrize("H, KV, D, shared", [(64, 1, 512, True), (32, 4, 128, False), (16, 1, 256, True)])
def test_pages_of_a_whole_unit_and_more(page, H, KV, D, shared):
    m = lib()
    g = gen(page + D)
    lens, ns, window = [1, 127, 128, 700, 5000, 260], [1, 1, 90, 1, 1, 130], 0
    scale = 1 / math.sqrt(D)
    for window in (0, 100):
        first = [max(0, L - n + 1 - window) if window else 0 for n, L in zip(ns, lens)]
        c = Cache(g, lens, page, KV, D, shared, first=first)
        cu = cu_of(ns)
        q = normal(g, cu[-1], H, D, std=2.0)
        out, lse = attend(c, q, cu, window=window, max_q=130)
        ref.check_attention(out, lse, ref.attention(q, c.k, c.v, c.table, cu, lens, scale, window))
        lse = ref.attention(q, c.k, None, c.table, cu, lens, scale, window)[1].float()
        acc = torch.full((len(lens), 5000), -3.0, device="cuda")
        a = m.paged_weights_args(q, lse, c.k, c.table, i32(cu), c.kv_len, acc, max_q=130, window=window)
        want, tol = ref.weights(q, lse, c.k, c.table, cu, lens, scale, acc, None, window)
        ws = ws_for(m.dsv4_paged_attn_weights_workspace_size(a))
        m.dsv4_paged_attn_weights(a, ws)
        assert m.dsv4_read_error_word(ws) == (0, 0)
        assert ((acc.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("page", [128, 384])
@pytest.mark.parametrize("n", [1, 70])
def test_a_large_page_outside_the_pool_is_hidden(page, n):
    """Whole units are hidden; a sequence with no other page answers as one that sees nothing."""
    m = lib()
    g = gen(page + n)
    lens, ns, D, H = [3 * page + 50, page], [n, n], 128, 8
    c = Cache(g, lens, page, 1, D)
    q = normal(g, 2 * n, H, D)
    c.table[0, 1] = c.k.shape[0]
    c.table[1, 0] = -5
    out, lse = torch.empty_like(q), torch.empty(2 * n, H, device="cuda")
    cu = cu_of(ns)
    a = m.paged_attn_args(q, out, c.k, c.table, i32(cu), c.kv_len, lse=lse, max_q=n)
    ws = ws_for(m.dsv4_paged_attn_workspace_size(a))
    m.dsv4_paged_attn(a, ws)
    assert m.dsv4_read_error_word(ws) == (m.DSV4_ERR_BAD_INDEX, m.DSV4_EWORD_BAD_INDEX)
    assert (out[n:] == 0).all() and (lse[n:] == -math.inf).all()
    seen = torch.tensor([j for j in range(lens[0]) if j // page != 1], device="cuda")
    k = c.k[c.table[0].long()[seen // page], seen % page, 0].double()
    weight = torch.zeros(lens[0], dtype=torch.float64, device="cuda")
    for t in range(n):
        z = q[t].double() @ k.t() / math.sqrt(D)
        z[:, seen > lens[0] - n + t] = -math.inf
        p = torch.softmax(z, 1)
        weight[seen] += p.sum(0)
        tol = ref.BF16_STEP * (p @ k).abs() + (ref.BF16_STEP + 2.0 ** -12) * (p @ k.abs())
        assert ((out[t].double() - p @ k).abs() <= tol).all()
    acc = torch.zeros(2, lens[0], device="cuda")
    b = m.paged_weights_args(q, lse, c.k, c.table, i32(cu), c.kv_len, acc, max_q=n)
    ws = ws_for(m.dsv4_paged_attn_weights_workspace_size(b))
    m.dsv4_paged_attn_weights(b, ws)
    assert m.dsv4_read_error_word(ws)[1] == m.DSV4_EWORD_BAD_INDEX
    assert (acc[1] == 0).all() and (acc[0, page:2 * page] == 0).all()
    assert ((acc[0].double() - weight).abs() <= 2.0 ** -12 * weight).all()


@pytest.mark.parametrize("page", [16, 128, 384])
@pytest.mark.parametrize("place", ["in", "out"])
def test_evict_with_large_pages_and_bad_pages_and_lengths(page, place):
    """A row whose old or new page lies outside the pool does not move, everything else does; lengths are clamped to the
    rows that tables and acc hold; each is reported, and no other row of the pool changes."""
    m = lib()
    g = gen(page)
    D, budget, recent, rows = 128, 150, 30, 900
    lens = [700, 900, 40, 500]
    c = Cache(g, lens, page, 2, D, False, spare=2 + 4 * (-(-budget // page)), poison=False)
    per = -(-budget // page)
    free = sorted(set(range(c.k.shape[0])) - set(c.table.flatten().tolist()))
    if place == "in":
        wide = torch.zeros(4, max(c.table.shape[1], per), dtype=torch.int32, device="cuda")
        wide[:, :c.table.shape[1]] = c.table
        out_table = c.table = wide
    else:
        out_table = i32(free[:4 * per]).view(4, per)
    acc = (normal(g, 4, rows, dtype=torch.float32).abs() * 64).round() / 64
    full = c.table.shape[1] * page
    for bad in ("none", "page in", "page out", "lengths", "acc rows"):
        k, v, table, to = c.k.clone(), c.v.clone(), c.table.clone(), out_table.clone()
        if place == "in":
            to = table
        n, weight = c.kv_len.clone(), acc.clone()
        if bad == "page in":
            table[0, -(-700 // page) - 1] = k.shape[0]   # (of the recent rows, which are kept)
        if bad == "page out" and place == "out":
            to[1, 0] = -1
        if bad == "lengths":
            n.copy_(i32([-3, 1 << 30, 40, 500]))
        if bad == "acc rows":
            weight = acc[:, :450].contiguous()
        cap = min(full, weight.shape[1])
        now = [min(max(x, 0), cap) for x in n.tolist()]
        kept = ref.evict(now, weight.cpu(), budget, recent)
        pool, tab, dest = k.shape[0], table.tolist(), to.tolist()
        want_k, want_v = k.clone(), v.clone()
        broken = False
        for s, r in enumerate(kept):
            for i, j in enumerate(r):
                a, b = tab[s][j // page], dest[s][i // page]
                if place == "in" and i == j:
                    continue
                if not (0 <= a < pool and 0 <= b < pool):
                    broken = True
                    continue
                want_k[b, i % page] = k[a, j % page]
                want_v[b, i % page] = v[a, j % page]
        keep = torch.full((4, budget), -5, dtype=torch.int32, device="cuda")
        len_out = torch.full((4,), -9, dtype=torch.int32, device="cuda")
        got = torch.full_like(weight, -9.0)
        a = m.paged_evict_args(k, table, n, weight, keep, budget=budget, recent=recent, v_pages=v, out_table=to, kv_len_out=len_out,
                               acc_out=got)
        ws = ws_for(m.dsv4_paged_evict_workspace_size(a))
        m.dsv4_paged_evict(a, ws)
        flagged = broken or now != n.tolist()
        assert flagged == (bad != "none" and not (bad == "page out" and place == "in"))
        assert m.dsv4_read_error_word(ws)[1] == (m.DSV4_EWORD_BAD_INDEX if flagged else 0), bad
        assert len_out.tolist() == [len(r) for r in kept]
        assert torch.equal(k, want_k) and torch.equal(v, want_v), bad
        for s, r in enumerate(kept):
            assert keep[s].tolist() == r + [-1] * (budget - len(r))
            assert torch.equal(got[s, :len(r)], weight[s, r]) and (got[s, len(r):] == -9).all()


@pytest.mark.parametrize("longest", [700, 40000])
def test_a_graph_of_a_whole_step(longest):
    """Append, attention, weights and eviction in place, captured as one graph: each replay gives the bits of the eager step."""
    m = lib()
    g = gen(longest)
    B, H, D, page, budget = 3, 8, 128, 64, 500
    lens = [longest, longest // 2, 90]
    c = Cache(g, lens, page, 1, D, poison=False)
    x = normal(g, B, H + 1, D, std=1.5)
    pos = i32(lens).long()
    slots = torch.stack([c.table[s, (n - 1) // page].long() * page + (n - 1) % page for s, n in enumerate(lens)])
    cu = i32([0, 1, 2, 3])
    q, out = torch.empty(B, H, D, dtype=BF, device="cuda"), torch.empty(B, H, D, dtype=BF, device="cuda")
    lse = torch.empty(B, H, device="cuda")
    acc = (torch.rand(B, c.table.shape[1] * page, generator=g, device="cuda") * 64).round() / 64
    keep = torch.empty(B, budget, dtype=torch.int32, device="cuda")
    state = [c.k, c.kv_len, acc]
    start = [t.clone() for t in state]
    n = m.norm_rope_args(x[:, :H], q, pos, k=x[:, H:], k_pages=c.k, slots=slots)
    a = m.paged_attn_args(q, out, c.k, c.table, cu, c.kv_len, max_q=1, lse=lse, out_rope_pos=pos)
    w = m.paged_weights_args(q, lse, c.k, c.table, cu, c.kv_len, acc, acc_in=acc, max_q=1)
    e = m.paged_evict_args(c.k, c.table, c.kv_len, acc, keep, budget=budget, recent=64)
    sizes = (m.dsv4_paged_attn_workspace_size(a), m.dsv4_paged_attn_weights_workspace_size(w), m.dsv4_paged_evict_workspace_size(e))
    spaces = [ws_for(s) for s in sizes]

    def step():
        m.dsv4_norm_rope_append(n)
        m.dsv4_paged_attn(a, spaces[0])
        m.dsv4_paged_attn_weights(w, spaces[1])
        m.dsv4_paged_evict(e, spaces[2])

    def results():
        assert all(m.dsv4_read_error_word(s) == (0, 0) for s in spaces)
        return [t.clone() for t in (q, out, lse, keep, *state)]

    step()
    want = results()
    assert want[5].tolist() == [min(x, budget) for x in lens]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t, s in zip(state, start):
            t.copy_(s)
        keep.fill_(-5)
        for s in spaces:
            s.fill_(0x5A)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(results(), want))
