"""Attention behind shared prefixes on the GPU against the plain 64-bit form over each sequence's own table, at the group
sizes, lengths, layouts and masks where it can go wrong. Tolerances: paged_reference.py."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(ns):
    out = [0]
    for n in ns:
        out.append(out[-1] + n)
    return out


class Cache:
    """Sequences of `lens` rows; those of group g (start[g] .. start[g + 1] - 1) have the first pre[g] rows in common: whole
    pages are the same ones (or, with copies, pages of the same contents), the rest is copied. What no one sees holds NaN,
    table entries past the rows name no page."""

    def __init__(self, g, lens, start, pre, page, kv, dim, shared=True, copies=False, poison=True):
        self.lens, self.page, self.start, self.pre = lens, page, start, pre
        per = max(1, max(-(-n // page) for n in lens))
        pool = sum(-(-n // page) for n in lens) + 3
        self.k = normal(g, pool, page, kv, dim)
        self.v = None if shared else normal(g, pool, page, kv, dim)
        order = torch.randperm(pool, generator=g, device="cuda").tolist()
        table = [[(1 << 30) if i % 2 else -7 for i in range(per)] for _ in lens]
        used = torch.zeros(pool, page, dtype=torch.bool, device="cuda")
        for s, n in enumerate(lens):
            grp = [i for i in range(len(pre)) if start[i] <= s < start[i + 1]]
            first, common = (start[grp[0]], min(pre[grp[0]], n, lens[start[grp[0]]])) if grp else (s, 0)
            for i in range(-(-n // page)):
                whole = (i + 1) * page <= common and s != first
                table[s][i] = table[first][i] if whole and not copies else order.pop()
                if s != first and not (whole and not copies):
                    c = min(max(common - i * page, 0), page)
                    for p in (self.k, self.v):
                        if p is not None and c:
                            p[table[s][i], :c] = p[table[first][i], :c]
            j = torch.arange(n, device="cuda")
            used[torch.tensor(table[s], device="cuda")[j // page], j % page] = True
        if poison:
            for p in (self.k, self.v):
                if p is not None:
                    p[~used] = float("nan")
        self.table, self.kv_len = i32(table), i32(lens)


def args_of(c, q, cu, out, lse, *, sink=None, pos=None, rope=64, scale=None, start="own", pre=None):
    start = c.start if start == "own" else start
    return lib().paged_prefix_args(q, out, c.k, c.table, i32(cu), c.kv_len, i32(c.pre if pre is None else pre),
                                   group_start=None if start is None else i32(start), v_pages=c.v, sink=sink, lse=lse, scale=scale,
                                   out_rope_pos=pos, out_rope_dim=rope)


def workspace(a):
    return torch.full((lib().dsv4_paged_prefix_attn_workspace_size(a),), 0xFF, dtype=torch.uint8, device="cuda")


def attend(c, q, cu, *, err=0, **kw):
    m = lib()
    T, H, D = q.shape
    out = torch.full((T, H, D), 7.0, dtype=BF, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    a = args_of(c, q, cu, out, lse, **kw)
    ws = workspace(a)
    m.dsv4_paged_prefix_attn(a, ws)
    assert m.dsv4_read_error_word(ws)[1] == err
    again = torch.full_like(out, 3.0)
    a = args_of(c, q, cu, again, None, **kw)
    m.dsv4_paged_prefix_attn(a, ws)
    n = cu[-1]
    assert torch.equal(again[:n].view(torch.int16), out[:n].view(torch.int16)) and (again[n:] == 3).all()
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    return out[:n], lse[:n]


def check(c, q, cu, out, lse, *, sink=None, pos=None, rope=64, scale=None):
    n = cu[-1]
    ref.check_attention(out, lse, ref.attention(q[:n], c.k, c.v, c.table, cu, c.lens, 1 / math.sqrt(q.shape[2]) if scale is None else scale,
                                                sink=sink, rope=rope if pos is not None else 0, pos=None if pos is None else pos[:n]))


# (query heads, KV heads, channels, K = V)
SHAPES = [(8, 1, 128, True), (32, 8, 128, False), (16, 1, 512, True), (64, 1, 512, True), (12, 2, 256, False), (16, 2, 256, True),
          (5, 5, 128, False), (1, 1, 512, True), (200, 1, 128, True), (24, 3, 512, False), (160, 1, 256, True), (10, 2, 128, True)]


@pytest.mark.parametrize("H, KV, D, shared", SHAPES)
@pytest.mark.parametrize("page", [8, 48, 64, 256])
def test_single_tokens(H, KV, D, shared, page):
    g = gen(H + D + page)
    pre = [300, 128, 1]
    lens = [301, 310, 450, 301, 700, 129, 257, 130, 2, 9]
    c = Cache(g, lens, [0, 5, 8, 10], pre, page, KV, D, shared)
    q = normal(g, len(lens) + 2, H, D, std=2.0)
    sink = normal(g, H, dtype=torch.float32)
    cu = cu_of([1] * len(lens))
    out, lse = attend(c, q, cu, sink=sink)
    check(c, q, cu, out, lse, sink=sink)


@pytest.mark.parametrize("H, KV, D, shared", SHAPES)
@pytest.mark.parametrize("pre", [0, 5, 127, 129, 260])
def test_chunks(H, KV, D, shared, pre):
    """Ragged chunks behind one prefix, some without tokens, one longer than two tiles of queries."""
    g = gen(H + D + pre)
    ns = [5, 0, 1, 70, 33, 0, 1]
    lens = [pre + 5, pre + 40, pre + 1, pre + 70, pre + 140, pre, pre + 333]
    c = Cache(g, lens, [0, 7], [pre], 16, KV, D, shared)
    cu = cu_of(ns)
    q = normal(g, cu[-1] + 1, H, D, std=2.0)
    out, lse = attend(c, q, cu, start=None)
    check(c, q, cu, out, lse)


@pytest.mark.parametrize("D, shared", [(128, False), (256, True), (512, True)])
def test_groups_of_every_kind(D, shared):
    """Groups without sequences, without tokens, of one sequence, whose first sequence has no token, sequences outside every
    group, and prefixes of no row."""
    g = gen(D)
    lens = [50, 300, 300, 20, 200, 210, 220, 90, 95, 64, 64]
    ns = [1, 1, 3, 2, 0, 4, 1, 0, 0, 1, 1]
    start, pre = [1, 1, 3, 4, 7, 9, 10], [40, 250, 9, 130, 60, 0]
    c = Cache(g, lens, start, pre, 16, 2, D, shared)
    cu = cu_of(ns)
    q = normal(g, cu[-1], 8, D, std=2.0)
    out, lse = attend(c, q, cu)
    check(c, q, cu, out, lse)


@pytest.mark.parametrize("D", [128, 256, 512])
def test_prefixes_end_before_tokens_inside_them(D):
    """A chunk that begins inside the prefix (or before the cache: tokens that see nothing) cuts it for its group."""
    g = gen(D + 1)
    lens = [300, 290, 400, 150, 160, 4, 160]
    ns = [1, 45, 1, 1, 1, 9, 1]
    c = Cache(g, lens, [0, 3, 7], [280, 150], 8, 1, D, copies=True)
    cu = cu_of(ns)
    q = normal(g, cu[-1], 16, D, std=2.0)
    for sink in (None, normal(g, 16, dtype=torch.float32)):
        out, lse = attend(c, q, cu, sink=sink)
        r = ref.attention(q, c.k, None, c.table, cu, lens, D ** -0.5, sink=sink)
        if sink is not None:
            for t in range(cu[5], cu[5] + 5):
                r[1][t] = sink.double()
        ref.check_attention(out, lse, r)
        assert (out[cu[5]:cu[5] + 5] == 0).all()


@pytest.mark.parametrize("H, KV, D, shared", [(64, 1, 512, True), (32, 8, 128, False), (8, 1, 128, True), (16, 2, 256, True)])
def test_long_prefixes_are_split_and_merged(H, KV, D, shared):
    g = gen(7)
    lens = [20000 + n for n in (1, 700, 128, 5)]
    c = Cache(g, lens, [0, 4], [20000], 64, KV, D, shared)
    q = normal(g, 4, H, D, std=2.0)
    q[0, :2] *= 8
    q[1, :2] = 0
    pos = torch.tensor([5, 1 << 40, 123456, -3], device="cuda")
    sink = normal(g, H, dtype=torch.float32)
    cu = cu_of([1] * 4)
    out, lse = attend(c, q, cu, sink=sink, pos=pos)
    check(c, q, cu, out, lse, sink=sink, pos=pos)


@pytest.mark.parametrize("rope", [2, 64, 128])
@pytest.mark.parametrize("D", [128, 256, 512])
def test_output_rotation(rope, D):
    g = gen(rope)
    c = Cache(g, [400, 420, 390], [0, 3], [380], 32, 1, D)
    cu = cu_of([3, 20, 1])
    q = normal(g, cu[-1], 6, D, std=2.0)
    pos = torch.randint(0, 1 << 20, (cu[-1],), generator=g, device="cuda")
    out, lse = attend(c, q, cu, pos=pos, rope=rope)
    check(c, q, cu, out, lse, pos=pos, rope=rope)


@pytest.mark.parametrize("D, H, batch", [(512, 64, 2), (128, 8, 40), (256, 16, 12), (128, 8, 3)])
def test_scores_that_grow_along_the_cache(D, H, batch):
    """Each unit outruns the reference maximum of the one before: the running output is rescaled every time."""
    g = gen(11)
    lens = [1500 + s for s in range(batch)]
    c = Cache(g, lens, [0, batch], [1400], 64, 1, D, poison=False)
    for s in range(batch):
        j = torch.arange(lens[s], device="cuda")
        if s == 0 or batch == 3:
            page = c.table[s].long()[j // 64]
            c.k[page, j % 64, 0] = (c.k[page, j % 64, 0].float() * 0.1 + (j / 100)[:, None]).to(BF)
    for s in range(1, batch):                                         # the prefix's last rows are copies
        for i in range(1400 // 64, -(-lens[s] // 64)):
            n = min(max(1400 - i * 64, 0), 64)
            c.k[c.table[s, i].long(), :n] = c.k[c.table[0, i].long(), :n]
    q = (normal(g, batch, H, D).float() * 0.1 + 1).to(BF)
    q[:, H // 2:] *= -1
    cu = cu_of([1] * batch)
    out, lse = attend(c, q, cu)
    check(c, q, cu, out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_scales_and_strides(scale):
    g = gen(5)
    c = Cache(g, [300, 317], [0, 2], [290], 16, 2, 128, False)
    x = normal(g, 9, 14, 128)
    q = x[:, 3:11]
    cu = [0, 2, 9]
    out, lse = attend(c, q, cu, scale=scale)
    check(c, q, cu, out, lse, scale=scale)


@pytest.mark.parametrize("D, batch", [(128, 2), (128, 40), (256, 3), (512, 3)])
def test_a_nan_query_and_scores_of_minus_infinity(D, batch):
    g = gen(D)
    lens = [200 + s for s in range(batch)]
    c = Cache(g, lens, [0, batch], [190], 16, 1, D)
    q = normal(g, batch, 8, D, std=2.0)
    q[1, 3, 5] = float("nan")
    cu = cu_of([1] * batch)
    clean = q.clone()
    clean[1, 3, 5] = 0
    out, lse = attend(c, q, cu)
    want, wl = attend(c, clean, cu)
    assert torch.isnan(out[1, 3].float()).all() and torch.isnan(lse[1, 3])
    out[1, 3], lse[1, 3], want[1, 3], wl[1, 3] = 0, 0, 0, 0
    assert torch.equal(out, want) and torch.equal(lse, wl)
    # the first rows at -inf weigh nothing beside the others
    c.k[c.table[0, 0].long(), :, 0] = -1e38
    q = normal(g, batch, 8, D).abs() + 0.5                            # their scores overflow to -inf
    out, lse = attend(c, q, cu)
    ref.check_attention(out, lse, ref.attention(q, c.k, None, c.table, cu, lens, D ** -0.5)[:3] +
                        (ref.attention(q, c.k.clamp(min=-100), None, c.table, cu, lens, D ** -0.5)[3],))


@pytest.mark.parametrize("D", [128, 512])
def test_pages_outside_the_pool_are_hidden(D):
    g = gen(D)
    lens, page = [300, 310, 333], 16
    c = Cache(g, lens, [0, 3], [256], page, 1, D)
    q = normal(g, 3, 8, D, std=2.0)
    cu = [0, 1, 2, 3]
    c.table[0, 3] = -2                                                # of the prefix, as the group reads it
    c.table[2, 17] = 1 << 20                                          # of one sequence's own rows
    out, lse = attend(c, q, cu, err=1)
    for s in range(3):
        rows = [j for j in range(lens[s]) if not (48 <= j < 64 or (s == 2 and 272 <= j < 288))]
        t = c.table[s if s else 1].tolist() if s else c.table[1].tolist()[:16] + c.table[0].tolist()[16:]
        at = torch.tensor([t[j // page] * page + j % page for j in rows], device="cuda")
        k = c.k.flatten(0, 1)[at, 0][:, None]
        one = ref.attention(q[s:s + 1], k[None], None, i32([[0]]), [0, 1], [len(rows)], D ** -0.5)
        ref.check_attention(out[s:s + 1], lse[s:s + 1], one)


def test_counts_out_of_range_are_clamped_and_flagged():
    g = gen(2)
    c = Cache(g, [100, 120], [0, 2], [90], 16, 1, 128)
    q = normal(g, 2, 8, 128, std=2.0)
    cu = [0, 1, 2]
    for pre, start, flagged in (([-5], [0, 2], 1), ([1 << 30], [0, 2], 1), ([90], [0, 5], 1), ([90], [-3, 2], 1), ([90], [2, 0], 1), ([99], [0, 2], 0)):
        if pre == [1 << 30] or pre == [99]:
            c2 = Cache(gen(3), [100, 120], [0, 2], [99], 16, 1, 128)   # a prefix up to the first's own row
        else:
            c2 = c
        out, lse = attend(c2, q, cu, err=flagged, pre=pre, start=start)
        check(c2, q, cu, out, lse)


@pytest.mark.parametrize("D", [128, 256, 512])
def test_graphs_share_a_workspace(D):
    """Two captured graphs on one workspace, replayed in turn while lengths and prefixes change on the device."""
    m = lib()
    g = gen(D)
    lens = [500, 520, 600]
    c = Cache(g, lens, [0, 3], [480], 16, 1, D)
    q = [normal(g, 3, 8, D, std=2.0), normal(g, 3, 16, D, std=2.0)]
    out = [torch.zeros_like(x) for x in q]
    lse = [torch.zeros(3, x.shape[1], device="cuda") for x in q]
    cu = cu_of([1] * 3)
    calls = [args_of(c, x, cu, o, l) for x, o, l in zip(q, out, lse)]
    pre = [a.tensors[6] for a in calls]
    ws = max((workspace(a) for a in calls), key=lambda w: w.numel())
    for a in calls:
        m.dsv4_paged_prefix_attn(a, ws)
    graphs = []
    for a in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.dsv4_paged_prefix_attn(a, ws)
        graphs.append(graph)
    for P, cut in ((480, 0), (128, 7), (0, 15), (400, 19)):
        c.lens = [n - cut for n in lens]
        c.kv_len.copy_(i32(c.lens))
        for x in pre:
            x.fill_(P)
        for graph in graphs:
            graph.replay()
        for x, o, l in zip(q, out, lse):
            check(c, x, cu, o, l)
        assert m.dsv4_read_error_word(ws) == (0, 0)


def test_streams_and_empty_calls():
    m = lib()
    g = gen(4)
    c = Cache(g, [200, 210], [0, 2], [190], 16, 1, 128)
    q = normal(g, 2, 8, 128, std=2.0)
    out, lse = torch.zeros_like(q), torch.zeros(2, 8, device="cuda")
    a = args_of(c, q, [0, 1, 2], out, lse)
    ws = workspace(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.dsv4_paged_prefix_attn(a, ws, stream=s)
    s.synchronize()
    check(c, q, [0, 1, 2], out, lse)
    empty = torch.empty(0, 8, 128, dtype=BF, device="cuda")
    a = m.paged_prefix_args(empty, empty, c.k, c.table, i32([0, 0, 0]), c.kv_len, i32([190]))
    m.dsv4_paged_prefix_attn(a, ws)
    assert m.dsv4_read_error_word(ws) == (0, 0)
    out.fill_(7)
    a = args_of(c, q, [0, 0, 0], out, None)                           # tokens, but none of a sequence
    m.dsv4_paged_prefix_attn(a, ws)
    assert m.dsv4_read_error_word(ws) == (0, 0) and (out == 7).all()


@pytest.mark.parametrize("H, KV, D, batch", [(32, 8, 128, 130), (16, 1, 512, 40), (16, 2, 256, 70)])
def test_many_sequences_equal_the_unshared_call(H, KV, D, batch):
    """Against dsv4_paged_attn on the same tables, whose own tolerance is the same."""
    m = lib()
    g = gen(D)
    pre, page = 1000, 16
    lens = [pre + 1 + (s * 37) % 300 for s in range(batch)]
    c = Cache(g, lens, [0, batch // 3, batch], [pre, pre - 77], page, KV, D, D != 128)
    q = normal(g, batch, H, D, std=2.0)
    cu = cu_of([1] * batch)
    out, lse = attend(c, q, cu)
    want, wl = torch.empty_like(q), torch.empty(batch, H, device="cuda")
    a = m.paged_attn_args(q, want, c.k, c.table, i32(cu), c.kv_len, v_pages=c.v, lse=wl, max_q=1)
    ws = torch.empty(m.dsv4_paged_attn_workspace_size(a), dtype=torch.uint8, device="cuda")
    m.dsv4_paged_attn(a, ws)
    # both within (2^-8 of |out| + (2^-8 + 2^-9) of sum p |v|) of the exact values: sum p |v| is at most max |v| (below 6 here)
    assert ((out.float() - want.float()).abs() <= 2 * (2.0 ** -8 * want.float().abs() + 1.5 * 2.0 ** -8 * 6)).all()
    assert ((lse - wl).abs() <= 2.0 ** -12).all()
    some = [0, batch // 2, batch - 1]
    for s in some:
        one = ref.attention(q[s:s + 1], c.k, c.v, c.table[s:s + 1], [0, 1], [lens[s]], D ** -0.5)
        ref.check_attention(out[s:s + 1], lse[s:s + 1], one)


@pytest.mark.parametrize("D", [128, 512])
def test_a_wait_that_runs_out_is_reported(D):
    """With the first query copy left unissued the call ends, reports the time-out, and the next call is right."""
    m = lib()
    g = gen(1)
    c = Cache(g, [900, 910], [0, 2], [890], 16, 1, D)
    q = normal(g, 2, 8, D, std=2.0)
    out, lse = torch.zeros_like(q), torch.zeros(2, 8, device="cuda")
    a = args_of(c, q, [0, 1, 2], out, lse)
    ws = workspace(a)
    try:
        m.dsv4_test_wait_fault(m.DSV4_WAIT_FAULT_PAGED_PREFIX, 1000)
        m.dsv4_paged_prefix_attn(a, ws)
        st, word = m.dsv4_read_error_word(ws)
        assert st == m.DSV4_ERR_TIMEOUT and word & m.DSV4_EWORD_TIMEOUT
    finally:
        m.dsv4_test_wait_fault(m.DSV4_WAIT_FAULT_NONE, 0)
    m.dsv4_paged_prefix_attn(a, ws)
    assert m.dsv4_read_error_word(ws) == (0, 0)
    check(c, q, [0, 1, 2], out, lse)
