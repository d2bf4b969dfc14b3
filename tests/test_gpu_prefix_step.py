"""Serving steps behind a shared prefix in one graph (plan, rotation with append, attention), and a line of very many short
segments."""
from __future__ import annotations

import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import paged_reference as ref  # noqa: E402
from test_gpu_prefix import Cache, attend, cu_of, gen, i32, lib, normal  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_sparse_attention_08_gb300 import _build
    _build.build()


@pytest.mark.parametrize("H, KV, D, shared", [(8, 2, 128, False), (16, 1, 512, True)])
def test_steps_behind_a_prefix_in_one_graph(H, KV, D, shared):
    """Three sequences share 40 rows (two whole pages, and 8 rows that each has in a page of its own), a fourth has a
    prefix to itself. The first one ends and its own pages go back, so the others' prefix is then the two whole pages, still
    read through its table; it comes back as a request that shares them, its first token inside the prefix as it is given then."""
    m = lib()
    g = gen(D)
    B, page, width, pool, T, pre = 4, 16, 10, 40, 20, 40
    r = random.Random(5)
    ids = list(range(pool))
    r.shuffle(ids)
    kp = normal(g, pool, page, KV, D)
    vp = None if shared else normal(g, pool, page, KV, D)
    kv, keep = [45, 40, 58, 33], [2, 2, 2, 0]
    held = [-(-n // page) for n in kv]
    rows = []
    for s in range(B):
        rows.append([rows[0][j] if 0 < s < 3 and j < 2 else ids.pop() if j < held[s] else -1 for j in range(width)])
        if 0 < s < 3:
            for p in (kp, vp):
                if p is not None:
                    p[rows[s][2], :pre - 32] = p[rows[0][2], :pre - 32]
    table, free, count = i32(rows), i32(ids + [-1] * (pool - len(ids))), i32([len(ids)])
    kvt, heldt, keept, new, cu = i32(kv), i32(held), i32(keep), i32([0] * B), i32([0] * (B + 1))
    slots, pos = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    x = normal(g, T, H + 2 * KV, D)
    q, out = normal(g, T, H, D), normal(g, T, H, D)
    lse = torch.empty(T, H, device="cuda")
    plen = i32([pre, 20])
    plan = m.paged_plan_args(new, kvt, heldt, table, free, count, cu, slots, page_size=page, num_pages=pool, pos=pos, shared=keept)
    rot = m.rope_args(x[:, :H], q, pos, k=x[:, H:H + KV], k_out=kp, v=None if shared else x[:, H + KV:], v_out=vp, slots=slots,
                      rope_dim=64)
    att = m.paged_prefix_args(q, out, kp, table, cu, kvt, plen, group_start=i32([0, 3, 4]), v_pages=vp, lse=lse)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (m.dsv4_paged_plan_workspace_size(plan),
                                                                    m.dsv4_paged_prefix_attn_workspace_size(att))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.dsv4_paged_plan(plan, ws[0])
        m.dsv4_rope(rot)
        m.dsv4_paged_prefix_attn(att, ws[1])
    for ns, first, p in (([1, 9, 1, 2], 45, 40), ([1, 1, 1, 1], 46, 40), ([0, 1, 4, 1], 0, 32), ([3, 1, 0, 1], 32, 40),
                         ([1, 1, 1, 16], 35, 32)):
        kvt[0], plen[0] = first, p
        new.copy_(i32(ns))
        x.normal_(generator=g)
        out.fill_(7.0)
        lens, free_before, held_before = [a + b for a, b in zip(kvt.tolist(), ns)], int(count), heldt.tolist()
        graph.replay()
        assert m.dsv4_read_error_word(ws[0]) == (0, 0) and m.dsv4_read_error_word(ws[1]) == (0, 0)
        want = [max(-(-n // page), min(k, h)) for n, k, h in zip(lens, keep, held_before)]
        assert kvt.tolist() == lens and heldt.tolist() == want and cu.tolist() == cu_of(ns)
        assert int(count) == free_before + sum(held_before) - sum(want)
        n, c = sum(ns), cu_of(ns)
        for s in range(B):
            j = torch.arange(lens[s] - ns[s], lens[s], device="cuda")
            at = table[s].long()[j // page]
            assert torch.equal(kp[at, j % page][..., :D - 64], x[c[s]:c[s + 1], H:H + KV, :D - 64])
            if vp is not None:
                assert torch.equal(vp[at, j % page], x[c[s]:c[s + 1], H + KV:])
        ref.check_attention(out[:n], lse[:n], ref.attention(q[:n], kp, vp, table, c, lens, D ** -0.5))
        assert (out[n:] == 7).all()


@pytest.mark.parametrize("H, KV, D, shared, q", [(64, 1, 128, True, 1), (128, 1, 128, True, 3), (64, 1, 256, True, 2), (8, 2, 128, False, 1)])
def test_many_segments_of_one_unit(H, KV, D, shared, q):
    """Behind the prefix every sequence has a unit of rows or less: the loads of one CTA run many segments ahead of its
    outputs. Against dsv4_paged_attn on the same tables."""
    m = lib()
    g = gen(H)
    batch, pre, page = 1500, 250, 32
    lens = [pre + q + (s * 29) % 100 for s in range(batch)]
    c = Cache(g, lens, [0, 700, 701, batch], [pre, 100, pre - 3], page, KV, D, shared)
    x = normal(g, batch * q, H, D, std=2.0)
    cu = cu_of([q] * batch)
    out, lse = attend(c, x, cu)
    want, wl = torch.empty_like(x), torch.empty(batch * q, H, device="cuda")
    a = m.paged_attn_args(x, want, c.k, c.table, i32(cu), c.kv_len, v_pages=c.v, lse=wl, max_q=q)
    ws = torch.empty(m.dsv4_paged_attn_workspace_size(a), dtype=torch.uint8, device="cuda")
    m.dsv4_paged_attn(a, ws)
    # both within 2^-8 of |out| + 1.5 x 2^-8 of sum p |v| of the exact values; sum p |v| is at most max |v|
    top = (c.k if c.v is None else c.v).float().nan_to_num().abs().max()
    assert ((out.float() - want.float()).abs() <= 2 * 2.0 ** -8 * (want.float().abs() + 1.5 * top)).all()
    assert ((lse - wl).abs() <= 2.0 ** -12).all()
    for s in (0, 699, 700, batch - 1):
        one = ref.attention(x[s * q:(s + 1) * q], c.k, c.v, c.table[s:s + 1], [0, q], [lens[s]], D ** -0.5)
        ref.check_attention(out[s * q:(s + 1) * q], lse[s * q:(s + 1) * q], one)


@pytest.mark.parametrize("H, KV, D, shared, batch", [(32, 1, 128, True, 82), (32, 2, 256, False, 42), (64, 1, 512, True, 12)])
def test_many_queries_beside_one_that_is_cut_into_many_parts(H, KV, D, shared, batch):
    """Two sequences behind a prefix that most of the device works on, the rest behind a short one."""
    g = gen(batch)
    lens = [20011, 20060] + [21 + (s * 13) % 150 for s in range(batch - 2)]
    c = Cache(g, lens, [0, 2, batch], [20000, 20], 64, KV, D, shared)
    q = normal(g, batch, H, D, std=2.0)
    sink = normal(g, H, dtype=torch.float32)
    cu = cu_of([1] * batch)
    out, lse = attend(c, q, cu, sink=sink)
    ref.check_attention(out, lse, ref.attention(q, c.k, c.v, c.table, cu, lens, D ** -0.5, sink=sink))


def test_pages_past_32_bit_offsets():
    """A pool of 2^31 elements and more, of which the last pages are appended to and read."""
    m = lib()
    g = gen(9)
    H, D, page, pool, pre, own = 16, 512, 64, 66000, 130, 70
    kp = torch.empty(pool, page, 1, D, dtype=torch.bfloat16, device="cuda")
    assert kp.numel() > 2 ** 31
    ids = list(range(pool - 1, pool - 9, -1))
    table = i32([[ids[0], ids[1], ids[2], ids[3]], [ids[0], ids[1], ids[4], ids[5]]])
    lens = [pre + own, pre + own - 9]
    slots, x = [], []
    shared = normal(g, pre, 1, D)
    for s in range(2):                       # both append the prefix's rows where their pages are their own
        first = 0 if s == 0 else 128
        slots += [int(table[s, r // page]) * page + r % page for r in range(first, lens[s])]
        x += [shared[first:], normal(g, lens[s] - pre, 1, D)]
    x, T = torch.cat(x), len(slots)
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    m.dsv4_rope(m.rope_args(None, None, pos, k=x, k_out=kp, slots=torch.tensor(slots, device="cuda"), rope_dim=64))
    at = torch.tensor(slots, device="cuda")
    assert torch.equal(kp[at // page, at % page], x)          # (at position 0 nothing turns)
    q = normal(g, 2, H, D, std=2.0)
    out, lse = torch.empty_like(q), torch.empty(2, H, device="cuda")
    a = m.paged_prefix_args(q, out, kp, table, i32([0, 1, 2]), i32(lens), i32([pre]), lse=lse)
    ws = torch.empty(m.dsv4_paged_prefix_attn_workspace_size(a), dtype=torch.uint8, device="cuda")
    m.dsv4_paged_prefix_attn(a, ws)
    assert m.dsv4_read_error_word(ws) == (0, 0)
    ref.check_attention(out, lse, ref.attention(q, kp, None, table, [0, 1, 2], lens, D ** -0.5))
