"""Plans and rotary positions of a step on the GPU, against their plain forms, at the sizes, layouts and counts where
they can go wrong. Integers and copied channels are compared bit for bit; the tolerance of the rotation is derived in
step_reference.py."""
from __future__ import annotations

import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import step_reference as ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def i64(x):
    return torch.tensor(x, dtype=torch.int64, device="cuda")


# ------------------------------------------------------------------ plans
class Plan:
    """A plan's arrays on the GPU, built from lists."""

    def __init__(self, new, kv, held, shared, nxt, table, free, count, *, page, pool, total, in_place=False, optional=True):
        m = lib()
        self.lists = (new, kv, held, shared, nxt, table, free, count)
        self.kw = dict(page=page, pool=pool, total=total)
        B = len(kv)
        self.new, self.kv, self.held = None if new is None else i32(new), i32(kv), i32(held)
        self.shared, self.nxt = None if shared is None else i32(shared), None if nxt is None else i64(nxt)
        self.table = i32(table).view(B, -1) if B else torch.zeros(0, 4, dtype=torch.int32, device="cuda")
        self.free, self.count = i32(free), i32([count])
        self.cu = i32([77] * (B + 1))
        self.slots, self.pos, self.seq = i64([77] * total), i64([77] * total), i32([77] * total)
        out = {}
        self.kv_out, self.held_out, self.nxt_out, self.count_out = self.kv, self.held, self.nxt, self.count
        if not in_place:
            self.kv_out, self.held_out, self.count_out = i32([77] * B), i32([77] * B), i32([77])
            self.nxt_out = None if nxt is None else i64([77] * B)
            out = dict(kv_len_out=self.kv_out, held_out=self.held_out, free_count_out=self.count_out, next_pos_out=self.nxt_out)
        more = dict(pos=self.pos, seq=self.seq) if optional else {}
        self.args = m.paged_plan_args(self.new, self.kv, self.held, self.table, self.free, self.count, self.cu, self.slots,
                                      page_size=page, num_pages=pool, shared=self.shared, next_pos=self.nxt, **more, **out)
        self.ws = torch.full((m.dsv4_paged_plan_workspace_size(self.args),), 0xA5, dtype=torch.uint8, device="cuda")
        self.optional = optional

    def call(self):
        lib().dsv4_paged_plan(self.args, self.ws)

    def check(self):
        want, err = ref.plan(*self.lists, **self.kw)
        assert lib().dsv4_read_error_word(self.ws)[1] == err
        got = dict(cu_q=self.cu, slots=self.slots, table=self.table, free=self.free, kv_len=self.kv_out, held=self.held_out)
        if self.optional:
            got.update(pos=self.pos, seq=self.seq)
        if self.nxt is not None:
            got["next_pos"] = self.nxt_out
        for k, t in got.items():
            assert t.tolist() == want[k], k
        assert self.count_out.tolist() == [want["count"]]
        return want, err


def random_plan(r, B, q, ctx, page, *, spare, extra=0, total=None, **kw):
    """Requests in the middle of their lives; `spare` free pages beyond what the step needs."""
    kv = [r.choice([0, r.randint(0, ctx), page * r.randint(0, ctx // page)]) for _ in range(B)]
    new = [r.choice([0, 1, r.randint(0, q)]) for _ in range(B)]
    held = [max(0, -(-n // page) + r.choice([0, 0, 0, 1, 3])) for n in kv]
    shared = [r.choice([0, min(2, h), h + 1]) for h in held]
    width = max(max(h, -(-(a + b) // page)) for a, b, h in zip(kv, new, held)) + 1
    need = sum(max(0, -(-(a + b) // page) - h) for a, b, h in zip(kv, new, held))
    left = max(0, need + spare)
    pool = sum(held) + left + 5
    ids = list(range(pool))
    r.shuffle(ids)
    table = [[ids.pop() if j < h else -9 for j in range(width)] for h in held]
    free = [ids.pop() for _ in range(left)]
    cap = left + sum(held) + extra
    return Plan(new, kv, held, shared, [r.randint(0, 1 << 33) for _ in kv], table, free + [-5] * (cap - left), left, page=page, pool=pool,
                total=sum(new) + 7 if total is None else total, **kw)


@pytest.mark.parametrize("B, q, ctx, page", [(1, 1, 100, 16), (16, 1, 8192, 64), (33, 5, 300, 8), (513, 40, 500, 48),
                                             (2048, 3, 200, 24), (7, 3000, 9000, 16), (2000, 97, 5000, 128), (3, 9, 70000, 65536)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plans(B, q, ctx, page, in_place):
    r = random.Random(B * 31 + q)
    p = random_plan(r, B, q, ctx, page, spare=3, in_place=in_place)
    p.call()
    _, err = p.check()
    assert err == 0


@pytest.mark.parametrize("spare", [-1, -4, -10 ** 6])
@pytest.mark.parametrize("B", [5, 300])
def test_plans_with_too_few_pages(spare, B):
    """The first that the stack cannot serve, and all behind it that need a page, keep what they have."""
    r = random.Random(B - spare)
    p = random_plan(r, B, 60, 400, 16, spare=spare)
    p.call()
    want, err = p.check()
    assert err in (0, ref.NO_PAGES)                                   # (what is given back may be enough)
    assert err or spare != -10 ** 6


def test_plans_where_returned_pages_are_taken_at_once():
    """Nothing free: what ended requests give back serves the others in the same step, shared pages stay."""
    p = Plan([16, 0, 40, 0], [16, 0, 0, 5], [1, 3, 0, 4], [0, 1, 0, 0], None, [[1, -1, -1, -1], [2, 3, 4, -1], [-1] * 4, [5, 6, 7, 8]],
             [-1] * 6, 0, page=16, pool=9, total=64)
    p.call()
    want, err = p.check()
    assert err == 0 and want["table"][0][1] == 8 and want["table"][2][:3] == [7, 6, 4] and want["count"] == 1


@pytest.mark.parametrize("what", ["new", "kv", "held", "shared", "count", "count_high", "tokens", "width", "page", "room"])
def test_plans_with_counts_out_of_range(what):
    new, kv, held, shared = [3, 2, 20], [10, 0, 16], [1, 0, 4], [0, 0, 0]
    table = [[0, -1, -1, -1], [-1] * 4, [1, 2, 3, 4]]
    free, count, total = [5, 6, 7, 8, -1, -1, -1], 4, 40
    if what == "new":
        new[1] = -3
    if what == "kv":
        kv[2], kv[1] = 100, -1
    if what == "held":
        held[0], held[1] = 9, -2
        table[0] = [0, 9, 10, 11]
    if what == "shared":
        shared[2] = -1
    if what == "count":
        count = -4
    if what == "count_high":
        count = 9
    if what == "tokens":
        total = 4
    if what == "width":
        new[0] = 55
    if what == "page":
        table[0][0], free[3] = 99, -2
    if what == "room":
        free, kv[2], new[2], new[0], new[1] = free[:5], 0, 0, 0, 0
    p = Plan(new, kv, held, shared, [5, 6, 7], table, free, count, page=16, pool=20, total=total)
    p.call()
    _, err = p.check()
    assert err & ref.BAD_INDEX or (what == "count" and err)


def test_plans_of_nothing():
    for B, total in ((0, 5), (4, 0), (0, 0)):
        p = Plan([0] * B, [3] * B, [1] * B, None, None, [[i] * 2 for i in range(B)], [9], 1, page=8, pool=12, total=total)
        p.call()
        assert p.check()[1] == 0
    p = Plan(None, [3, 0], [4, 2], None, None, [[0, 1, 2, 3], [4, 5, 6, 7]], [-1] * 8, 0, page=8, pool=12, total=3, optional=False)
    p.call()
    assert p.check()[0]["count"] == 5


def test_plans_replayed_from_a_graph_in_place():
    """Twenty steps of one captured call, the state carried on; a second graph of another batch between them."""
    r = random.Random(4)
    mk = lambda seed: random_plan(random.Random(seed), 40, 3, 200, 8, spare=900, in_place=True)  # noqa: E731
    plans = [mk(1), mk(2)]
    width = 400 // 8 + 40
    for p in plans:                                                   # room for all steps
        new, kv, held, shared, nxt, table, free, count = p.lists
        table = [row + [-9] * (width - len(row)) for row in table]
        p.__init__(new, kv, held, [0] * len(kv), nxt, table, free, count, page=8, pool=p.kw["pool"], total=150, in_place=True)
    graphs = []
    for p in plans:
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            p.call()
        graphs.append(g)
    for step in range(20):
        for p, g in zip(plans, graphs):
            g.replay()
            want, err = p.check()
            assert err == 0
            new = [r.choice([0, 1, 3]) for _ in p.lists[0]]
            kv = list(want["kv_len"])
            if step % 5 == 4:                                         # a request ends, another loses half its rows
                kv[step], kv[step + 1] = 0, kv[step + 1] // 2
            p.new.copy_(i32(new))
            p.kv.copy_(i32(kv))
            p.lists = (new, kv, want["held"], p.lists[3], want["next_pos"], want["table"], want["free"], want["count"])


def test_plans_on_another_stream():
    r = random.Random(8)
    p = random_plan(r, 64, 9, 700, 16, spare=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lib().dsv4_paged_plan(p.args, p.ws, stream=s)
    s.synchronize()
    p.check()


# ------------------------------------------------------------------ rotary positions
def check_rope(got, x, pos, freqs, first, layout, inverse=False, magnitude=1.0, where=None):
    want, tol = ref.rope(x, pos, freqs, first, layout, inverse, magnitude)
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if where is not None:
        bad &= where[:, None, None]
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off; worst {(err / tol.clamp(min=1e-300))[bad].max():.2f} times the tolerance"


PARTS = [(128, 128, 0), (128, 64, 64), (128, 64, 0), (64, 64, 0), (512, 64, 448), (256, 256, 0), (96, 46, 50), (192, 2, 190), (8, 8, 0),
         (8, 2, 4), (1024, 512, 8), (128, 30, 34), (72, 40, 16)]


@pytest.mark.parametrize("dim, rope, first", PARTS)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(dim, rope, first, layout, dtype, inverse):
    m = lib()
    g = gen(dim + rope)
    dt = TYPES[dtype]
    for T, H, KV in ((1, 1, 1), (3, 5, 2), (700, 3, 1)):
        x = torch.empty(T, H + KV + 1, dim, dtype=dt, device="cuda").normal_(generator=g)
        q, k = x[:, :H], x[:, H:H + KV]
        pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
        qo = torch.full((T, H, dim), 9.0, dtype=dt, device="cuda")
        ko = torch.full((T, KV + 2, dim), 9.0, dtype=dt, device="cuda")
        m.dsv4_rope(m.rope_args(q, qo, pos, k=k, k_out=ko[:, 1:1 + KV], rope_dim=rope, first=first, layout=layout, inverse=inverse))
        f = ref.frequencies(rope, 1e4, "none")
        check_rope(qo, q, pos, f, first, layout, inverse)
        check_rope(ko[:, 1:1 + KV], k, pos, f, first, layout, inverse)
        assert (ko[:, 0] == 9).all() and (ko[:, -1] == 9).all()


@pytest.mark.parametrize("scaling", ["linear", "turns", "index"])
@pytest.mark.parametrize("factor, original, fast, slow, theta", [(8.0, 4096, 32.0, 1.0, 1e4), (40.0, 4096, 32.0, 1.0, 1e6), (1.0, 128, 2.0, 1.0, 1e4),
                                                                 (4.0, 8, 32.0, 1.0, 1e4), (2.0, 1 << 30, 4.0, 1.0, 5e5)])
def test_scaled_frequencies(scaling, factor, original, fast, slow, theta):
    m = lib()
    g = gen(3)
    for rope, layout, mag in ((128, "half", 1.0), (64, "interleaved", 1.2079)):
        x = torch.empty(50, 4, 128, device="cuda").normal_(generator=g)
        pos = torch.randint(0, 1 << 17, (50,), generator=g, device="cuda")
        out = torch.empty_like(x)
        m.dsv4_rope(m.rope_args(x, out, pos, rope_dim=rope, first=0, layout=layout, rope_theta=theta, scaling=scaling, factor=factor,
                                original_len=original, beta_fast=fast, beta_slow=slow, magnitude=mag))
        check_rope(out, x, pos, ref.frequencies(rope, theta, scaling, factor, original, fast, slow), 0, layout, magnitude=mag)


def test_far_and_negative_positions():
    m = lib()
    x = torch.empty(6, 2, 64, device="cuda").normal_(generator=gen(1))
    pos = i64([0, -1, 1 << 31, 1 << 40, -(1 << 33), 123456789012])
    out = torch.empty_like(x)
    m.dsv4_rope(m.rope_args(x, out, pos, rope_dim=64, layout="half"))
    check_rope(out, x, pos, ref.frequencies(64, 1e4, "none"), 0, "half")
    assert torch.equal(out[0], x[0])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [1, 50, 900])
def test_append(layout, dtype, T):
    """Rows by slot; tokens without one store nothing, and no other row changes."""
    m = lib()
    g = gen(T)
    dt, H, KV, D, page = TYPES[dtype], 8, 2, 96, 24
    x = torch.empty(T, H + 2 * KV, D, dtype=dt, device="cuda").normal_(generator=g)
    n = T // page + 3
    kp = torch.empty(n, page, KV, D, dtype=dt, device="cuda").normal_(generator=g)
    vp = kp.clone()
    k0, v0 = kp.clone(), vp.clone()
    slots = torch.randperm(n * page, generator=g, device="cuda")[:T]
    slots[::7] = -1
    slots[3::11] = n * page + 5
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
    q, k, v = x[:, :H], x[:, H:H + KV], x[:, H + KV:]
    qo = torch.empty(T, H, D, dtype=dt, device="cuda")
    m.dsv4_rope(m.rope_args(q, qo, pos, k=k, k_out=kp, v=v, v_out=vp, slots=slots, rope_dim=64, first=16, layout=layout))
    f = ref.frequencies(64, 1e4, "none")
    check_rope(qo, q, pos, f, 16, layout)
    on = (slots >= 0) & (slots < n * page)
    at = torch.where(on, slots, 0)
    check_rope(kp.flatten(0, 1)[at], k, pos, f, 16, layout, where=on)
    assert torch.equal(vp.flatten(0, 1)[at][on], v[on])
    rest = torch.ones(n * page, dtype=torch.bool, device="cuda")
    rest[at[on]] = False
    assert torch.equal(kp.flatten(0, 1)[rest], k0.flatten(0, 1)[rest]) and torch.equal(vp.flatten(0, 1)[rest], v0.flatten(0, 1)[rest])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dim, rope, first", [(128, 128, 0), (128, 64, 64), (96, 46, 50)])
def test_in_place_and_alone(layout, dim, rope, first):
    m = lib()
    x = torch.empty(40, 6, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(2))
    pos = torch.arange(40, device="cuda") * 1000
    kw = dict(rope_dim=rope, first=first, layout=layout)
    q, k = torch.empty_like(x), torch.empty_like(x)
    m.dsv4_rope(m.rope_args(x, q, pos, **kw))
    m.dsv4_rope(m.rope_args(None, None, pos, k=x, k_out=k, **kw))
    y = x.clone()
    m.dsv4_rope(m.rope_args(y[:, :4], y[:, :4], pos, k=y[:, 4:], k_out=y[:, 4:], **kw))
    assert torch.equal(q, k) and torch.equal(q, y)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_channels_outside_the_part_are_copied(layout):
    """Also NaN and infinities, bit for bit; inside, a NaN stays with its pair."""
    m = lib()
    x = torch.empty(5, 3, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(6))
    x[:, :, :10] = float("inf")
    x[:, :, 5] = float("nan")
    x[:, :, 50:] = float("-inf")
    x[1, 2, 20] = float("nan")
    out = torch.empty_like(x)
    m.dsv4_rope(m.rope_args(x, out, torch.arange(5, device="cuda"), rope_dim=40, first=10, layout=layout))
    same = [i for i in range(64) if not 10 <= i < 50]
    assert torch.equal(out.view(torch.int16)[..., same], x.view(torch.int16)[..., same])
    nan = torch.isnan(out[..., 10:50]).nonzero().tolist()
    assert nan == [[1, 2, 10], [1, 2, 11 if layout == "interleaved" else 30]]


def test_backward_is_the_transpose():
    """The gradient of sum(w * rope(x)) is the inverse rotation of w, also by differences of the plain form."""
    m = lib()
    g = gen(9)
    x, w = (torch.empty(7, 4, 32, device="cuda").normal_(generator=g) for _ in range(2))
    pos = torch.randint(0, 5000, (7,), generator=g, device="cuda")
    kw = dict(rope_dim=24, first=4, layout="half", scaling="turns", factor=4.0, original_len=64, beta_fast=4.0, magnitude=1.3)
    grad = torch.empty_like(w)
    m.dsv4_rope(m.rope_args(w, grad, pos, inverse=True, **kw))
    f = ref.frequencies(24, 1e4, "turns", 4.0, 64, 4.0, 1.0)
    xd = x.double().requires_grad_()
    y, _ = ref.rope(xd.detach(), pos, f, 4, "half", magnitude=1.3)
    for i, c in ((0, 4), (3, 17), (6, 31), (2, 0)):
        d = xd.detach().clone()
        d[i, 1, c] += 1e-3
        y1, _ = ref.rope(d, pos, f, 4, "half", magnitude=1.3)
        diff = ((y1 - y) * w.double()).sum() / 1e-3
        assert abs(diff - grad[i, 1, c]) <= 1e-5                       # linear: 64-bit rounding over the step, and grad's fp32
    check_rope(grad, w, pos, f, 4, "half", True, 1.3)


def test_rope_in_graphs_and_streams():
    m = lib()
    x = torch.empty(30, 8, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(2))
    pos = torch.arange(30, device="cuda")
    out = torch.empty_like(x)
    a = m.rope_args(x, out, pos, rope_dim=128, layout="half")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.dsv4_rope(a)
    f = ref.frequencies(128, 1e4, "none")
    for step in range(3):
        pos += 1
        g.replay()
        check_rope(out, x, pos, f, 0, "half")
    out.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.dsv4_rope(a, stream=s)
    s.synchronize()
    check_rope(out, x, pos, f, 0, "half")
    e = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    m.dsv4_rope(m.rope_args(e, e, pos[:0], rope_dim=64))


def test_a_step_in_one_graph():
    """Plan, rotation with append, attention: three steps of one graph over lengths that stay on the device."""
    import paged_reference as pref
    m = lib()
    g = gen(12)
    B, H, KV, D, page, T = 3, 8, 2, 128, 16, 12
    r = random.Random(3)
    kv = [40, 0, 90]
    held = [-(-n // page) for n in kv]
    width, pool = 12, 40
    ids = list(range(pool))
    r.shuffle(ids)
    table = i32([[ids.pop() if j < h else -1 for j in range(width)] for h in held])
    free = i32(ids + [-1] * (pool - len(ids)))
    count, kvt, heldt = i32([len(ids)]), i32(kv), i32(held)
    new, cu = i32([0] * B), i32([0] * (B + 1))
    slots, pos = i64([0] * T), i64([0] * T)
    kp = torch.empty(pool, page, KV, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    vp = torch.empty_like(kp).normal_(generator=g)
    x = torch.empty(T, H + 2 * KV, D, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, H, device="cuda")
    plan = m.paged_plan_args(new, kvt, heldt, table, free, count, cu, slots, page_size=page, num_pages=pool, pos=pos)
    rot = m.rope_args(x[:, :H], q, pos, k=x[:, H:H + KV], k_out=kp, v=x[:, H + KV:], v_out=vp, slots=slots, rope_dim=128, layout="half")
    att = m.paged_attn_args(q, out, kp, table, cu, kvt, v_pages=vp, lse=lse)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (m.dsv4_paged_plan_workspace_size(plan),
                                                                    m.dsv4_paged_attn_workspace_size(att))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.dsv4_paged_plan(plan, ws[0])
        m.dsv4_rope(rot)
        m.dsv4_paged_attn(att, ws[1])
    for ns in ([1, 9, 1], [1, 1, 1], [4, 0, 8]):
        new.copy_(i32(ns))
        x.normal_(generator=g)
        out.fill_(7.0)
        before = kvt.tolist()
        graph.replay()
        assert m.dsv4_read_error_word(ws[0]) == (0, 0) and m.dsv4_read_error_word(ws[1]) == (0, 0)
        lens = [a + b for a, b in zip(before, ns)]
        assert kvt.tolist() == lens
        c = cu.tolist()
        f = ref.frequencies(128, 1e4, "none")
        n = c[-1]
        check_rope(q[:n], x[:n, :H], pos[:n], f, 0, "half")
        for s in range(B):
            rows = torch.arange(before[s], lens[s], device="cuda")
            at = table[s].long()[rows // page]
            check_rope(kp[at, rows % page], x[c[s]:c[s + 1], H:H + KV], rows, f, 0, "half")
            assert torch.equal(vp[at, rows % page], x[c[s]:c[s + 1], H + KV:])
        pref.check_attention(out[:n], lse[:n], pref.attention(q[:n], kp, vp, table, c, lens, D ** -0.5))
        assert (out[n:] == 7).all()
