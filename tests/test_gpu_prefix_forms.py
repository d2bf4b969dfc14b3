"""Attention behind shared prefixes: every sequence of large batches against the 64-bit form, and the forms of tiles, head
blocks, halves of V's channels and scales that the dispatch admits."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import paged_reference as ref  # noqa: E402
from test_gpu_prefix import Cache, args_of, attend, check, cu_of, gen, i32, lib, normal, workspace  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_sparse_attention_08_gb300 import _build
    _build.build()


@pytest.mark.parametrize("H, KV, D, shared, q", [(64, 1, 128, True, 1), (128, 1, 128, True, 3), (64, 1, 256, True, 2), (8, 2, 128, False, 1),
                                                 (64, 1, 512, True, 1)])
def test_every_sequence_of_many_short_segments(H, KV, D, shared, q):
    """Segments of one unit, whose descriptions run far ahead of the outputs: no sequence may get another's."""
    g = gen(H + q)
    batch, pre, page = 1500, 250, 32
    lens = [pre + q + (s * 29) % 100 for s in range(batch)]
    c = Cache(g, lens, [0, 700, 701, batch], [pre, 100, pre - 3], page, KV, D, shared)
    x = normal(g, batch * q, H, D, std=2.0)
    cu = cu_of([q] * batch)
    out, lse = attend(c, x, cu)
    check(c, x, cu, out, lse)


@pytest.mark.parametrize("H, KV, D, batch", [(32, 8, 128, 130), (16, 1, 512, 40), (16, 2, 256, 70)])
def test_every_sequence_behind_two_prefixes(H, KV, D, batch):
    g = gen(D + batch)
    pre = 1000
    lens = [pre + 1 + (s * 37) % 300 for s in range(batch)]
    c = Cache(g, lens, [0, batch // 3, batch], [pre, pre - 77], 16, KV, D, D != 128)
    q = normal(g, batch, H, D, std=2.0)
    sink = normal(g, H, dtype=torch.float32)
    cu = cu_of([1] * batch)
    out, lse = attend(c, q, cu, sink=sink)
    check(c, q, cu, out, lse, sink=sink)


# head blocks (more heads per KV head than a tile has rows) beside halves of V's channels, in whole and partial blocks
@pytest.mark.parametrize("H, KV, D, shared", [(200, 1, 512, True), (256, 1, 512, False), (258, 2, 512, True), (1024, 1, 512, True),
                                              (300, 1, 256, True), (300, 1, 128, False)])
@pytest.mark.parametrize("ns", [[1, 1, 1], [3, 1, 20]])
def test_head_blocks(H, KV, D, shared, ns):
    g = gen(H)
    lens = [290 + n for n in ns]
    c = Cache(g, lens, [0, 2, 3], [280, 130], 48, KV, D, shared)
    cu = cu_of(ns)
    q = normal(g, cu[-1], H, D, std=2.0)
    sink = normal(g, H, dtype=torch.float32)
    pos = torch.arange(cu[-1], device="cuda") * 1000
    out, lse = attend(c, q, cu, sink=sink, pos=pos)
    check(c, q, cu, out, lse, sink=sink, pos=pos)


def test_head_blocks_of_a_prefix_cut_into_many_parts():
    """Partial results per head block and half of V's channels."""
    g = gen(17)
    lens = [9001, 9040]
    c = Cache(g, lens, [0, 2], [9000], 64, 1, 512)
    q = normal(g, 2, 200, 512, std=2.0)
    out, lse = attend(c, q, [0, 1, 2])
    check(c, q, [0, 1, 2], out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.05, -1.0, 1.0])
@pytest.mark.parametrize("D, shared", [(128, True), (128, False), (256, True), (256, False), (512, True), (512, False)])
@pytest.mark.parametrize("ns", [[1, 1], [2, 70]])
def test_scales_in_every_form(scale, D, shared, ns):
    """Also with two tiles of queries over one unit (more than 32 tokens of four heads at 128 channels)."""
    g = gen(D + ns[1])
    lens = [300 + ns[0], 320 + ns[1]]
    c = Cache(g, lens, [0, 2], [290], 16, 2, D, shared)
    cu = cu_of(ns)
    q = normal(g, cu[-1], 8, D)
    sink = normal(g, 8, dtype=torch.float32)
    out, lse = attend(c, q, cu, scale=scale, sink=sink)
    check(c, q, cu, out, lse, scale=scale, sink=sink)


@pytest.mark.parametrize("D", [128, 512])
def test_two_calls_at_once(D):
    """On two streams, each with its own workspace, beside the call without prefixes on a third."""
    m = lib()
    g = gen(D + 3)
    lens = [3000 + s for s in (1, 50, 200)]
    c = Cache(g, lens, [0, 3], [3000], 16, 1, D)
    cu = cu_of([1] * 3)
    calls = []
    for _ in range(2):
        q = normal(g, 3, 16, D, std=2.0)
        out, lse = torch.zeros_like(q), torch.zeros(3, 16, device="cuda")
        a = args_of(c, q, cu, out, lse)
        calls.append((lambda a=a, ws=workspace(a), s=torch.cuda.Stream(): m.dsv4_paged_prefix_attn(a, ws, stream=s), q, out, lse))
    q = normal(g, 3, 16, D, std=2.0)
    out, lse = torch.zeros_like(q), torch.zeros(3, 16, device="cuda")
    a = m.paged_attn_args(q, out, c.k, c.table, i32(cu), c.kv_len, lse=lse, max_q=1)
    ws = torch.empty(m.dsv4_paged_attn_workspace_size(a), dtype=torch.uint8, device="cuda")
    calls.append((lambda s=torch.cuda.Stream(): m.dsv4_paged_attn(a, ws, stream=s), q, out, lse))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, *_ in calls:
            call()
    torch.cuda.synchronize()
    for _, q, out, lse in calls:
        check(c, q, cu, out, lse)
