"""CPU-only checks of the step entry points: bad arguments are refused on the host before any CUDA call, and
workspaces are sized without one."""
from __future__ import annotations

import ctypes

import pytest

FAKE = 0x7F0000000000   # aligned fake device addresses: never dereferenced on the host path


@pytest.fixture(scope="module")
def lib():
    from compressed_sparse_attention_08_gb300 import _build, _abi
    _build.build()
    return _abi.library()


def _p(i, off=0):
    return ctypes.c_void_p(FAKE + 4096 * i + off)


def _plan(**over):
    from compressed_sparse_attention_08_gb300._abi import PagedPlanArgs
    a = dict(new_len=_p(1), kv_len=_p(2), held=_p(3), shared=_p(4), next_pos=_p(5), block_table=_p(6), free_pages=_p(7),
             free_count=_p(8), cu_q=_p(9), kv_len_out=_p(10), held_out=_p(11), next_pos_out=_p(12), free_count_out=_p(13),
             slots=_p(14), pos=_p(15), seq=_p(16), batch=4, total_q=64, page_size=16, num_pages=100, max_pages=16, free_cap=100)
    a.update(over)
    return PagedPlanArgs(**a)


def _rope(**over):
    from compressed_sparse_attention_08_gb300._abi import RopeArgs
    a = dict(q=_p(1), k=_p(2), v=_p(3), q_out=_p(4), k_out=_p(5), v_out=_p(6), slots=_p(7), pos=_p(8), q_stride=80 * 128,
             k_stride=80 * 128, v_stride=80 * 128, q_out_stride=64 * 128, k_out_stride=0, tokens=4, heads=64, kv_heads=8, dim=128,
             page_size=16, num_pages=8, dtype=0, rope_dim=64, first=64, layout=0, inverse=0, scaling=3, rope_theta=1e4, factor=8.0,
             original_len=4096, beta_fast=32.0, beta_slow=1.0, magnitude=1.0)
    a.update(over)
    return RopeArgs(**a)


def _prefix(**over):
    from compressed_sparse_attention_08_gb300._abi import PagedPrefixArgs
    a = dict(q=_p(1), k_pages=_p(2), v_pages=None, block_table=_p(3), cu_q=_p(4), kv_len=_p(5), prefix_len=_p(6), group_start=_p(7),
             sink=_p(8), out=_p(9), lse=_p(10), out_rope_pos=_p(11), q_stride=512 * 64, batch=4, groups=2, total_q=4, heads=64,
             kv_heads=1, dim=512, page_size=64, num_pages=100, max_pages=16, scale=0.04, out_rope_dim=64, out_rope_theta=1e4)
    a.update(over)
    return PagedPrefixArgs(**a)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(batch=2049), dict(groups=0), dict(groups=2049), dict(total_q=-1), dict(total_q=(1 << 24) + 1), dict(heads=0),
    dict(heads=1025), dict(heads=6, kv_heads=4), dict(kv_heads=0), dict(dim=64), dict(dim=384), dict(page_size=12), dict(page_size=0),
    dict(num_pages=0), dict(max_pages=0), dict(max_pages=1 << 25), dict(q_stride=8), dict(q_stride=512 * 64 + 4), dict(scale=float("nan")),
    dict(q=None), dict(q=_p(1, 8)), dict(k_pages=_p(2, 8)), dict(v_pages=_p(12, 8)), dict(block_table=None), dict(cu_q=None),
    dict(kv_len=None), dict(prefix_len=None), dict(prefix_len=_p(6, 2)), dict(group_start=None), dict(group_start=_p(7, 1)),
    dict(sink=_p(8, 2)), dict(out=None), dict(lse=_p(10, 2)), dict(out_rope_pos=_p(11, 4)), dict(out_rope_dim=0), dict(out_rope_dim=65),
    dict(out_rope_dim=130), dict(out_rope_theta=-1.0)])
def test_prefix_rejects_on_host(lib, bad):
    assert lib.dsv4_paged_prefix_attn(ctypes.byref(_prefix(**bad)), _p(20), 1 << 40, None) == 1, bad


def test_prefix_workspace(lib):
    size = lib.dsv4_paged_prefix_attn_workspace_size
    need = size(ctypes.byref(_prefix()))
    assert need > 256 and size(None) == 0 and size(ctypes.byref(_prefix(max_pages=1024))) == need
    more = size(ctypes.byref(_prefix(total_q=1004)))
    assert 2 * 1000 * 64 * 512 * 4 <= more - need <= 2 * 1000 * 64 * 520 * 4 + 4096
    assert size(ctypes.byref(_prefix(total_q=1 << 24, heads=1024, kv_heads=1024))) > 1 << 45       # (not wrapped)
    for bad in (dict(batch=-1), dict(groups=0), dict(kv_heads=0), dict(heads=6, kv_heads=4), dict(dim=0), dict(total_q=-1)):
        assert size(ctypes.byref(_prefix(**bad))) == 0, bad
    for ws, n in ((_p(20), need - 1), (None, need), (_p(20, 8), need)):
        assert lib.dsv4_paged_prefix_attn(ctypes.byref(_prefix()), ws, n, None) == 1
    assert lib.dsv4_paged_prefix_attn(None, _p(20), need, None) == 1


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(batch=2049), dict(total_q=-1), dict(total_q=(1 << 24) + 1), dict(page_size=0), dict(page_size=12),
    dict(page_size=65544), dict(num_pages=0), dict(max_pages=0), dict(max_pages=1 << 26), dict(free_cap=-1), dict(kv_len=None),
    dict(held=None), dict(block_table=None), dict(free_pages=None), dict(free_count=None), dict(free_count_out=None), dict(cu_q=None),
    dict(kv_len_out=None), dict(held_out=None), dict(slots=None), dict(next_pos=None), dict(next_pos_out=None), dict(new_len=_p(1, 2)),
    dict(shared=_p(4, 1)), dict(slots=_p(14, 4)), dict(pos=_p(15, 4)), dict(seq=_p(16, 2)), dict(next_pos=_p(5, 4))])
def test_plan_rejects_on_host(lib, bad):
    assert lib.dsv4_paged_plan(ctypes.byref(_plan(**bad)), _p(20), 1 << 20, None) == 1, bad


def test_plan_workspace(lib):
    need = lib.dsv4_paged_plan_workspace_size(ctypes.byref(_plan()))
    assert need >= 256 and lib.dsv4_paged_plan_workspace_size(None) == 0
    assert lib.dsv4_paged_plan_workspace_size(ctypes.byref(_plan(batch=2049))) == 0
    for ws, n in ((_p(20), need - 1), (None, need), (_p(20, 8), need)):
        assert lib.dsv4_paged_plan(ctypes.byref(_plan()), ws, n, None) == 1
    assert lib.dsv4_paged_plan(None, _p(20), need, None) == 1


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(heads=-1), dict(heads=1025), dict(kv_heads=1025), dict(dim=0), dict(dim=12),
    dict(dim=1032), dict(dtype=3), dict(dtype=-1), dict(rope_dim=0), dict(rope_dim=63), dict(rope_dim=130), dict(first=-2), dict(first=66),
    dict(first=63), dict(layout=2), dict(layout=-1), dict(inverse=2), dict(scaling=4), dict(scaling=-1), dict(rope_theta=0.0),
    dict(rope_theta=NAN), dict(rope_theta=1.0), dict(factor=0.0), dict(factor=INF), dict(original_len=0), dict(beta_slow=0.0),
    dict(beta_fast=1.0), dict(beta_fast=INF), dict(magnitude=NAN), dict(pos=None), dict(pos=_p(8, 4)), dict(slots=_p(7, 4)), dict(q=None),
    dict(q=_p(1, 8)), dict(q_out=None), dict(q_stride=8), dict(q_stride=80 * 128 + 4), dict(q_out_stride=0), dict(k=None), dict(k_out=None),
    dict(k_out=_p(5, 8)), dict(v=None), dict(v_out=None), dict(v_stride=8), dict(slots=None),
    dict(slots=None, v=None, v_out=None), dict(slots=None, v=None, v_out=None, k_out=_p(2), k_out_stride=8 * 128), dict(k_out=_p(2)),
    dict(page_size=0), dict(num_pages=0), dict(heads=0), dict(kv_heads=0), dict(q_out=_p(1))])
def test_rope_rejects_on_host(lib, bad):
    assert lib.dsv4_rope(ctypes.byref(_rope(**bad)), None) == 1, bad


def test_binding_refuses_shapes_and_types():
    torch = pytest.importorskip("torch")
    import compressed_sparse_attention_08_gb300 as m
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        m.rope_args(q, q, pos, rope_dim=64)
    with pytest.raises(TypeError, match="fp32"):
        m.rope_args(q.double(), q.double(), pos, rope_dim=64)
    with pytest.raises(ValueError, match="layout"):
        m.rope_args(q, q, pos, rope_dim=64, layout="other")
    with pytest.raises(ValueError, match="outputs"):
        m.rope_args(q, None, pos, rope_dim=64)
    with pytest.raises(ValueError, match="slots"):
        m.rope_args(q, q, pos, k=q, k_out=q, v=q, v_out=q, rope_dim=64)
    with pytest.raises(ValueError, match="pool"):
        m.rope_args(q, q, pos, k=q, k_out=q, slots=pos, rope_dim=64)
    with pytest.raises(ValueError, match="pos"):
        m.rope_args(q, q, pos[:1], rope_dim=64)
    n, t = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="cu_q"):
        m.paged_plan_args(n, n, n, t, n, n[:1], n, pos, page_size=16, num_pages=4)
    with pytest.raises(ValueError, match="held"):
        m.paged_plan_args(n, n, n[:1], t, n, n[:1], torch.zeros(3), pos, page_size=16, num_pages=4)
    pages = torch.zeros(4, 16, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        m.paged_prefix_args(q, q, pages, t, torch.zeros(3, dtype=torch.int32), n, n[:1])
    with pytest.raises(ValueError, match="next_pos"):
        m.paged_plan_args(n, n, n, t, n, n[:1], torch.zeros(3), pos, page_size=16, num_pages=4, next_pos_out=pos)


@pytest.mark.parametrize("struct, name", [("PagedPlanArgs", "total_q"), ("RopeArgs", "rope_dim"), ("RopeArgs", "first")])
def test_counts_do_not_wrap(struct, name):
    from compressed_sparse_attention_08_gb300 import _abi
    cls = getattr(_abi, struct)
    fields = [f for f, _ in cls._fields_]
    values = [0] * len(fields)
    values[fields.index(name)] = (1 << 32) + 64
    with pytest.raises(ValueError, match=name):
        _abi._struct(cls, *values)


def test_the_status_of_missing_pages_has_words(lib):
    from compressed_sparse_attention_08_gb300 import _abi
    assert "pages" in _abi.dsv4_status_string(_abi.DSV4_ERR_NO_PAGES)
