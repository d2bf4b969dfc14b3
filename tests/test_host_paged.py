"""CPU-only checks of the paged-cache entry points: bad arguments are refused on the host before any
CUDA call, and workspaces are sized without one."""
from __future__ import annotations

import ctypes
import gc
import subprocess
import sys
import weakref

import pytest

FAKE = 0x7F0000000000   # aligned fake device addresses: never dereferenced on the host path


@pytest.fixture(scope="module")
def lib():
    from compressed_sparse_attention_08_gb300 import _build, _abi
    _build.build()
    return _abi.library()


def _p(i, off=0):
    return ctypes.c_void_p(FAKE + 4096 * i + off)


def _norm(**over):
    from compressed_sparse_attention_08_gb300._abi import NormRopeArgs
    a = dict(q=_p(1), k=_p(2), v=_p(3), q_out=_p(4), k_pages=_p(5), v_pages=_p(6), slots=_p(7), pos=_p(8), gamma_q=_p(9),
             gamma_k=_p(10), q_stride=512 * 64, k_stride=512, v_stride=512, q_out_stride=512 * 64, tokens=4, heads=64,
             kv_heads=1, dim=512, page_size=64, num_pages=8, rope_dim=64, eps=1e-6, rope_theta=1e4)
    a.update(over)
    return NormRopeArgs(**a)


def _attn(**over):
    from compressed_sparse_attention_08_gb300._abi import PagedAttnArgs
    a = dict(q=_p(1), k_pages=_p(2), v_pages=None, block_table=_p(3), cu_q=_p(4), kv_len=_p(5), sink=_p(6), out=_p(7),
             lse=_p(8), out_rope_pos=_p(9), q_stride=512 * 64, batch=4, total_q=4, heads=64, kv_heads=1, dim=512,
             page_size=64, num_pages=100, max_pages=16, max_q=1, window=0, scale=0.04, out_rope_dim=64, out_rope_theta=1e4)
    a.update(over)
    return PagedAttnArgs(**a)


def _weights(**over):
    from compressed_sparse_attention_08_gb300._abi import PagedWeightsArgs
    a = dict(q=_p(1), lse=_p(2), k_pages=_p(3), block_table=_p(4), cu_q=_p(5), kv_len=_p(6), acc_in=None, acc=_p(7),
             q_stride=512 * 64, batch=4, total_q=4, heads=64, kv_heads=1, dim=512, page_size=64, num_pages=100, max_pages=16,
             max_q=1, window=0, acc_rows=1024, scale=0.04)
    a.update(over)
    return PagedWeightsArgs(**a)


def _evict(**over):
    from compressed_sparse_attention_08_gb300._abi import PagedEvictArgs
    a = dict(k_pages=_p(1), v_pages=None, block_table=_p(2), out_table=_p(3), kv_len=_p(4), kv_len_out=_p(5), acc=_p(6),
             acc_out=_p(7), keep=_p(8), batch=4, kv_heads=1, dim=512, page_size=64, num_pages=100, max_pages=16, out_pages=8,
             acc_rows=1024, budget=500, recent=100)
    a.update(over)
    return PagedEvictArgs(**a)


COMMON = [dict(dim=64), dict(dim=384), dict(kv_heads=0), dict(page_size=0), dict(page_size=12), dict(page_size=65544),
          dict(num_pages=0)]
TABLES = COMMON + [dict(batch=-1), dict(batch=2049), dict(max_pages=0), dict(max_pages=1 << 25),
                   dict(batch=2048, max_pages=1 << 24), dict(block_table=None), dict(kv_len=_p(5, 2))]
QUERIES = [dict(heads=0), dict(heads=1025), dict(heads=6, kv_heads=4), dict(q_stride=512 * 64 - 8), dict(q_stride=512 * 64 + 4),
           dict(total_q=-1), dict(max_q=0), dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None),
           dict(cu_q=None), dict(k_pages=_p(2, 8))]


@pytest.mark.parametrize("bad", COMMON + [
    dict(tokens=-1), dict(heads=-1), dict(q=None), dict(q_out=None), dict(k=None), dict(v=None), dict(v_pages=None),
    dict(slots=None), dict(pos=None), dict(gamma_q=_p(9, 4)), dict(q_stride=8), dict(k_stride=516), dict(v_stride=8),
    dict(q_out_stride=512 * 64 + 2), dict(rope_dim=63), dict(rope_dim=130), dict(rope_dim=-2), dict(eps=-1.0),
    dict(eps=float("nan")), dict(rope_theta=0.0), dict(heads=0), dict(q_out=_p(1), q_out_stride=512 * 65),
    dict(kv_heads=0)])
def test_norm_rope_rejects_on_host(lib, bad):
    assert lib.dsv4_norm_rope_append(ctypes.byref(_norm(**bad)), None) == 1, bad


@pytest.mark.parametrize("bad", TABLES + QUERIES + [
    dict(v_pages=_p(10, 8)),
    dict(out=None), dict(lse=_p(8, 2)), dict(sink=_p(6, 2)), dict(out_rope_pos=_p(9, 4)), dict(out_rope_dim=0), dict(out_rope_dim=65),
    dict(out_rope_dim=130), dict(out_rope_theta=-1.0)])
def test_attention_rejects_on_host(lib, bad):
    assert lib.dsv4_paged_attn(ctypes.byref(_attn(**bad)), _p(20), 1 << 40, None) == 1, bad


@pytest.mark.parametrize("bad", TABLES + QUERIES + [dict(lse=None), dict(acc=None), dict(acc_rows=0)])
def test_weights_reject_on_host(lib, bad):
    assert lib.dsv4_paged_attn_weights(ctypes.byref(_weights(**bad)), _p(20), 1 << 40, None) == 1, bad


@pytest.mark.parametrize("bad", TABLES + [
    dict(out_table=None), dict(kv_len_out=None), dict(acc=None), dict(acc_out=_p(7, 2)), dict(keep=None), dict(out_pages=0),
    dict(out_table=_p(2), out_pages=8),             # in place: one table, one width
    dict(acc_rows=0), dict(budget=0), dict(budget=513), dict(budget=1025, out_pages=32), dict(recent=-1), dict(recent=501)])
def test_evict_rejects_on_host(lib, bad):
    assert lib.dsv4_paged_evict(ctypes.byref(_evict(**bad)), _p(20), 1 << 40, None) == 1, bad


@pytest.mark.parametrize("make, name", [(_attn, "dsv4_paged_attn"), (_weights, "dsv4_paged_attn_weights"),
                                        (_evict, "dsv4_paged_evict")])
def test_workspaces(lib, make, name):
    call, size = getattr(lib, name), getattr(lib, name + "_workspace_size")
    a = make()
    need = size(ctypes.byref(a))
    assert need > 256 and size(None) == 0
    assert call(ctypes.byref(a), _p(20), need - 1, None) == 1
    assert call(ctypes.byref(a), None, need, None) == 1
    assert call(ctypes.byref(a), _p(20, 8), need, None) == 1
    assert call(None, _p(20), need, None) == 1
    if make is not _evict:                          # lengths do not enter
        assert size(ctypes.byref(make(max_pages=1024, total_q=4000))) == need


# what enters a workspace's size, at values that the calls refuse
SIZED = [(_attn, "dsv4_paged_attn", x) for x in (
    dict(kv_heads=0), dict(kv_heads=-1), dict(heads=0), dict(heads=1025), dict(heads=6, kv_heads=4), dict(dim=64), dict(dim=0),
    dict(dim=-512), dict(max_q=0), dict(max_q=-5), dict(batch=-1), dict(batch=2049))]
SIZED += [(_weights, "dsv4_paged_attn_weights", x) for x in (dict(kv_heads=0), dict(heads=0), dict(dim=64), dict(batch=-1))]
SIZED += [(_evict, "dsv4_paged_evict", x) for x in (
    dict(batch=-1), dict(batch=2049), dict(budget=0), dict(budget=-1, recent=-2), dict(recent=-1), dict(recent=501),
    dict(acc_rows=0), dict(acc_rows=-1), dict(budget=1025), dict(budget=-(1 << 31), recent=1))]


@pytest.mark.parametrize("make, name, bad", SIZED)
def test_workspace_sizes_of_refused_counts(name, make, bad):
    """A size is asked for before the call checks its arguments: it is 0 for counts that the call refuses. In a process of
    its own, since a division by a count of 0 would end it."""
    code = (f"import sys, ctypes; sys.path[:0] = {sys.path!r}; import test_host_paged as t\n"
            f"from compressed_sparse_attention_08_gb300 import _abi\n"
            f"print(_abi.library().{name}_workspace_size(ctypes.byref(t.{make.__name__}(**{bad!r}))))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, f"ended with {r.returncode}: {r.stderr[-300:]}"
    assert r.stdout.split()[-1] == "0"


def test_binding_refuses_shapes_and_types():
    torch = pytest.importorskip("torch")
    import compressed_sparse_attention_08_gb300 as m
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    pages = torch.zeros(4, 16, 1, 128, dtype=torch.bfloat16)
    t, cu, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        m.paged_attn_args(q, q, pages, t, cu, n)
    with pytest.raises(ValueError, match="CUDA"):
        m.norm_rope_args(q, q, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="keep"):
        m.paged_evict_args(pages, t, n, torch.zeros(1, 32), torch.zeros(1, 9, dtype=torch.int32), budget=8, recent=0)


def test_a_dropped_struct_frees_its_tensors():
    """The struct holds its tensors, and nothing holds the struct: they go with it, without the cyclic collector."""
    torch = pytest.importorskip("torch")
    from compressed_sparse_attention_08_gb300 import _abi
    t = torch.zeros(4)
    held = weakref.ref(t)
    a = _abi._held(_abi.PagedAttnArgs(), t)
    del t
    assert held() is not None
    gc.disable()
    try:
        del a
        assert held() is None
    finally:
        gc.enable()


def test_a_struct_is_passed_as_it_is(lib):
    """The calls take the struct itself (what the binding hands over)."""
    a = _attn()
    assert lib.dsv4_paged_attn_workspace_size(a) == lib.dsv4_paged_attn_workspace_size(ctypes.byref(a)) > 256
    assert lib.dsv4_paged_attn(_attn(window=-1), _p(20), 1 << 40, None) == 1
    assert lib.dsv4_norm_rope_append(_norm(eps=-1.0), None) == 1


@pytest.mark.parametrize("struct, name, value", [
    ("PagedAttnArgs", "window", (1 << 32) + 5), ("PagedAttnArgs", "max_q", 1 << 31), ("PagedWeightsArgs", "window", -(1 << 31) - 1),
    ("PagedWeightsArgs", "acc_rows", (1 << 32) + 512), ("PagedEvictArgs", "recent", 1 << 32), ("NormRopeArgs", "rope_dim", (1 << 32) + 64)])
def test_counts_do_not_wrap(struct, name, value):
    """A number past 32 bits is refused, not cut to its low bits (a window of 2^32 + 5 rows is not one of 5)."""
    from compressed_sparse_attention_08_gb300 import _abi
    cls = getattr(_abi, struct)
    fields = [f for f, _ in cls._fields_]
    values = [0] * len(fields)
    for v in ((1 << 31) - 1, -(1 << 31)):
        values[fields.index(name)] = v
        assert getattr(_abi._struct(cls, *values), name) == v
    values[fields.index(name)] = value
    with pytest.raises(ValueError, match=name):
        _abi._struct(cls, *values)
    with pytest.raises(ValueError, match="fields"):
        _abi._struct(cls, *values[:-1])


def test_builders_do_not_wrap_counts(monkeypatch):
    """The same through the builders, on tensors that only stand in for device ones."""
    torch = pytest.importorskip("torch")
    from compressed_sparse_attention_08_gb300 import _abi
    monkeypatch.setattr(_abi, "_ptr", lambda t, *a, **k: None if t is None else ctypes.c_void_p(FAKE))
    monkeypatch.setattr(_abi, "_heads_ptr", lambda t, *a, **k: (None, 0) if t is None else (ctypes.c_void_p(FAKE), t.stride(0)))
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    pages = torch.zeros(4, 16, 1, 128, dtype=torch.bfloat16)
    table, cu, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    lse, acc, keep = torch.zeros(2, 8), torch.zeros(1, 32), torch.zeros(1, 8, dtype=torch.int32)
    far = (1 << 32) + 5
    assert _abi.paged_attn_args(q, q, pages, table, cu, n, window=5).window == 5
    for bad in (dict(window=far), dict(max_q=far)):
        with pytest.raises(ValueError, match="out of range"):
            _abi.paged_attn_args(q, q, pages, table, cu, n, **bad)
        with pytest.raises(ValueError, match="out of range"):
            _abi.paged_weights_args(q, lse, pages, table, cu, n, acc, **bad)
    with pytest.raises(ValueError, match="out of range"):
        _abi.paged_attn_args(q, q, pages, table, cu, n, out_rope_pos=torch.zeros(2, dtype=torch.int64), out_rope_dim=far)
    with pytest.raises(ValueError, match="out of range"):
        _abi.paged_evict_args(pages, table, n, acc, keep, budget=8, recent=1 << 32)
    with pytest.raises(ValueError, match="out of range"):
        _abi.norm_rope_args(q, q, torch.zeros(2, dtype=torch.int64), rope_dim=far)


def test_wait_fault_controls(lib):
    """The test control knows the four kernels with bounded waits on copies, and nothing between them."""
    from compressed_sparse_attention_08_gb300 import _abi
    known = [_abi.DSV4_WAIT_FAULT_NONE, _abi.DSV4_WAIT_FAULT_SCORER_STAGE, _abi.DSV4_WAIT_FAULT_ATTN_QUERY,
             _abi.DSV4_WAIT_FAULT_PAGED_ATTN, _abi.DSV4_WAIT_FAULT_PAGED_WEIGHTS]
    try:
        assert [lib.dsv4_test_wait_fault(x, 1000) for x in range(-1, 20)] == [0 if x in known else 1 for x in range(-1, 20)]
        assert all(lib.dsv4_test_wait_fault(x, 2000001) == 1 for x in known)
    finally:
        assert lib.dsv4_test_wait_fault(0, 0) == 0
