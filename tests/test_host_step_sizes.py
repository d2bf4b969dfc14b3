"""CPU-only: the workspace of the shared-prefix attention is what the header says, magnitudes that fp32 does not hold are refused."""
from __future__ import annotations

import ctypes

import pytest

from test_host_step import _prefix, _rope, lib  # noqa: F401


@pytest.mark.parametrize("dim", [128, 256, 512])
@pytest.mark.parametrize("groups, total_q, heads", [(1, 1, 8), (2048, 1, 8), (7, 1000, 64)])
def test_prefix_workspace_is_as_described(lib, dim, groups, total_q, heads):  # noqa: F811
    a = _prefix(dim=dim, groups=groups, total_q=total_q, heads=heads, kv_heads=1, q_stride=dim * heads)
    size = lib.dsv4_paged_prefix_attn_workspace_size(ctypes.byref(a))
    per_sm = 128 * (min(dim, 256) + 2) * 4 * (2 if dim == 128 else 1) + groups * 4
    most = 2 * total_q * heads * (dim + 8) * 4 + 160 * per_sm + 4096       # (the header, the error words, alignment)
    assert most - 2 * total_q * heads * 8 * 4 - 8 * per_sm - 8192 <= size <= most     # 152 SMs or more


@pytest.mark.parametrize("magnitude", [1e39, -1e39, 1.8e308])
def test_rope_refuses_magnitudes_past_fp32(lib, magnitude):  # noqa: F811
    """The products are in fp32: such a factor would be an infinity there."""
    assert lib.dsv4_rope(ctypes.byref(_rope(magnitude=magnitude)), None) == 1
