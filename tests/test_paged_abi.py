"""Struct layouts and refusals of dsa_paged_attn, dsa_paged_attn_mass and dsa_cache_evict: every
bad argument is answered before any CUDA call, so this needs no GPU."""
import ctypes
import os
import subprocess

import pytest

import dsa_sparse_attention_mla_gb300 as dsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
PTR = 0x10000


@pytest.mark.parametrize("ctype,mirror", [("dsa_paged_args_t", dsa.DsaPagedArgs), ("dsa_evict_args_t", dsa.DsaEvictArgs)])
def test_struct_layout_matches_header(tmp_path, ctype, mirror):
    fields = [f[0] for f in mirror._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dsa.h"\nint main(void){\n'
                   f'printf("%zu\\n", sizeof({ctype}));\n' +
                   "".join(f'printf("%zu\\n", offsetof({ctype}, {f}));\n' for f in fields) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(mirror)
    assert vals[1:] == [getattr(mirror, f).offset for f in fields]


def _paged():
    a = dsa.DsaPagedArgs()
    a.q = a.cache = a.block_table = a.lengths = a.out = a.workspace = PTR
    a.T, a.H, a.kind, a.num_slots = 4, 64, dsa.CACHE_FP8_SCALED, 640
    a.q_stride_t, a.q_stride_h = 64 * 256, 256
    a.out_stride_t, a.out_stride_h = 64 * 256, 256
    a.d_nope, a.d_rope, a.d_v = 256, 0, 256
    a.bt_stride, a.page_size, a.max_pages, a.num_requests = 10, 64, 10, 4
    a.sm_scale = 1 / 16
    a.workspace_bytes = 0
    return a


PAGED_BAD = [
    ("kind", 2, INVALID), ("T", -1, INVALID), ("H", 0, INVALID), ("H", 129, UNSUPPORTED), ("T", (1 << 24) + 1, UNSUPPORTED),
    ("d_nope", 512, UNSUPPORTED), ("d_rope", 64, UNSUPPORTED), ("d_v", 128, UNSUPPORTED),
    ("q", 0, INVALID), ("q", PTR + 8, INVALID), ("cache", 0, INVALID), ("cache", PTR + 8, INVALID), ("lengths", 0, INVALID),
    ("num_slots", -1, INVALID), ("num_requests", 0, INVALID), ("num_requests", 3, INVALID),
    ("q_stride_t", 64 * 256 + 4, INVALID), ("q_stride_h", 257, INVALID), ("q_stride_t", -8, INVALID),
    ("page_size", 0, INVALID), ("max_pages", -1, INVALID), ("max_pages", 11, INVALID),
    ("sm_scale", float("nan"), INVALID), ("sm_scale", float("inf"), INVALID),
    ("logit_cap", -1.0, INVALID), ("logit_cap", float("inf"), INVALID), ("logit_cap", float("nan"), INVALID),
]


@pytest.mark.parametrize("field,value,want", PAGED_BAD + [
    ("out", 0, INVALID), ("out", PTR + 2, INVALID), ("out_stride_h", 248, INVALID), ("out_stride_t", 64, INVALID),
    ("out_stride_h", 260, INVALID)])
def test_paged_attn_refusals(dsa_lib, field, value, want):
    a = _paged()
    setattr(a, field, value)
    assert dsa_lib.dsa_paged_attn(ctypes.byref(a), None) == want


@pytest.mark.parametrize("field,value,want", PAGED_BAD + [("lse", 0, INVALID)])
def test_paged_mass_refusals(dsa_lib, field, value, want):
    a = _paged()
    a.lse = PTR
    setattr(a, field, value)
    assert dsa_lib.dsa_paged_attn_mass(ctypes.byref(a), PTR, 640, PTR, 640, 640, None) == want


def test_paged_more_refusals(dsa_lib):
    L = dsa_lib
    a = _paged()
    a.key_positions, a.kp_stride, a.kp_width = PTR, 9, 10
    assert L.dsa_paged_attn(ctypes.byref(a), None) == INVALID
    assert L.dsa_paged_attn(None, None) == INVALID
    a = _paged()
    a.lse = PTR
    assert L.dsa_paged_attn_mass(ctypes.byref(a), None, 640, PTR, 640, 640, None) == INVALID
    assert L.dsa_paged_attn_mass(ctypes.byref(a), PTR, 640, None, 640, 640, None) == INVALID
    assert L.dsa_paged_attn_mass(ctypes.byref(a), PTR, 639, PTR, 640, 640, None) == INVALID
    assert L.dsa_paged_attn_mass(ctypes.byref(a), PTR, 640, PTR, 639, 640, None) == INVALID
    assert L.dsa_paged_attn_mass(ctypes.byref(a), PTR, 640, PTR, 640, -1, None) == INVALID
    # in place means the same rows
    assert L.dsa_paged_attn_mass(ctypes.byref(a), PTR, 640, PTR, 648, 640, None) == INVALID
    # rows' costs that do not fit 31 bits; the mass's rows bound them too
    b = _paged()
    b.T = b.num_requests = 1 << 24
    b.bt_stride = b.max_pages = 1000
    b.lse = PTR
    assert L.dsa_paged_attn(ctypes.byref(b), None) == UNSUPPORTED
    assert L.dsa_paged_attn_mass(ctypes.byref(b), PTR, 64000, PTR, 64000, 64000, None) == UNSUPPORTED
    b.num_slots = 1 << 31
    assert L.dsa_paged_attn(ctypes.byref(b), None) == UNSUPPORTED
    a.T = 0
    assert L.dsa_paged_attn(ctypes.byref(a), None) == OK
    n = ctypes.c_size_t(0)
    assert L.dsa_paged_attn_workspace_size(None, ctypes.byref(n)) == INVALID
    assert L.dsa_paged_attn_workspace_size(ctypes.byref(a), None) == INVALID


def _evict():
    a = dsa.DsaEvictArgs()
    a.cache = a.block_table = a.lengths = a.mass = a.mass_out = a.lengths_out = a.workspace = PTR
    a.kind, a.num_slots, a.d_nope, a.d_rope = dsa.CACHE_FP8_SCALED, 640, 256, 0
    a.bt_stride, a.page_size, a.max_pages, a.num_requests = 10, 64, 10, 4
    a.budget, a.width = 128, 640
    a.mass_stride = a.mass_out_stride = 640
    a.workspace_bytes = dsa.dsa_cache_evict_workspace_size(4, 640)
    return a


@pytest.mark.parametrize("field,value,want", [
    ("kind", 5, INVALID), ("d_nope", 384, UNSUPPORTED), ("d_rope", 64, UNSUPPORTED), ("num_requests", -1, INVALID),
    ("cache", 0, INVALID), ("cache", PTR + 4, INVALID), ("num_slots", -1, INVALID), ("lengths", 0, INVALID),
    ("mass", 0, INVALID), ("mass_out", 0, INVALID), ("lengths_out", 0, INVALID), ("page_size", 0, INVALID),
    ("max_pages", 11, INVALID), ("block_table", 0, INVALID), ("sink", -1, INVALID), ("recent", -1, INVALID),
    ("budget", -1, INVALID), ("width", 0, INVALID), ("width", (1 << 30) + 1, INVALID), ("mass_stride", 639, INVALID),
    ("mass_out_stride", 639, INVALID), ("mass_out_stride", 648, INVALID), ("workspace", 0, INVALID),
    ("workspace", PTR + 4, INVALID), ("workspace_bytes", 100, SMALL), ("num_requests", 0, OK),
    ("num_requests", 65536, UNSUPPORTED)])
def test_evict_refusals(dsa_lib, field, value, want):
    a = _evict()
    setattr(a, field, value)
    assert dsa_lib.dsa_cache_evict(ctypes.byref(a), None) == want


def test_evict_positions_refusals(dsa_lib):
    for fields in ({"positions": PTR, "positions_stride": 640}, {"positions": PTR, "positions_stride": 639,
                   "positions_out": 2 * PTR, "positions_out_stride": 640},
                   {"positions": PTR, "positions_stride": 640, "positions_out": PTR, "positions_out_stride": 641},
                   {"positions_out": PTR, "positions_out_stride": 639}):
        a = _evict()
        for k, v in fields.items():
            setattr(a, k, v)
        assert dsa_lib.dsa_cache_evict(ctypes.byref(a), None) == INVALID, fields
    assert dsa_lib.dsa_cache_evict(None, None) == INVALID
    n = ctypes.c_size_t(0)
    assert dsa_lib.dsa_cache_evict_workspace_size(-1, 10, ctypes.byref(n)) == INVALID
    assert dsa_lib.dsa_cache_evict_workspace_size(1, 0, ctypes.byref(n)) == INVALID
    assert dsa_lib.dsa_cache_evict_workspace_size(1, 10, None) == INVALID


def test_binding_refusals():
    """The binding's own checks come before the library's and need no GPU either."""
    import torch

    q = torch.zeros((2, 4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_paged_attn(q, q[0], dsa.CACHE_BF16, None, torch.zeros(2, dtype=torch.int32), 1.0)
    with pytest.raises(ValueError, match="lse"):
        dsa.dsa_paged_attn_mass(q, q[0], dsa.CACHE_BF16, None, None, 1.0, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_cache_evict(torch.zeros((64, 264), dtype=torch.uint8), dsa.CACHE_FP8_SCALED, None,
                            torch.zeros(1, dtype=torch.int32), torch.zeros((1, 64)), 8)


@pytest.mark.parametrize("value", [1 << 31, 1 << 32, -(1 << 31) - 1])
@pytest.mark.parametrize("name", ["budget", "sink", "recent", "page_size"])
def test_binding_refuses_integers_that_would_wrap(name, value):
    """2**32 as a budget would arrive as 0 and evict everything."""
    import torch

    args = (torch.zeros((64, 264), dtype=torch.uint8), dsa.CACHE_FP8_SCALED, None, torch.zeros(1, dtype=torch.int32),
            torch.zeros((1, 64)))
    with pytest.raises(ValueError, match=f"{name} must fit 32 bits"):
        dsa.dsa_cache_evict(*args, **{name: value})
    if name == "page_size":
        q = torch.zeros((2, 4, 256), dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="page_size must fit 32 bits"):
            dsa.dsa_paged_attn(q, q[0], dsa.CACHE_BF16, None, torch.zeros(2, dtype=torch.int32), 1.0, page_size=value)


def test_evict_needs_one_budget():
    """Without a budget nothing says what may go (0 would evict every position); with both, which holds?"""
    import torch

    args = (torch.zeros((64, 264), dtype=torch.uint8), dsa.CACHE_FP8_SCALED, None, torch.zeros(1, dtype=torch.int32),
            torch.zeros((1, 64)))
    budgets = torch.zeros(1, dtype=torch.int32)
    for kw in ({}, {"budget": None}, {"budget": 8, "budgets": budgets}, {"budget": 0, "budgets": budgets}):
        with pytest.raises(ValueError, match="one of budget and budgets"):
            dsa.dsa_cache_evict(*args, **kw)
    # either alone gets as far as the device check
    for kw in ({"budget": 0}, {"budgets": budgets}):
        with pytest.raises(ValueError, match="CUDA"):
            dsa.dsa_cache_evict(*args, **kw)
