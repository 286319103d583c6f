"""Struct layouts and refusals of dsa_batch_plan, dsa_qk_norm_rope, dsa_block_pool, dsa_block_scores
and dsa_block_select: every bad argument is answered before any CUDA call, so this needs no GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, 1, 2
PTR = 0x10000


@pytest.mark.parametrize("ctype,mirror", [("dsa_plan_args_t", dsa.DsaPlanArgs), ("dsa_qk_args_t", dsa.DsaQkArgs)])
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


def _plan():
    a = dsa.DsaPlanArgs()
    for name in ("lengths", "new_tokens", "held", "block_table", "free_pages", "num_free", "lengths_out", "held_out",
                 "num_free_out", "cu_tokens", "req_of_token", "positions", "token_lengths", "out_loc"):
        setattr(a, name, PTR)
    a.num_requests, a.bt_stride, a.page_size, a.max_pages, a.free_capacity, a.T = 4, 10, 64, 10, 100, 8
    return a


@pytest.mark.parametrize("field,value,want", [
    ("num_requests", -1, INVALID), ("num_requests", (1 << 20) + 1, UNSUPPORTED), ("T", -1, INVALID),
    ("T", (1 << 30) + 1, UNSUPPORTED), ("free_capacity", -1, INVALID), ("free_capacity", 1 << 31, UNSUPPORTED),
    ("page_size", 0, INVALID), ("page_size", -64, INVALID), ("max_pages", -1, INVALID), ("max_pages", 11, INVALID),
    ("out_loc", PTR + 4, INVALID), ("positions", PTR + 2, INVALID), ("error_word", PTR + 1, INVALID)] + [
    (n, 0, INVALID) for n in ("lengths", "new_tokens", "held", "block_table", "free_pages", "num_free", "lengths_out",
                              "held_out", "num_free_out", "cu_tokens", "req_of_token", "positions", "token_lengths",
                              "out_loc")])
def test_plan_refusals(dsa_lib, field, value, want):
    a = _plan()
    setattr(a, field, value)
    assert dsa_lib.dsa_batch_plan(ctypes.byref(a), None) == want


def _qk():
    a = dsa.DsaQkArgs()
    a.T, a.d_nope, a.d_rope, a.H, a.eps = 4, 512, 64, 16, 1e-6
    a.q = a.q_out = a.k = a.cache = a.out_loc = a.positions = a.cos_sin = a.q_weight = a.k_weight = PTR
    a.q_out = PTR + (1 << 20)
    a.q_stride_t = a.q_out_stride_t = 16 * 576
    a.q_stride_h = a.q_out_stride_h = a.k_stride_t = 576
    a.kind, a.num_slots, a.cs_stride, a.num_positions, a.q_norm, a.k_norm = dsa.CACHE_FP8_SCALED, 64, 64, 100, 576, 512
    return a


@pytest.mark.parametrize("field,value,want", [
    ("T", -1, INVALID), ("T", (1 << 24) + 1, UNSUPPORTED), ("d_nope", 256, UNSUPPORTED), ("d_rope", 0, UNSUPPORTED),
    ("H", 0, INVALID), ("H", 129, UNSUPPORTED), ("eps", 0.0, INVALID), ("eps", -1.0, INVALID),
    ("eps", float("nan"), INVALID), ("eps", float("inf"), INVALID), ("q", PTR + 8, INVALID), ("q_out", 0, INVALID),
    ("q_out", PTR + 8, INVALID), ("q_weight", PTR + 8, INVALID), ("k_weight", PTR + 2, INVALID), ("q_norm", 64, INVALID),
    ("k_norm", 577, INVALID), ("q_norm", -1, INVALID), ("q_stride_t", -8, INVALID), ("q_stride_h", 577, INVALID),
    ("q_out_stride_h", 568, INVALID), ("q_out_stride_t", 576, INVALID), ("q_out_stride_t", 16 * 576 - 8, INVALID),
    ("q_out", PTR, OK), ("k", PTR + 2, INVALID), ("k_stride_t", 570, INVALID), ("k_stride_t", -576, INVALID),
    ("kind", 2, INVALID), ("cache", 0, INVALID), ("cache", PTR + 8, INVALID), ("num_slots", -1, INVALID),
    ("out_loc", PTR + 4, INVALID), ("positions", 0, INVALID), ("positions", PTR + 2, INVALID), ("cs_stride", 63, INVALID),
    ("num_positions", -1, INVALID), ("cos_sin", PTR + 2, INVALID)])
def test_qk_refusals(dsa_lib, field, value, want):
    a = _qk()
    setattr(a, field, value)
    if want == OK:  # in place wants equal strides
        a.q_stride_t, want = 17 * 576, INVALID
    assert dsa_lib.dsa_qk_norm_rope(ctypes.byref(a), None) == want


def test_qk_more_refusals(dsa_lib):
    a = _qk()
    a.q = a.k = 0
    assert dsa_lib.dsa_qk_norm_rope(ctypes.byref(a), None) == INVALID
    a.T = 0
    assert dsa_lib.dsa_qk_norm_rope(ctypes.byref(a), None) == OK
    a = _qk()  # no rotation without RoPE columns
    a.d_nope, a.d_rope, a.q_norm, a.k_norm = 256, 0, 256, 0
    assert dsa_lib.dsa_qk_norm_rope(ctypes.byref(a), None) == INVALID
    assert dsa_lib.dsa_qk_norm_rope(None, None) == INVALID


POOL = dict(cache=PTR, kind=1, num_slots=640, block_table=PTR, bt_stride=10, page_size=64, max_pages=10, num_requests=4,
            positions=PTR, req=None, T=4, lengths=PTR, summary=PTR, num_pages=10, err=None, stream=None)


@pytest.mark.parametrize("field,value,want", [
    ("kind", 2, INVALID), ("T", -1, INVALID), ("T", (1 << 24) + 1, UNSUPPORTED), ("T", 5, INVALID), ("T", 0, OK),
    ("page_size", 0, INVALID), ("max_pages", -1, INVALID), ("max_pages", 11, INVALID), ("num_slots", -1, INVALID),
    ("num_slots", 1 << 31, UNSUPPORTED), ("num_pages", -1, INVALID), ("num_requests", 0, INVALID), ("cache", None, INVALID),
    ("cache", PTR + 8, INVALID), ("block_table", None, INVALID), ("positions", None, INVALID), ("lengths", None, INVALID),
    ("summary", None, INVALID), ("summary", PTR + 8, INVALID), ("req", PTR + 2, INVALID), ("err", PTR + 2, INVALID)])
def test_pool_refusals(dsa_lib, field, value, want):
    a = dict(POOL)
    a[field] = value
    assert dsa_lib.dsa_block_pool(*a.values()) == want


SCORES = dict(q=PTR, q_st=64 * 256, q_sh=256, T=4, H=64, summary=PTR, num_pages=10, block_table=PTR, bt_stride=10,
              page_size=64, max_pages=10, num_requests=4, req=None, lengths=PTR, scale=0.0625, weights=None, scores=PTR,
              score_stride=10, width=10, err=None, stream=None)


@pytest.mark.parametrize("field,value,want", [
    ("T", -1, INVALID), ("T", (1 << 24) + 1, UNSUPPORTED), ("T", 5, INVALID), ("T", 0, OK), ("H", 0, INVALID),
    ("H", 129, UNSUPPORTED), ("q", None, INVALID), ("q", PTR + 8, INVALID), ("q_st", 100, INVALID), ("q_st", -256, INVALID),
    ("q_sh", 257, INVALID), ("q_sh", -8, INVALID), ("summary", None, INVALID), ("summary", PTR + 8, INVALID),
    ("num_pages", -1, INVALID), ("block_table", None, INVALID), ("bt_stride", 9, INVALID), ("page_size", 0, INVALID),
    ("max_pages", -1, INVALID), ("num_requests", 0, INVALID), ("lengths", None, INVALID), ("scale", 0.0, INVALID),
    ("scale", -1.0, INVALID), ("scale", float("nan"), INVALID), ("scale", float("inf"), INVALID),
    ("weights", PTR + 2, INVALID), ("scores", None, INVALID), ("score_stride", 9, INVALID), ("width", 0, INVALID),
    ("lengths", PTR + 1, INVALID)])
def test_scores_refusals(dsa_lib, field, value, want):
    a = dict(SCORES)
    a[field] = value
    assert dsa_lib.dsa_block_scores(*a.values()) == want


def test_scores_width_limit(dsa_lib):
    a = dict(SCORES, width=(1 << 24) + 1, score_stride=(1 << 24) + 1)
    assert dsa_lib.dsa_block_scores(*a.values()) == UNSUPPORTED


SELECT = dict(scores=PTR, score_stride=10, width=10, T=4, block_table=PTR, bt_stride=10, page_size=64, max_pages=10,
              num_requests=4, req=None, lengths=PTR, K=4, sink=1, recent=2, blocks=PTR, blocks_stride=4, table=PTR,
              table_stride=4, lengths_out=PTR, err=None, stream=None)


@pytest.mark.parametrize("field,value,want", [
    ("T", -1, INVALID), ("T", (1 << 24) + 1, UNSUPPORTED), ("T", 5, INVALID), ("T", 0, OK), ("scores", None, INVALID),
    ("score_stride", 9, INVALID), ("width", 0, INVALID), ("block_table", None, INVALID), ("bt_stride", 9, INVALID),
    ("page_size", 0, INVALID), ("max_pages", -1, INVALID), ("num_requests", 0, INVALID), ("lengths", None, INVALID),
    ("K", 0, INVALID), ("K", 2, INVALID), ("sink", -1, INVALID), ("sink", 3, INVALID), ("recent", -1, INVALID),
    ("recent", (1 << 31) - 1, INVALID), ("blocks_stride", 3, INVALID), ("table", None, INVALID),
    ("table_stride", 3, INVALID), ("lengths_out", None, INVALID), ("scores", PTR + 2, INVALID), ("err", PTR + 3, INVALID)])
def test_select_refusals(dsa_lib, field, value, want):
    a = dict(SELECT)
    a[field] = value
    assert dsa_lib.dsa_block_select(*a.values()) == want


def test_select_limits(dsa_lib):
    a = dict(SELECT, K=16385, blocks_stride=16385, table_stride=16385)
    assert dsa_lib.dsa_block_select(*a.values()) == UNSUPPORTED
    a = dict(SELECT, width=(1 << 24) + 1, score_stride=(1 << 24) + 1)
    assert dsa_lib.dsa_block_select(*a.values()) == UNSUPPORTED


def test_binding_wants_cuda_tensors(dsa_lib):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.dsa_batch_plan(i, i, i, torch.zeros((4, 2), dtype=torch.int32), i, i[:1], 4, page_size=64)
    with pytest.raises(ValueError):
        dsa.dsa_qk_norm_rope(torch.zeros((1, 1, 256), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        dsa.dsa_qk_norm_rope()
    with pytest.raises(ValueError):
        dsa.dsa_block_pool(torch.zeros((64, 264), dtype=torch.uint8), dsa.CACHE_FP8_SCALED, i, i, i, i, page_size=64)
    with pytest.raises(ValueError):
        dsa.dsa_block_scores(torch.zeros((1, 1, 256), dtype=torch.bfloat16), i, i, i, 1.0, page_size=64)
    with pytest.raises(ValueError):
        dsa.dsa_block_select(torch.zeros((1, 1)), i, i, 1, page_size=64)
    with pytest.raises(ValueError):
        dsa.dsa_block_select(torch.zeros((1, 1)), i, i, 1 << 32, page_size=64)
