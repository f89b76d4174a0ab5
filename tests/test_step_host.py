"""A step's calls beside the attention without a GPU: struct layouts against the
header, what the C ABI and the binding refuse before any CUDA call, pins of the
host references."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import step_reference as S
from sparse_mla_decode_token_gb300 import binding as B
from sparse_mla_decode_token_gb300 import build as smla_build
from sparse_mla_decode_token_gb300 import cache as C
from sparse_mla_decode_token_gb300 import search, slots

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return B.lib()


def test_struct_layouts_match_the_header(tmp_path):
    structs = {"smla_token_slots_args": slots.SmlaTokenSlotsArgs, "smla_sparse_slots_args": slots.SmlaSparseSlotsArgs,
               "smla_beam_args": search.SmlaBeamArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{os.path.join(ROOT, "include", "smla.h")}"',
             "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'  printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "layout.c").write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(tmp_path / "layout.c"), "-o", str(tmp_path / "layout")], check=True)
    out = dict(l.split() for l in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(out[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(out[f"{name}.{f}"]) == getattr(cls, f).offset, f


def refused(status, code, needle):
    assert status == code and needle in B.smla_last_error(), B.smla_last_error()


def beam_struct():
    a = search.SmlaBeamArgs()
    a.batch, a.beams, a.vocab, a.num_out, a.dtype = 2, 4, 1000, 4, 0
    a.logits, a.scores, a.out_scores, a.out_parents, a.out_tokens = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
    a.workspace, a.workspace_bytes = 0x100000, 1 << 20
    return a


INVALID, UNSUPPORTED = B.SMLA_ERR_INVALID_ARG, B.SMLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("field,value,code,needle", [
    ("batch", -1, INVALID, "batch"),
    ("batch", 1 << 30, UNSUPPORTED, "32-bit"),
    ("beams", 0, UNSUPPORTED, "beams"),
    ("beams", 65, UNSUPPORTED, "beams"),
    ("vocab", 0, INVALID, "vocab"),
    ("num_out", 0, UNSUPPORTED, "num_out"),
    ("num_out", 65, UNSUPPORTED, "num_out"),
    ("dtype", 3, INVALID, "dtype"),
    ("dtype", -1, INVALID, "dtype"),
    ("logits_stride", 999, INVALID, "logits_stride"),
    ("logits", None, INVALID, "logits is required"),
    ("logits", 0x10001, INVALID, "logits must be 2-byte"),
    ("scores", None, INVALID, "scores is required"),
    ("scores", 0x20002, INVALID, "scores must be 4-byte"),
    ("out_scores", None, INVALID, "out_scores is required"),
    ("out_parents", 0x20002, INVALID, "out_parents must be 4-byte"),
    ("out_tokens", None, INVALID, "out_tokens is required"),
    ("out_scores", 0x20010, INVALID, "out_scores must be scores"),
    ("out_scores", 0x1fff0, INVALID, "out_scores must be scores"),
    ("error_word", 0x20002, INVALID, "error_word must be 4-byte"),
])
def test_beam_errors(lib, field, value, code, needle):
    a = beam_struct()
    setattr(a, field, value)
    refused(lib.smla_beam_select(ctypes.byref(a), None), code, needle)


def test_no_requests_is_nothing_to_do(lib):
    a = beam_struct()
    a.batch, a.logits, a.workspace = 0, None, None
    assert lib.smla_beam_select(ctypes.byref(a), None) == B.SMLA_OK
    assert lib.smla_beam_select(None, None) == INVALID
    s = sparse_struct()
    s.sum_q, s.seq_lens = 0, None
    assert lib.smla_sparse_slots(ctypes.byref(s), None) == B.SMLA_OK
    p = C.SmlaPagesArgs()
    p.rows, p.max_pages, p.page_size, p.num_pages = 0, 4, 64, 10
    assert lib.smla_pages_reorder(ctypes.byref(p), None) == B.SMLA_OK
    assert lib.smla_pages_shared_prefix(ctypes.byref(p), None, 0, None, None) == B.SMLA_OK


def token_struct():
    a = slots.SmlaTokenSlotsArgs()
    a.lens, a.new_lens, a.batch, a.max_tokens = 0x10000, 0x20000, 4, 16
    a.block_tables, a.max_pages, a.page_size = 0x30000, 4, 64
    a.cum_seq_lens_q, a.requests, a.positions, a.slots = 0x40000, 0x50000, 0x60000, 0x70000
    return a


@pytest.mark.parametrize("field,value,needle", [
    ("batch", -1, "batch"), ("max_tokens", -1, "max_tokens"), ("max_pages", 0, "max_pages"), ("page_size", 0, "page_size"),
    ("max_pages", 1 << 26, "2^31"), ("block_table_stride", 3, "stride"), ("block_tables", None, "block_tables is required"),
    ("slots", 0x70004, "8-byte"), ("lens", None, "lens is required"), ("new_lens", 0x2, "new_lens must be 4-byte"),
    ("cum_seq_lens_q", None, "cum_seq_lens_q is required"), ("requests", 0x2, "requests must be"),
    ("positions", 0x2, "positions must be"), ("cum_seq_lens_q", 0xfff0, "overlap"), ("requests", 0x2000c, "overlap"),
    ("positions", 0xffc8, "overlap"), ("error_word", 0x2, "error_word must be"),
])
def test_token_slots_errors(lib, field, value, needle):
    a = token_struct()
    setattr(a, field, value)
    refused(lib.smla_token_slots(ctypes.byref(a), None), INVALID, needle)


def sparse_struct():
    a = slots.SmlaSparseSlotsArgs()
    a.sum_q, a.batch, a.seq_lens = 8, 4, 0x10000
    a.swa_tables, a.swa_max_pages, a.swa_page_size = 0x20000, 4, 64
    a.comp_tables, a.comp_max_pages, a.comp_page_size, a.compress_ratio, a.num_selected = 0x30000, 4, 64, 4, 16
    a.selected, a.sparse_indices, a.topk_lens = 0x40000, 0x50000, 0x60000
    return a


@pytest.mark.parametrize("field,value,needle", [
    ("sum_q", -1, "sum_q"), ("sum_q", 9, "multiple of batch"), ("batch", 0, "batch"), ("swa_max_pages", 0, "swa_tables"),
    ("swa_page_size", 0, "swa_tables"), ("swa_table_stride", 3, "swa_tables"), ("comp_max_pages", 0, "comp_tables"),
    ("comp_page_size", -1, "comp_tables"), ("comp_max_pages", 1 << 26, "2^31"), ("compress_ratio", 0, "compress_ratio"),
    ("num_selected", -1, "num_selected"), ("num_selected", (1 << 30) + 1, "2^30"), ("selected_stride", 15, "selected_stride"),
    ("indices_row_stride", 143, "indices_row_stride"), ("seq_lens", None, "seq_lens is required"),
    ("swa_tables", None, "swa_tables is required"), ("comp_tables", None, "comp_tables is required"),
    ("selected", 0x2, "selected must be"), ("sparse_indices", None, "sparse_indices is required"),
    ("topk_lens", 0x2, "topk_lens must be"), ("error_word", 0x2, "error_word must be"),
    ("cum_seq_lens_q", 0x2, "cum_seq_lens_q must be"),
])
def test_sparse_slots_errors(lib, field, value, needle):
    a = sparse_struct()
    setattr(a, field, value)
    refused(lib.smla_sparse_slots(ctypes.byref(a), None), INVALID, needle)


def pages_struct():
    a = C.SmlaPagesArgs()
    a.block_tables, a.ref_counts, a.lens, a.parents, a.out_lens = 0x10000, 0x20000, 0x30000, 0x50000, 0x60000
    a.rows, a.max_pages, a.page_size, a.num_pages = 8, 4, 64, 100
    a.workspace, a.workspace_bytes = 0x100000, 256
    return a


@pytest.mark.parametrize("field,value,code,needle", [
    ("rows", -1, INVALID, "rows"), ("max_pages", 0, INVALID, "max_pages"), ("num_pages", 0, INVALID, "num_pages"),
    ("parents", None, INVALID, "parents is required"), ("out_lens", 0x30004, INVALID, "overlap"),
    ("out_lens", 0x5001c, INVALID, "parents"), ("ref_counts", None, INVALID, "ref_counts is required"), ("workspace", None, B.SMLA_ERR_WORKSPACE_TOO_SMALL, "workspace"),
    ("workspace_bytes", 127, B.SMLA_ERR_WORKSPACE_TOO_SMALL, "256 needed"), ("workspace", 0x100010, INVALID, "256-byte"),
    ("block_table_stride", 3, INVALID, "block_table_stride"),
])
def test_reorder_errors(lib, field, value, code, needle):
    a = pages_struct()
    setattr(a, field, value)
    refused(lib.smla_pages_reorder(ctypes.byref(a), None), code, needle)


def test_shared_prefix_errors(lib):
    a = pages_struct()
    refused(lib.smla_pages_shared_prefix(ctypes.byref(a), 0x1000, -1, 0x2000, None), INVALID, "num_groups")
    refused(lib.smla_pages_shared_prefix(ctypes.byref(a), None, 2, 0x2000, None), INVALID, "group_starts is required")
    refused(lib.smla_pages_shared_prefix(ctypes.byref(a), 0x1000, 2, 0x2001, None), INVALID, "prefix_lens must be")
    refused(lib.smla_pages_shared_prefix(ctypes.byref(a), 0x1000, 2, 0x1008, None), INVALID, "overlap")
    refused(lib.smla_pages_shared_prefix(ctypes.byref(a), 0x1000, 2, 0x3001c, None), INVALID, "overlap")
    a.block_tables = None
    refused(lib.smla_pages_shared_prefix(ctypes.byref(a), 0x1000, 2, 0x2000, None), INVALID, "block_tables is required")


def test_the_binding_names_what_is_wrong(lib):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    logits, scores, ws = torch.zeros(8, 100, dtype=torch.bfloat16), torch.zeros(2, 4), torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(TypeError, match="logits"):
        search.beam_select(logits.double(), scores, ws)
    with pytest.raises(ValueError, match="logits must be"):
        search.beam_select(logits[:7], scores, ws)
    with pytest.raises(ValueError, match="rows overlap"):
        search.beam_select(logits[:1].expand(8, 100), scores, ws)
    with pytest.raises(TypeError, match="finished"):
        search.beam_select(logits, scores, ws, finished=scores)
    with pytest.raises(ValueError, match="finished"):
        search.beam_select(logits, scores, ws, finished=torch.zeros(2, 3, dtype=torch.bool))
    with pytest.raises(ValueError, match="one CUDA device"):
        search.beam_select(logits, scores, ws)
    with pytest.raises(ValueError, match="one CUDA device"):
        slots.token_slots(i32(3), i32(3), i32(3, 4), max_tokens=5, page_size=64)
    with pytest.raises(ValueError, match="rows for 3"):
        slots.token_slots(i32(3), i32(3), i32(2, 4), max_tokens=5, page_size=64)
    with pytest.raises(ValueError, match="slots need"):
        slots.token_slots(i32(3), i32(3), max_tokens=5, out=slots.StepSlots(i32(4), i32(5), i32(5), torch.zeros(5).long()))
    with pytest.raises(ValueError, match="new_lens has 2"):
        slots.token_slots(i32(3), i32(2), max_tokens=5)
    with pytest.raises(ValueError, match="selected must be"):
        slots.sparse_slots(i32(3), i32(3, 4), 6, page_size=64, selected=i32(5, 8), compressed_tables=i32(3, 4))
    with pytest.raises(ValueError, match="compressed_tables"):
        slots.sparse_slots(i32(3), i32(3, 4), 6, page_size=64, selected=i32(6, 8))
    with pytest.raises(ValueError, match="sparse_indices must be"):
        slots.sparse_slots(i32(3), i32(3, 4), 6, page_size=64, sparse_indices=i32(6, 127))
    with pytest.raises(ValueError, match="one CUDA device"):
        slots.sparse_slots(i32(3), i32(3, 4), 6, page_size=64)
    with pytest.raises(ValueError, match="parents has 2"):
        C.pages_reorder(i32(3, 4), i32(9), i32(3), i32(2), i32(3), ws, page_size=64)
    with pytest.raises(ValueError, match="one CUDA device"):
        C.pages_reorder(i32(3, 4), i32(9), i32(3), i32(3), i32(3), ws, page_size=64)
    with pytest.raises(ValueError, match="group_starts has 2"):
        C.pages_shared_prefix(i32(3, 4), i32(3), i32(2), i32(2), page_size=64)


def test_beam_reference_on_worked_examples():
    logits = np.log(np.array([[0.5, 0.25, 0.25], [0.125, 0.75, 0.125]]))
    scores = np.log(np.array([[0.5, 0.5]]))
    best, rows, tokens = S.beam_best(S.beam_scores(logits, scores), 4)
    assert rows.tolist() == [[1, 0, 0, 0]] and tokens.tolist() == [[1, 0, 1, 2]]
    np.testing.assert_allclose(np.exp(best), [[0.375, 0.25, 0.125, 0.125]])
    best, rows, tokens = S.beam_best(S.beam_scores(logits, scores, np.array([[False, True]]), 2), 5)
    assert rows.tolist() == [[1, 0, 0, 0, -1]] and tokens.tolist() == [[2, 0, 1, 2, -1]]


def test_reorder_reference_keeps_counts():
    rng = np.random.default_rng(1)
    tables = rng.integers(0, 50, (6, 5)).astype(np.int32)
    lens = np.array([5, 10, 0, 3, 8, 1])
    for b, n in enumerate(lens):
        tables[b, -(-n // 2):] = -1
    refs = np.bincount(tables[tables >= 0], minlength=50)
    out, after, lengths, flag = S.reorder(tables, refs, lens, [1, 1, 0, -1, 5, 9], 2)
    assert flag and lengths.tolist() == [10, 10, 5, 0, 1, 1]
    assert np.array_equal(after, np.bincount(out[out >= 0], minlength=50))
    assert S.shared_prefix(out, lengths, [0, 2, 3, 6], 2).tolist() == [10, 4, 0]


def test_slot_references_by_hand():
    tables = np.array([[7, 2], [5, -1]])
    cum, request, position, at = S.token_slots([3, 0], [6, 2], 7, tables, 4)
    assert cum.tolist() == [0, 3, 5] and request.tolist() == [0, 0, 0, 1, 1, -1, -1]
    assert position.tolist() == [3, 4, 5, 0, 1, -1, -1] and at.tolist() == [31, 8, 9, 20, 21, -1, -1]
    out, topk = S.sparse_slots([6, 2], cum, 6, tables, 4, np.array([[1], [3]]), 8, 2, np.array([[0, 3]] * 6))
    assert out[2, :7].tolist() == [28, 29, 30, 31, 8, 9, -1] and topk.tolist() == [129, 129, 129, 128, 129, 0]
    assert out[2, 128:].tolist() == [8, -1] and out[4, 128:].tolist() == [24, -1]


def prefix_struct():
    a = C.SmlaPrefixArgs()
    a.cache.rows, a.cache.scales, a.cache.block_tables, a.cache.seq_lens = 0x10000, 0x20000, 0x30000, 0x40000
    a.cache.num_pages, a.cache.page_size, a.cache.block_rows, a.cache.max_pages, a.cache.batch = 10, 64, 16, 4, 2
    a.sum_q, a.num_heads, a.num_groups, a.group_starts, a.prefix_lens = 4, 16, 1, 0x70000, 0x80000
    a.q, a.out = 0x50000, 0x60000
    return a


@pytest.mark.parametrize("field,value,code,needle", [
    ("sum_q", -1, INVALID, "sum_q"), ("sum_q", 5, INVALID, "multiple of batch"), ("num_heads", 129, UNSUPPORTED, "num_heads"),
    ("num_groups", -1, INVALID, "num_groups"), ("group_starts", None, INVALID, "group_starts is required"),
    ("prefix_lens", 0x2, INVALID, "prefix_lens must be"), ("q", 0x50008, INVALID, "q must be 16-byte"),
    ("q_stride_token", 16 * 512 - 8, INVALID, "q_stride_token"), ("out", None, INVALID, "out is required"),
    ("out_lse", 0x2, INVALID, "out_lse must be"), ("sinks", 0x2, INVALID, "sinks must be"),
    ("error_word", 0x2, INVALID, "error_word must be"),
])
def test_prefix_errors(lib, field, value, code, needle):
    a = prefix_struct()
    setattr(a, field, value)
    refused(lib.smla_prefix_attention(ctypes.byref(a), None), code, needle)


def test_prefix_layout_and_empty_calls(lib, tmp_path):
    src = tmp_path / "layout.c"
    fields = [f for f, _ in C.SmlaPrefixArgs._fields_]
    src.write_text("\n".join(["#include <stdio.h>", "#include <stddef.h>", f'#include "{os.path.join(ROOT, "include", "smla.h")}"',
                              "int main(void) {", '  printf("%zu\\n", sizeof(smla_prefix_args));'] +
                             [f'  printf("%zu\\n", offsetof(smla_prefix_args, {f}));' for f in fields] + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [ctypes.sizeof(C.SmlaPrefixArgs)] + [getattr(C.SmlaPrefixArgs, f).offset for f in fields]
    a = prefix_struct()
    a.sum_q, a.q = 0, None
    assert lib.smla_prefix_attention(ctypes.byref(a), None) == B.SMLA_OK
    assert lib.smla_prefix_attention(None, None) == INVALID
