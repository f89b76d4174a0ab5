"""A step's calls beside the attention that are refused without a GPU: outputs that
would overwrite what other threads still read."""
import ctypes

import pytest

from sparse_mla_decode_token_gb300 import binding as B
from test_step_host import INVALID, beam_struct, lib, pages_struct, refused, sparse_struct, token_struct  # noqa: F401  (lib: the library, built once a module)

PASSED = B.SMLA_ERR_CUDA                                             # all checks passed, and there is no GPU


def sparse(fields):
    """8 tokens of 4 requests, 16 columns selected; tables of 4 columns.  Addresses in bytes."""
    a = sparse_struct()
    for k, v in fields.items():
        setattr(a, k, v)
    return a


OUT, ROW = 0x50000, 144 * 4                                          # sparse_indices and its rows
SPARSE = [
    # the selection elsewhere in the table: the front columns, one column on, a row on, other rows' strides
    dict(selected=OUT, selected_stride=144), dict(selected=OUT + 129 * 4, selected_stride=144),
    dict(selected=OUT + 127 * 4, selected_stride=144), dict(selected=OUT + ROW + 128 * 4, selected_stride=144),
    dict(selected=OUT + 128 * 4), dict(selected=OUT + 128 * 4, selected_stride=288), dict(selected=OUT - 4),
    dict(selected=OUT + 8 * ROW - 4), dict(selected=OUT + 128 * 4, selected_stride=144, indices_row_stride=160),
    # the last of a wider table's gaps is not wide enough for it
    dict(selected=OUT + 144 * 4, selected_stride=159, indices_row_stride=159),
    dict(topk_lens=0x10000), dict(topk_lens=0x10000 - 28), dict(topk_lens=0x1000c), dict(sparse_indices=0x10000),
    dict(cum_seq_lens_q=0x60000), dict(cum_seq_lens_q=0x60000 - 16), dict(cum_seq_lens_q=OUT + 4),
    dict(topk_lens=0x20000), dict(topk_lens=0x2003c), dict(sparse_indices=0x20010), dict(sparse_indices=0x30000),
    dict(swa_table_stride=100, topk_lens=0x20000 + 400), dict(topk_lens=0x3003c), dict(topk_lens=0x40000),
    dict(topk_lens=0x40000 + 8 * 64 - 4), dict(topk_lens=OUT), dict(topk_lens=OUT + 8 * ROW - 4),
    dict(indices_row_stride=150, topk_lens=OUT + 149 * 4),
]


@pytest.mark.parametrize("fields", SPARSE)
def test_sparse_slots_that_would_overwrite_what_is_read(lib, fields):
    refused(lib.smla_sparse_slots(ctypes.byref(sparse(fields)), None), INVALID, "overlap")


# 16 tokens of 4 requests, tables of 4 columns: lens 0x10000, new_lens 0x20000, tables 0x30000, outputs 0x40000 and on
TOKENS = [
    dict(slots=0x10000), dict(slots=0x10008), dict(slots=0x10000 - 120), dict(slots=0x20000 - 8), dict(slots=0x30038),
    dict(cum_seq_lens_q=0x30000 - 16), dict(requests=0x3003c), dict(positions=0x30000 - 60),
    dict(block_table_stride=10, requests=0x30000 + 160 - 28), dict(requests=0x60000), dict(positions=0x70000),
    dict(requests=0x70000 + 124), dict(slots=0x40008), dict(cum_seq_lens_q=0x6003c),
]


@pytest.mark.parametrize("fields", TOKENS)
def test_token_slots_that_would_overwrite_what_is_read(lib, fields):
    a = token_struct()
    for k, v in fields.items():
        setattr(a, k, v)
    refused(lib.smla_token_slots(ctypes.byref(a), None), INVALID, "overlap")


@pytest.mark.parametrize("fields", [
    {}, dict(slots=0x10010), dict(slots=0x10000 - 128), dict(cum_seq_lens_q=0x30000 - 20), dict(requests=0x30040),
    dict(slots=None, requests=0x30000), dict(requests=None, positions=None), dict(max_tokens=0, requests=0x10000),
    dict(batch=0, slots=0x10000),
])
def test_token_slots_beside_one_another_pass(lib, fields):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are none of a GPU's")
    a = token_struct()
    for k, v in fields.items():
        setattr(a, k, v)
    assert lib.smla_token_slots(ctypes.byref(a), None) == PASSED, B.smla_last_error()


@pytest.mark.parametrize("fields", [
    {},
    dict(selected=OUT + 128 * 4, selected_stride=144), dict(selected=OUT + 128 * 4, selected_stride=200, indices_row_stride=200),
    dict(selected=OUT + 128 * 4, sum_q=1, batch=1), dict(selected=OUT + 144 * 4, selected_stride=160, indices_row_stride=160),
    dict(selected=OUT + 8 * ROW), dict(selected=OUT - 8 * 64), dict(selected=None), dict(topk_lens=0x10010),
    dict(topk_lens=0x10000 - 32), dict(cum_seq_lens_q=0x60020), dict(num_selected=0, comp_tables=OUT, selected=OUT),
    dict(swa_table_stride=100, topk_lens=0x20000 + 16), dict(indices_row_stride=152, topk_lens=OUT + 144 * 4),
])
def test_sparse_slots_beside_one_another_pass(lib, fields):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are none of a GPU's")
    assert lib.smla_sparse_slots(ctypes.byref(sparse(fields)), None) == PASSED, B.smla_last_error()


# 2 requests of 4 beams over 1000 BF16 logits: logits 0x10000 to 0x13e80, scores 0x20000, outputs of 32 bytes from 0x30000 on
BEAMS = [
    dict(out_parents=0x20000), dict(out_parents=0x2001c), dict(out_tokens=0x20000 - 28), dict(out_scores=0x20000, out_tokens=0x20004),
    dict(finished=0x30000), dict(finished=0x4001f), dict(finished=0x50000 - 4), dict(out_tokens=0x10000), dict(out_parents=0x13e7c),
    dict(out_scores=0x13000), dict(logits_stride=1002, out_tokens=0x10000 + 7 * 2004 + 1996), dict(logits_stride=1008, out_parents=0x10000 + 2008),
    dict(out_parents=0x30000), dict(out_tokens=0x4001c), dict(out_scores=0x50000), dict(out_scores=0x20000, num_out=3),
]


@pytest.mark.parametrize("fields", BEAMS)
def test_beam_outputs_that_would_overwrite_what_is_read(lib, fields):
    a = beam_struct()
    for k, v in fields.items():
        setattr(a, k, v)
    refused(lib.smla_beam_select(ctypes.byref(a), None), INVALID, "overlap")


@pytest.mark.parametrize("fields", [
    {}, dict(out_scores=0x20000), dict(out_parents=0x20020), dict(out_tokens=0x20000 - 32), dict(finished=0x30020),
    dict(finished=0x50000 - 8), dict(out_parents=0x13e80), dict(logits_stride=1020, out_parents=0x10000 + 2004), dict(num_out=3),
])
def test_beam_outputs_beside_one_another_pass(lib, fields):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are none of a GPU's")
    a = beam_struct()
    for k, v in fields.items():
        setattr(a, k, v)
    assert lib.smla_beam_select(ctypes.byref(a), None) == PASSED, B.smla_last_error()


@pytest.mark.parametrize("fields", [
    dict(out_lens=0x10000), dict(out_lens=0x1007c), dict(out_lens=0x20000 - 28), dict(out_lens=0x20000 + 396),
    dict(block_table_stride=100, out_lens=0x10000 + 2800),
])
def test_reordered_lengths_over_tables_or_counts(lib, fields):
    """8 requests of 4 columns: tables 0x10000, 100 counts 0x20000."""
    a = pages_struct()
    for k, v in fields.items():
        setattr(a, k, v)
    refused(lib.smla_pages_reorder(ctypes.byref(a), None), INVALID, "out_lens")


def test_shared_prefixes_over_the_tables(lib):
    a = pages_struct()
    for at in (0x10000, 0x1007c, 0x10000 - 4):
        refused(lib.smla_pages_shared_prefix(ctypes.byref(a), 0x1000, 2, at, None), INVALID, "overlap")
    a.block_table_stride = 100
    refused(lib.smla_pages_shared_prefix(ctypes.byref(a), 0x1000, 2, 0x10000 + 396, None), INVALID, "overlap")


def test_logits_of_more_bytes_than_a_number_holds(lib):
    """2^31 rows of 2^31 fp32 logits: too many, whatever lies where; from the first one on they hold all that is behind."""
    a = beam_struct()
    a.batch, a.beams, a.vocab, a.dtype, a.num_out = (1 << 25) - 1, 64, (1 << 31) - 1, 2, 1
    a.out_scores, a.out_parents, a.out_tokens, a.scores = 1 << 40, 1 << 41, 1 << 42, 1 << 43
    refused(lib.smla_beam_select(ctypes.byref(a), None), INVALID, "overlap")
    a.logits, a.logits_stride = 0x10000, (1 << 61) - 1               # rows so far apart that all lies behind the first
    a.out_tokens = 0x10000 + (1 << 33) - 8
    refused(lib.smla_beam_select(ctypes.byref(a), None), INVALID, "overlap")
