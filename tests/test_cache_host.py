"""The paged latent cache without a GPU: struct layouts against the header, what
the C ABI and the binding refuse before any CUDA call, and pins of the host
reference that the GPU tests compare with."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import cache_reference as R
from sparse_mla_decode_token_gb300 import binding as B
from sparse_mla_decode_token_gb300 import build as smla_build
from sparse_mla_decode_token_gb300 import cache as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return B.lib()


def test_struct_layouts_match_the_header(tmp_path):
    structs = {"smla_cache": C.SmlaCache, "smla_window_args": C.SmlaWindowArgs, "smla_append_args": C.SmlaAppendArgs,
               "smla_pages_args": C.SmlaPagesArgs, "smla_pool": C.SmlaPool}
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{os.path.join(ROOT, "include", "smla.h")}"',
             "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'  printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(src), "-o", str(tmp_path / "layout")], check=True)
    out = dict(l.split() for l in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(out[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(out[f"{name}.{f}"]) == getattr(cls, f).offset, f


def cache_struct():
    """Pointers are markers: host checks never follow them."""
    c = C.SmlaCache()
    c.rows, c.scales, c.block_tables, c.seq_lens = 0x10000, 0x20000, 0x30000, 0x40000
    c.num_pages, c.page_size, c.block_rows, c.max_pages, c.batch = 10, 64, 16, 4, 2
    return c


def window_struct():
    a = C.SmlaWindowArgs()
    a.cache = cache_struct()
    a.sum_q, a.num_heads, a.window = 4, 64, 128
    a.q, a.out = 0x50000, 0x60000
    return a


def append_struct():
    a = C.SmlaAppendArgs()
    a.cache, a.sum_q, a.latent = cache_struct(), 4, 0x50000
    return a


def pages_struct():
    a = C.SmlaPagesArgs()
    a.block_tables, a.ref_counts, a.lens, a.new_lens = 0x10000, 0x20000, 0x30000, 0x40000
    a.parents, a.out_lens = 0x50000, 0x60000
    a.move_src, a.move_dst, a.move_count, a.move_capacity = 0x70000, 0x80000, 0x90000, 64
    a.rows, a.max_pages, a.page_size, a.num_pages = 8, 4, 64, 100
    a.workspace, a.workspace_bytes = 0x100000, 1 << 20
    return a


def refused(status, code, needle):
    assert status == code and needle in B.smla_last_error(), B.smla_last_error()


CACHE_ERRORS = [
    ("batch", 0, B.SMLA_ERR_INVALID_ARG, "batch"),
    ("num_pages", 0, B.SMLA_ERR_INVALID_ARG, "num_pages"),
    ("num_pages", 1 << 31, B.SMLA_ERR_INVALID_ARG, "num_pages"),
    ("page_size", 12, B.SMLA_ERR_INVALID_ARG, "page_size"),
    ("page_size", 0, B.SMLA_ERR_INVALID_ARG, "page_size"),
    ("page_size", 1 << 21, B.SMLA_ERR_INVALID_ARG, "page_size"),
    ("block_rows", 0, B.SMLA_ERR_INVALID_ARG, "block_rows"),
    ("block_rows", 24, B.SMLA_ERR_INVALID_ARG, "block_rows"),
    ("max_pages", 0, B.SMLA_ERR_INVALID_ARG, "max_pages"),
    ("max_pages", 1 << 25, B.SMLA_ERR_INVALID_ARG, "max_pages"),
    ("row_stride", 500, B.SMLA_ERR_INVALID_ARG, "row_stride"),
    ("row_stride", 520, B.SMLA_ERR_INVALID_ARG, "row_stride"),
    ("page_stride", 64 * 512 - 16, B.SMLA_ERR_INVALID_ARG, "page_stride"),
    ("page_stride", 64 * 512 + 8, B.SMLA_ERR_INVALID_ARG, "page_stride"),
    ("page_stride", 1 << 40, B.SMLA_ERR_UNSUPPORTED, "page_stride"),
    ("scale_stride", 3, B.SMLA_ERR_INVALID_ARG, "scale_stride"),
    ("block_table_stride", 3, B.SMLA_ERR_INVALID_ARG, "block_table_stride"),
    ("rows", None, B.SMLA_ERR_INVALID_ARG, "rows is required"),
    ("rows", 0x10008, B.SMLA_ERR_INVALID_ARG, "rows must be 16-byte"),
    ("scales", 0x20002, B.SMLA_ERR_INVALID_ARG, "scales must be 4-byte"),
    ("block_tables", None, B.SMLA_ERR_INVALID_ARG, "block_tables is required"),
    ("seq_lens", None, B.SMLA_ERR_INVALID_ARG, "seq_lens is required"),
    ("cum_seq_lens_q", 0x30001, B.SMLA_ERR_INVALID_ARG, "cum_seq_lens_q must be 4-byte"),
]


@pytest.mark.parametrize("field,value,code,needle", CACHE_ERRORS)
@pytest.mark.parametrize("call", ["window", "append"])
def test_cache_errors(lib, call, field, value, code, needle):
    a = window_struct() if call == "window" else append_struct()
    setattr(a.cache, field, value)
    f = lib.smla_window_attention if call == "window" else lib.smla_cache_append
    refused(f(ctypes.byref(a), None), code, needle)


@pytest.mark.parametrize("field,value,code,needle", [
    ("sum_q", -1, B.SMLA_ERR_INVALID_ARG, "sum_q"),
    ("sum_q", 5, B.SMLA_ERR_INVALID_ARG, "multiple of batch"),
    ("num_heads", 0, B.SMLA_ERR_UNSUPPORTED, "num_heads"),
    ("num_heads", 129, B.SMLA_ERR_UNSUPPORTED, "num_heads"),
    ("window", 0, B.SMLA_ERR_INVALID_ARG, "window"),
    ("first_tokens", -1, B.SMLA_ERR_INVALID_ARG, "first_tokens"),
    ("num_splits", 65, B.SMLA_ERR_INVALID_ARG, "num_splits"),
    ("num_splits", -1, B.SMLA_ERR_INVALID_ARG, "num_splits"),
    ("q_stride_token", 64 * 512 - 8, B.SMLA_ERR_INVALID_ARG, "q_stride_token"),
    ("q_stride_token", 64 * 512 + 4, B.SMLA_ERR_INVALID_ARG, "q_stride_token"),
    ("q", None, B.SMLA_ERR_INVALID_ARG, "q is required"),
    ("q", 0x50008, B.SMLA_ERR_INVALID_ARG, "q must be 16-byte"),
    ("out", 0x60008, B.SMLA_ERR_INVALID_ARG, "out must be 16-byte"),
    ("out_lse", 0x60002, B.SMLA_ERR_INVALID_ARG, "out_lse must be 4-byte"),
    ("sinks", 0x60002, B.SMLA_ERR_INVALID_ARG, "sinks must be 4-byte"),
    ("bmm1_scale_dev", 0x60002, B.SMLA_ERR_INVALID_ARG, "bmm1_scale_dev must be 4-byte"),
    ("error_word", 0x60002, B.SMLA_ERR_INVALID_ARG, "error_word must be 4-byte"),
])
def test_window_errors(lib, field, value, code, needle):
    a = window_struct()
    setattr(a, field, value)
    refused(lib.smla_window_attention(ctypes.byref(a), None), code, needle)


def test_append_errors_and_empty_calls(lib):
    a = append_struct()
    a.latent_stride = 508
    refused(lib.smla_cache_append(ctypes.byref(a), None), B.SMLA_ERR_INVALID_ARG, "latent_stride")
    a = append_struct()
    a.latent = 0x50004
    refused(lib.smla_cache_append(ctypes.byref(a), None), B.SMLA_ERR_INVALID_ARG, "latent must be 16-byte")
    for f in (lib.smla_window_attention, lib.smla_cache_append, lib.smla_pages_resize, lib.smla_pages_fork,
              lib.smla_pages_compact):
        refused(f(None, None), B.SMLA_ERR_INVALID_ARG, "NULL")
    w, p, a = window_struct(), pages_struct(), append_struct()
    w.sum_q = p.rows = a.sum_q = 0
    assert lib.smla_window_attention(ctypes.byref(w), None) == B.SMLA_OK
    assert lib.smla_cache_append(ctypes.byref(a), None) == B.SMLA_OK
    assert lib.smla_pages_fork(ctypes.byref(p), None) == B.SMLA_OK
    p.move_count = None                                    # (these two set it to 0 on the device)
    for f in (lib.smla_pages_resize, lib.smla_pages_compact):
        refused(f(ctypes.byref(p), None), B.SMLA_ERR_INVALID_ARG, "move_count is required")


@pytest.mark.parametrize("call,field,value,code,needle", [
    ("resize", "rows", -1, B.SMLA_ERR_INVALID_ARG, "rows"),
    ("resize", "max_pages", 0, B.SMLA_ERR_INVALID_ARG, "max_pages"),
    ("resize", "page_size", 0, B.SMLA_ERR_INVALID_ARG, "page_size"),
    ("resize", "page_size", 1 << 30, B.SMLA_ERR_INVALID_ARG, "max_pages"),
    ("resize", "rows", 1 << 29, B.SMLA_ERR_UNSUPPORTED, "2^30"),
    ("resize", "num_pages", 0, B.SMLA_ERR_INVALID_ARG, "num_pages"),
    ("resize", "block_table_stride", 3, B.SMLA_ERR_INVALID_ARG, "block_table_stride"),
    ("resize", "block_tables", None, B.SMLA_ERR_INVALID_ARG, "block_tables"),
    ("resize", "ref_counts", None, B.SMLA_ERR_INVALID_ARG, "ref_counts"),
    ("resize", "lens", None, B.SMLA_ERR_INVALID_ARG, "lens"),
    ("resize", "new_lens", None, B.SMLA_ERR_INVALID_ARG, "new_lens"),
    ("resize", "move_capacity", 7, B.SMLA_ERR_INVALID_ARG, "move_capacity"),
    ("resize", "move_count", None, B.SMLA_ERR_INVALID_ARG, "move_count"),
    ("resize", "move_src", None, B.SMLA_ERR_INVALID_ARG, "move_src"),
    ("resize", "workspace", None, B.SMLA_ERR_WORKSPACE_TOO_SMALL, "workspace"),
    ("resize", "workspace_bytes", 100, B.SMLA_ERR_WORKSPACE_TOO_SMALL, "workspace"),
    ("resize", "workspace", 0x100080, B.SMLA_ERR_INVALID_ARG, "256-byte"),
    ("compact", "move_capacity", 49, B.SMLA_ERR_INVALID_ARG, "move_capacity"),
    ("fork", "parents", None, B.SMLA_ERR_INVALID_ARG, "parents"),
    ("fork", "out_lens", None, B.SMLA_ERR_INVALID_ARG, "out_lens"),
    ("fork", "out_lens", 0x30000, B.SMLA_ERR_INVALID_ARG, "must not be lens"),
    ("fork", "out_lens", 0x30004, B.SMLA_ERR_INVALID_ARG, "overlap"),
    ("fork", "out_lens", 0x2fffc, B.SMLA_ERR_INVALID_ARG, "overlap"),
    ("fork", "error_word", 0x60002, B.SMLA_ERR_INVALID_ARG, "error_word"),
])
def test_pages_errors(lib, call, field, value, code, needle):
    a = pages_struct()
    setattr(a, field, value)
    refused(getattr(lib, f"smla_pages_{call}")(ctypes.byref(a), None), code, needle)


@pytest.mark.parametrize("pool,needle", [((None, 64, 64), "no base"), ((0x1000, 0, 64), "page_bytes"),
                                         ((0x1000, 1 << 31, 1 << 31), "page_bytes"), ((0x1000, 64, 32), "page_stride")])
def test_copy_errors(lib, pool, needle):
    array = (C.SmlaPool * 1)(pool)
    refused(lib.smla_pages_copy(ctypes.byref(array), 1, 10, 0x100, 0x200, 0x300, 5, None, None),
            B.SMLA_ERR_INVALID_ARG, needle)


def test_copy_counts_and_pointers(lib):
    array = (C.SmlaPool * 1)((0x1000, 64, 64))

    def call(pools=1, pages=10, src=0x100, capacity=5):
        return lib.smla_pages_copy(ctypes.byref(array), pools, pages, src, 0x200, 0x300, capacity, None, None)

    refused(call(pools=-1), B.SMLA_ERR_INVALID_ARG, "num_pools")
    refused(call(pages=0), B.SMLA_ERR_INVALID_ARG, "num_pages")
    refused(call(capacity=-1), B.SMLA_ERR_INVALID_ARG, "move_capacity")
    refused(call(src=None), B.SMLA_ERR_INVALID_ARG, "move_src")
    refused(call(src=0x102), B.SMLA_ERR_INVALID_ARG, "move_src")
    assert call(pools=0) == call(capacity=0) == B.SMLA_OK


def host_tensors(**over):
    kw = dict(q=torch.zeros(4, 64, 512, dtype=torch.bfloat16), rows=torch.zeros(10, 64, 512, dtype=torch.uint8),
              scales=torch.ones(10, 4), block_tables=torch.zeros(2, 4, dtype=torch.int32),
              seq_lens=torch.zeros(2, dtype=torch.int32), workspace_buffer=None, window=16)
    kw.update(over)
    return kw


@pytest.mark.parametrize("over,exc,match", [
    ({}, ValueError, "CUDA device"),
    (dict(q=torch.zeros(4, 64, 512)), TypeError, "bfloat16"),
    (dict(q=torch.zeros(4, 64, 256, dtype=torch.bfloat16)), ValueError, "contiguous heads"),
    (dict(q=torch.zeros(4, 512, 64, dtype=torch.bfloat16).transpose(1, 2)), ValueError, "contiguous heads"),
    (dict(rows=torch.zeros(10, 64, 512)), TypeError, "float8_e4m3fn"),
    (dict(rows=torch.zeros(10, 64, 500, dtype=torch.uint8)), ValueError, "contiguous rows"),
    (dict(rows=torch.zeros(1, 64, 512, dtype=torch.uint8).expand(10, 64, 512)), ValueError, "share memory"),
    (dict(scales=torch.ones(10, 4, dtype=torch.float64)), TypeError, "float32"),
    (dict(scales=torch.ones(9, 4)), ValueError, "scales"),
    (dict(scales=torch.ones(10, 5)), ValueError, "do not divide"),
    (dict(scales=torch.ones(10, 8)[:, ::2]), ValueError, "contiguous last dim"),
    (dict(block_tables=torch.zeros(2, 4, dtype=torch.int64)), TypeError, "int32"),
    (dict(block_tables=torch.zeros(4, 2, dtype=torch.int32).t()), ValueError, "contiguous last dim"),
    (dict(block_tables=torch.zeros(1, 4, dtype=torch.int32).expand(2, 4)), ValueError, "overlap"),
    (dict(seq_lens=torch.zeros(1, dtype=torch.int32)), ValueError, "seq_lens has 1"),
    (dict(seq_lens=torch.zeros(4, dtype=torch.int32)[::2]), ValueError, "contiguous"),
    (dict(seq_lens=torch.zeros(2, dtype=torch.int64)), TypeError, "int32"),
    (dict(cum_seq_lens_q=torch.zeros(2, dtype=torch.int32)), ValueError, "cum_seq_lens_q has 2"),
    (dict(sinks=torch.zeros(63)), ValueError, "sinks has 63"),
    (dict(sinks=torch.zeros(64, dtype=torch.bfloat16)), TypeError, "float32"),
    (dict(bmm1_scale=torch.ones(1, dtype=torch.float16)), TypeError, "bmm1_scale"),
    (dict(bmm2_scale=torch.ones(0)), ValueError, "bmm2_scale has 0"),
    (dict(out=torch.zeros(4, 64, 512)), ValueError, "out must be"),
    (dict(out=torch.zeros(4, 64, 512, dtype=torch.bfloat16), out_lse=torch.zeros(4, 63)), ValueError, "out_lse"),
    (dict(error_word=torch.zeros(1)), TypeError, "error_word"),
    (dict(workspace_buffer=torch.zeros(64, dtype=torch.uint8)[::2]), ValueError, "workspace"),
])
def test_binding_refuses_before_the_library(over, exc, match):
    with pytest.raises(exc, match=match):
        C.window_attention(**host_tensors(**over))


def test_binding_refuses_host_tensors_in_every_call():
    t = dict(block_tables=torch.zeros(2, 4, dtype=torch.int32), ref_counts=torch.zeros(9, dtype=torch.int32),
             lens=torch.zeros(2, dtype=torch.int32))
    moves = C.new_moves(4, "cpu")
    ws = torch.zeros(4096, dtype=torch.uint8)
    two = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        C.pages_resize(**t, new_lens=two, workspace_buffer=ws, page_size=16, moves=moves)
    with pytest.raises(ValueError, match="workspace"):
        C.pages_resize(**t, new_lens=two, workspace_buffer=None, page_size=16, moves=moves)
    with pytest.raises(ValueError, match="new_lens has 1"):
        C.pages_resize(**t, new_lens=two[:1], workspace_buffer=ws, page_size=16, moves=moves)
    with pytest.raises(ValueError, match="CUDA device"):
        C.pages_fork(**t, parents=two, out_lens=two.clone(), page_size=16)
    with pytest.raises(ValueError, match="CUDA device"):
        C.pages_compact(**t, workspace_buffer=ws, page_size=16, moves=moves)
    with pytest.raises(ValueError, match="CUDA device"):
        C.pages_copy([torch.zeros(9, 16)], moves)
    with pytest.raises(ValueError, match="pages must be contiguous"):
        C.pages_copy([torch.zeros(9, 16, 4)[:, :, ::2]], moves)
    with pytest.raises(ValueError, match="first pool's 9 pages"):
        C.pages_copy([torch.zeros(9, 16), torch.zeros(8, 16)], moves)
    with pytest.raises(ValueError, match="moves.dst has 3"):
        C.pages_copy([torch.zeros(9, 16)], (moves[0], moves[1][:3], moves[2]))
    with pytest.raises(ValueError, match="CUDA device"):
        C.append(torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(10, 64, 512, dtype=torch.uint8),
                 torch.ones(10, 4), t["block_tables"], t["lens"])
    with pytest.raises(ValueError, match="contiguous rows"):
        C.append(torch.zeros(512, 4, dtype=torch.bfloat16).t(), torch.zeros(10, 64, 512, dtype=torch.uint8),
                 torch.ones(10, 4), t["block_tables"], t["lens"])


def test_pages_workspace_grows_with_rows_and_pages(lib):
    def need(rows, pages):
        return C.pages_workspace_size(torch.zeros(rows, 4, dtype=torch.int32), torch.zeros(pages, dtype=torch.int32), 64)
    assert need(8, 100) >= 4 * (100 + 16) and need(8, 100) % 256 == 0
    assert need(8, 100000) > need(8, 100) and need(1000, 100) > need(8, 100)


# ------------------------------------------------------------ the reference

def test_reference_window_is_dense_attention_and_drops_unseen_rows():
    rng = np.random.default_rng(0)
    rows = R.to_e4m3(rng.normal(size=(3, 8, 512)))
    scales = np.array([[0.5, 2.0], [1.0, 0.25], [4.0, 1.0]], dtype=np.float32)
    cache = R.Cache(rows, scales, np.array([[2, 0, 1]]), np.array([20]), tokens=1)
    q = rng.normal(size=(1, 2, 512))
    full = np.concatenate([R.e4m3(rows[p]).reshape(2, 4, 512) * scales[p][:, None, None] for p in (2, 0, 1)]
                          ).reshape(24, 512)[:20]
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q), torch.from_numpy(full)[None],
                                                            torch.from_numpy(full)[None], scale=0.1)[0].numpy()
    out, lse, _, _ = R.window(cache, q, window=1000, bmm1=0.1)
    assert np.abs(out[0] - want).max() < 1e-12
    part, _, _, _ = R.window(cache, q, window=3, first=2, bmm1=0.1)
    seen = full[[0, 1, 17, 18, 19]]
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q), torch.from_numpy(seen)[None],
                                                            torch.from_numpy(seen)[None], scale=0.1)[0].numpy()
    assert np.abs(part[0] - want).max() < 1e-12


def test_reference_append_by_hand():
    rows, scales = np.zeros((1, 8, 512), np.uint8), np.ones((1, 2), np.float32)
    cache = R.Cache(rows, scales, np.array([[0]]), np.array([2]), tokens=2)
    x = np.zeros((2, 512), np.float32)
    x[0, 0], x[1, 1] = 448.0, 3.0
    R.append(cache, x)                                    # amax 448: scale 1
    assert scales[0, 0] == 1.0 and R.e4m3(rows[0, 0])[0] == 448.0 and R.e4m3(rows[0, 1])[1] == 3.0
    cache = R.Cache(rows, scales, np.array([[0]]), np.array([3]), tokens=1)
    y = np.zeros((1, 512), np.float32)
    y[0, 2] = 449.0                                       # one step over: the block's scale doubles
    R.append(cache, y)
    assert scales[0, 0] == 2.0 and R.e4m3(rows[0, 0])[0] == 224.0 and R.e4m3(rows[0, 1])[1] == 1.5
    assert R.e4m3(rows[0, 2])[2] == 224.0 and scales[0, 1] == 1.0


def test_reference_pages_by_hand():
    p = R.Pages(3, 4, 4, 8)
    assert p.resize(np.array([0, 0, 0]), np.array([6, 4, 0])) == ([], False)
    assert p.tables.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1], [-1] * 4]
    lens = p.fork(np.array([6, 4, 0]), np.array([-1, -1, 0]))
    assert lens.tolist() == [6, 4, 6] and p.refs.tolist() == [2, 2, 1, 0, 0, 0, 0, 0]
    moves, short = p.resize(lens, np.array([7, 5, 7]))    # both sharers of page 1 get a copy
    assert moves == [(1, 3), (1, 5)] and not short
    assert p.tables.tolist() == [[0, 3, -1, -1], [2, 4, -1, -1], [0, 5, -1, -1]]
    assert p.refs.tolist() == [2, 0, 1, 1, 1, 1, 0, 0]
    assert p.compact(np.array([7, 5, 7])) == [(5, 1)] and p.tables[2].tolist() == [0, 1, -1, -1]
    _, short = p.resize(np.array([7, 5, 7]), np.array([16, 16, 7]))
    assert short and p.tables[0].tolist() == [0, 3, 5, 6] and p.tables[1].tolist() == [2, 4, 7, -1]


def test_numbers_past_32_bits_are_refused():
    for name in ("window", "first_tokens", "num_splits"):
        with pytest.raises(ValueError, match=f"{name} .* 32-bit"):
            C.window_attention(**host_tensors(**{name: (1 << 32) + 5}))
    with pytest.raises(ValueError, match="page_size .* 32-bit"):
        C.pages_workspace_size(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32), (1 << 32) + 8)


def test_missing_extension_raises(monkeypatch, tmp_path):
    monkeypatch.setattr(C, "_extension", None)
    monkeypatch.setattr(C, "EXTENSION_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(ImportError, match="not built"):
        C.window_attention(**host_tensors())


def test_extension_leaves_what_is_not_plain_to_the_python_functions():
    """No tensors, host tensors and odd numbers of arguments never reach an entry point."""
    e = C.extension()
    x = torch.zeros(4, 512, dtype=torch.bfloat16)
    for f, n in ((e.window_attention, 17), (e.append, 8), (e.pages_resize, 9), (e.pages_fork, 8), (e.pages_compact, 8),
                 (e.pages_copy, 4)):
        assert f(*[None] * n) is None and f(*[x] * n) is None and f(*[3] * n) is None and f(*[[x]] * n) is None
        assert f(*[(x, x, x)] * n) is None
        with pytest.raises(TypeError, match="arguments"):
            f(*[None] * (n - 1))
