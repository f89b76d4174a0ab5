"""Edges of a step's calls on the GPU: positions past the tables behind shared prefixes, lengths that are none,
workspaces bracketed by memory that no call may write."""

import numpy as np
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from sparse_mla_decode_token_gb300 import binding as B
from sparse_mla_decode_token_gb300 import cache as C
from sparse_mla_decode_token_gb300 import search, slots
from test_prefix_gpu import SCALE, built, i32, make, on_gpu, queries  # noqa: F401  (built: the library, once a module)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def both(cache, starts, prefix, q, flag):
    """The prefix attention of a call and the window attention over whole sequences, each with its flags."""
    g, qt, s, p, cum = on_gpu(cache), queries(q)[0], i32(starts), i32(prefix), i32(cache.cum)
    results = []
    for shared in (True, False):
        kw = dict(group_starts=s, cum_seq_lens_q=cum) if shared else dict(window=1 << 30, cum_seq_lens_q=cum)
        size = (C.prefix_workspace_size if shared else C.window_workspace_size)(qt, *g, **kw)
        ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        if shared:
            out, lse = C.prefix_attention(qt, *g, ws, prefix_lens=p, bmm1_scale=SCALE, error_word=err, **kw)
        else:
            out, lse = C.window_attention(qt, *g, ws, bmm1_scale=SCALE, error_word=err, **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == flag, ("prefix" if shared else "window", int(err.item()))
        results.append((out.double().cpu().numpy(), lse.double().cpu().numpy()))
    return results


def close(got, want):
    # each within 2^-7 of the value (weights and output rounded to BF16) and of the weighted rows' size
    empty = np.isneginf(want[1])
    assert np.array_equal(np.isneginf(got[1]), empty) and np.all(got[0][empty] == 0)
    limit = 2.0 ** -7 * np.abs(want[0]) + 2.0 ** -8 * np.sqrt((want[0] ** 2).mean(axis=-1, keepdims=True)) * 8
    assert np.all(np.abs(got[0] - want[0]) <= limit)
    assert np.all(np.abs(got[1][~empty] - want[1][~empty]) <= 2.0 ** -15 * np.abs(want[1][~empty]))


@pytest.mark.parametrize("members,past", [(40, 1), (40, 300), (6, 1)])
def test_tokens_past_a_table_that_their_prefix_fills(members, past):
    """A shared prefix of all the table's rows; the new token of one member stands past them.  (40 members of 16 heads
    share it, 6 take each token by itself.)"""
    cache, starts, q, _ = make(members, [members], [4096], [0] * members, [1] * members, heads=16, shared=True)
    cache.tables = cache.tables[:, :64].copy()
    close(*both(cache, starts, [4096], q, 0))
    cache.lens[members - 2] += past
    close(*both(cache, starts, [4096], q, B.DEVERR_INDEX_OUT_OF_RANGE))


@pytest.mark.parametrize("members,heads", [(40, 16), (5, 16), (5, 64)])
@pytest.mark.parametrize("least", [-2 ** 31, -2 ** 31 + 1, -1])
def test_lengths_under_zero_are_none(members, heads, least):
    """Requests of a negative length, one of a group and one of none: their tokens see nothing, and as the group's tokens
    share what all of them see, it shares nothing.  (Prefixes of whole pages, which the members hold alike.)"""
    own, q_lens = [3 + b for b in range(members)], [1 + b % 3 for b in range(members)]
    cache, starts, q, _ = make(heads, [members, 2], [4032, 128], own + [4, 2], q_lens + [2, 1, 2], heads=heads, shared=True,
                               outside=[200])
    cache.lens[2] = cache.lens[members + 2] = least
    results = both(cache, starts, [4032, 128], q, 0)
    close(*results)
    for out, lse in results:
        for b in (2, members + 2):
            t = slice(cache.cum[b], cache.cum[b + 1])
            assert np.all(out[t] == 0) and np.all(np.isneginf(lse[t]))


def allocating_calls():
    """Calls that allocate their outputs, of a batch padded by two tokens in front and three behind: name -> (call, the
    outputs that tokens of no request leave alone)."""
    cache, starts, q, rng = make(3, [4], [150], [1, 2, 30, 4], [1, 2, 1, 1], heads=16)
    pad = np.concatenate([rng.normal(size=(2, 16, 512)), q, rng.normal(size=(3, 16, 512))])
    g, qt, cum = on_gpu(cache), queries(pad)[0], i32(cache.cum + 2)
    ws = torch.empty(1 << 25, dtype=torch.uint8, device=DEV)
    logits, scores = torch.randn(8, 500, device=DEV), torch.zeros(2, 4, device=DEV)
    lens = i32([3, 4])
    return {
        "window": (lambda: C.window_attention(qt, *g, ws, window=1 << 20, cum_seq_lens_q=cum), 2),
        "prefix": (lambda: C.prefix_attention(qt, *g, ws, group_starts=i32(starts), prefix_lens=i32([150]), cum_seq_lens_q=cum), 2),
        "beams": (lambda: search.beam_select(logits, scores, ws), 3),
        "tokens": (lambda: slots.token_slots(lens, lens + 1, i32([[1], [2]]), max_tokens=5, page_size=8), 4),
        "sparse": (lambda: slots.sparse_slots(lens, i32([[1], [2]]), 2, page_size=8), 2),
    }


def test_deterministic_fill_of_new_outputs():
    """torch fills new memory where it is asked for deterministic algorithms; what a call leaves alone is NaN then."""
    calls = allocating_calls()
    held = [torch.full((1 << 16,), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(8)]
    del held                                               # memory for the outputs that holds numbers
    torch.use_deterministic_algorithms(True)
    try:
        for name in ("window", "prefix"):
            out, lse = calls[name][0]()
            torch.cuda.synchronize()
            for t in (out, lse):
                assert bool(t[:2].isnan().all()) and bool(t[-3:].isnan().all()) and bool(t[2:-3].isfinite().all()), name
    finally:
        torch.use_deterministic_algorithms(False)


def test_dispatch_modes_see_new_outputs():
    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.empty = 0

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.empty += func.overloadpacket in (torch.ops.aten.empty, torch.ops.aten.empty_like)
            return func(*args, **(kwargs or {}))

    for name, (call, outputs) in allocating_calls().items():
        with Seen() as seen:
            call()
        assert seen.empty == outputs, name
    torch.cuda.synchronize()
