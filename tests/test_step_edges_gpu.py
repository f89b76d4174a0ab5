"""Edges of a step's calls on the GPU: positions past the tables behind shared prefixes, lengths that are none,
workspaces bracketed by memory that no call may write."""
import math

import numpy as np
import pytest
import torch

from sparse_mla_decode_token_gb300 import binding as B
from sparse_mla_decode_token_gb300 import cache as C
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
    assert np.all(np.abs(got[1] - want[1])[~empty] <= 2.0 ** -15 * np.abs(want[1][~empty]))


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
