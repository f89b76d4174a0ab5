"""Edges of a step's calls on the GPU: positions past the tables behind shared prefixes, lengths that are none, log sums,
new outputs, workspaces bracketed by memory that no call may write."""
import re

import numpy as np
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from sparse_mla_decode_token_gb300 import binding as B
from sparse_mla_decode_token_gb300 import cache as C
from sparse_mla_decode_token_gb300 import search, slots
from test_prefix_gpu import SCALE, built, i32, make, on_gpu, queries, widened  # noqa: F401  (built: the library, once a module)

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 1 << 16


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


def bracketed(call, size):
    """A workspace of junk, of exactly the bytes that `call` needs (at most `size`, which may cover other calls), and the
    bytes before and behind it that no call may write."""
    try:
        call(None)
        need = 0
    except B.SmlaError as e:
        need = int(re.search(r"0 bytes given, (\d+) needed", str(e)).group(1))
    assert need <= size
    memory = torch.full((need + 2 * GUARD,), 0xFF, dtype=torch.uint8, device=DEV)
    memory[:GUARD] = memory[GUARD + need:] = 99
    return memory[GUARD:GUARD + need], (memory[:GUARD], memory[GUARD + need:])


def untouched(guards):
    return all(bool((g == 99).all()) for g in guards)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("cum", [None, [0, 3, 1, 4], [2, 0, 9, 4], [0, 4, 4, -3], [-5, 1, 2, 9]])
@pytest.mark.parametrize("heads", [16, 100])
def test_prefix_attention_stays_in_its_workspace(cum, wide, heads):
    """Offsets in order and offsets that fall or lie outside the batch."""
    cache, starts, q, _ = make(18, [3], [70], [2, 3, 4], [1, 2, 1], heads=heads, shared=True)
    if wide:
        cache.tables = widened(cache.tables, 4, heads)
    qt, g, s = queries(q)[0], on_gpu(cache), i32(starts)
    c = i32(cache.cum if cum is None else cum)
    call = lambda ws: C.prefix_attention(qt, *g, ws, group_starts=s, prefix_lens=i32([70]), cum_seq_lens_q=c, bmm1_scale=SCALE)
    ws, guards = bracketed(call, C.prefix_workspace_size(qt, *g, group_starts=s, cum_seq_lens_q=c))
    call(ws)
    torch.cuda.synchronize()
    assert untouched(guards)


@pytest.mark.parametrize("members,prefix,heads", [([9, 2], [3000, 40], 16), ([40], [1000], 33), ([1], [9000], 64), ([3, 3], [130, 4000], 128)])
def test_long_prefixes_stay_in_their_workspace(members, prefix, heads):
    n = sum(members)
    cache, starts, q, _ = make(21, members, prefix, [1 + 37 * b % 300 for b in range(n)], [1] * n, heads=heads, shared=True)
    for tables in (cache.tables, widened(cache.tables, n, heads)):
        cache.tables = tables
        qt, g, s = queries(q)[0], on_gpu(cache), i32(starts)
        call = lambda ws: C.prefix_attention(qt, *g, ws, group_starts=s, prefix_lens=i32(prefix), bmm1_scale=SCALE)
        ws, guards = bracketed(call, C.prefix_workspace_size(qt, *g, group_starts=s))
        call(ws)
        torch.cuda.synchronize()
        assert untouched(guards)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("batch,beams,vocab,keep", [(1, 1, 1, 1), (3, 2, 255, 5), (2, 64, 777, 64), (1, 7, 50021, 33), (40, 3, 2000, 3)])
def test_beam_selection_stays_in_its_workspace(batch, beams, vocab, keep, dtype):
    logits, scores = torch.randn(batch * beams, vocab, device=DEV).to(dtype), torch.zeros(batch, beams, device=DEV)
    call = lambda ws: search.beam_select(logits, scores, ws, num_out=keep)
    ws, guards = bracketed(call, search.beam_workspace_size(logits, scores, num_out=keep))
    call(ws)
    torch.cuda.synchronize()
    assert untouched(guards)


@pytest.mark.parametrize("rows,width", [(1, 1), (7, 33), (64, 130), (300, 600)])
def test_reordering_stays_in_its_workspace(rows, width):
    rng = np.random.default_rng(rows)
    tables = i32(rng.permutation(rows * width).reshape(rows, width))
    counts, lens, out = i32(np.ones(rows * width)), i32(rng.integers(0, width * 8 + 1, rows)), i32(np.zeros(rows))
    parents, nothing = i32(rng.integers(-1, rows, rows)), torch.empty(0, dtype=torch.uint8, device=DEV)
    call = lambda ws: C.pages_reorder(tables, counts, lens, parents, out, nothing if ws is None else ws, page_size=8)
    ws, guards = bracketed(call, C.reorder_workspace_size(tables))
    call(ws)
    torch.cuda.synchronize()
    assert untouched(guards)


@pytest.mark.parametrize("heads", [16, 64])
def test_one_workspace_for_steps_of_fewer_tokens(heads):
    """Sized for the largest step; the smaller ones, which are split more, give what they give in one of their own."""
    cache, starts, q, _ = make(6, [40], [2000], [1 + b for b in range(40)], [1] * 40, heads=heads, shared=True)
    g, qt, s, p = on_gpu(cache), queries(q)[0], i32([0, 40]), i32([2000])
    large = torch.empty(C.prefix_workspace_size(qt, *g, group_starts=s), dtype=torch.uint8, device=DEV)
    window = torch.empty(C.window_workspace_size(qt, *g, window=1 << 20), dtype=torch.uint8, device=DEV)
    for n in (40, 39, 20, 3, 1):
        part = (g[0], g[1], g[2][:n], g[3][:n])
        for shared in (True, False):
            kw = dict(group_starts=i32([0, n]), prefix_lens=p) if shared else dict(window=1 << 20)
            call = C.prefix_attention if shared else C.window_attention
            want = call(qt[:n], *part, torch.empty(1 << 26, dtype=torch.uint8, device=DEV), bmm1_scale=SCALE, **kw)
            got = call(qt[:n], *part, large if shared else window, bmm1_scale=SCALE, **kw)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (n, shared)
    logits, scores = torch.randn(160, 128000, device=DEV).to(torch.bfloat16), torch.zeros(20, 8, device=DEV)
    ws = torch.empty(search.beam_workspace_size(logits, scores), dtype=torch.uint8, device=DEV)
    for n in (20, 19, 1):
        want = search.beam_select(logits[:8 * n], scores[:n], torch.empty(1 << 24, dtype=torch.uint8, device=DEV))
        got = search.beam_select(logits[:8 * n], scores[:n], ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n


@pytest.mark.parametrize("dtype,spread", [(torch.bfloat16, 2.0), (torch.float32, 0.0), (torch.float32, 6.0), (torch.float16, 0.5)])
def test_log_sums_of_beams_within_their_bound(dtype, spread):
    """Scores are off by less than 2^-17 and their own rounding, and continuations of different beams are out of order by
    less than 2^-16 at most; one beam's stand in the order of its logits."""
    gen = torch.Generator(device=DEV).manual_seed(41)
    batch, beams, vocab, keep = 6, 16, 150001, 64
    logits = (torch.randn(batch * beams, vocab, generator=gen, device=DEV) * spread + 3).to(dtype)
    scores = -torch.rand(batch, beams, generator=gen, device=DEV) * 2.0 ** -14          # beams that are hardly apart
    ws = torch.empty(search.beam_workspace_size(logits, scores, num_out=keep), dtype=torch.uint8, device=DEV)
    best = search.beam_select(logits, scores, ws, num_out=keep)
    torch.cuda.synchronize()
    x = logits.double()
    total = (x - torch.logsumexp(x, dim=1, keepdim=True) + scores.double().view(-1, 1)).view(batch, -1)
    want = torch.topk(total, keep).values
    parents, tokens = best.parents.long(), best.tokens.long()
    mine = total.gather(1, (parents % beams) * vocab + tokens)                          # the chosen ones' own scores
    half = 2.0 ** -24 * mine.abs()
    assert bool(((best.scores.double() - mine).abs() <= 2.0 ** -17 + half).all())
    assert bool(((mine - want).abs() <= 2.0 ** -16).all()) and bool((mine[:, 1:] - mine[:, :-1] <= 2.0 ** -16).all())
    for r in range(batch):
        chosen = list(zip(parents[r].tolist(), tokens[r].tolist()))
        assert len(set(chosen)) == keep
        for p in set(parents[r].tolist()):
            of = [t for q, t in chosen if q == p]
            assert of == torch.sort(x[p], descending=True, stable=True).indices[:len(of)].tolist()
