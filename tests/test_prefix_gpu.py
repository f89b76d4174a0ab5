"""Attention of groups that share prefixes on the GPU, against the cache's 64-bit
reference with the prefix looked up through the group's first request."""
import math

import numpy as np
import pytest
import torch

import cache_reference as R
from sparse_mla_decode_token_gb300 import binding as B
from sparse_mla_decode_token_gb300 import cache as C

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1 / math.sqrt(512)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_decode_token_gb300 import build
    build.build()
    B.lib()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Grouped(R.Cache):
    """Rows before a group's prefix come from the pages of its first request that has new tokens."""

    def groups(self, starts, prefix):
        self.first, self.prefix = np.arange(len(self.lens)), np.zeros(len(self.lens), dtype=int)
        for g, p in enumerate(prefix):
            of = range(starts[g], starts[g + 1])
            seen = [int(self.lens[b]) - int(self.cum[b + 1] - self.cum[b]) + 1 for b in of if self.cum[b + 1] > self.cum[b]]
            lead = min([b for b in of if self.cum[b + 1] > self.cum[b]], default=starts[g])
            for b in of:
                self.first[b], self.prefix[b] = lead, max(0, min([int(p)] + seen))
        return self

    def page(self, b, j):
        return super().page(int(self.first[b]) if j < self.prefix[b] else b, j)


def make(seed, members, prefix, own, q_lens, *, heads, page_size=64, block=16, shared=False, outside=()):
    """Groups of `members` requests with `prefix` rows each and own[b] behind; what no request may read (a member's
    columns of the prefix unless `shared`, rows of no request, their scales) is NaN or no page.  `outside`: lengths of
    requests behind the last group."""
    rng = np.random.default_rng(seed)
    starts = np.concatenate([[0], np.cumsum(members)])
    group = np.repeat(np.arange(len(members)), members)
    lens = np.concatenate([np.asarray(prefix)[group] + np.asarray(own), outside]).astype(int)
    width = max(1, -(-int(lens.max()) // page_size))
    tables = np.full((len(lens), width + 1), -77, dtype=np.int32)
    pages = sum(-(-int(n) // page_size) for n in lens) + 3
    order = list(rng.permutation(pages))
    rows = np.full((pages, page_size, 512), 0x7F, dtype=np.uint8)
    scales = np.full((pages, page_size // block), np.nan, dtype=np.float32)

    def fill(page, n):
        for r in range(0, n, block):
            scales[page, r // block] = 2.0 ** rng.integers(-8, -5)
            k = min(block, n - r)
            rows[page, r:r + k] = R.to_e4m3(rng.normal(size=(k, 512)) * 100.0)

    for b, n in enumerate(lens):
        g = group[b] if b < len(group) else None
        lead = 0 if g is None or b == starts[g] else int(prefix[g]) // page_size
        for c in range(-(-int(n) // page_size)):
            if c < lead:
                if shared:
                    tables[b, c] = tables[starts[g], c]
                continue
            tables[b, c] = order.pop()
            fill(tables[b, c], min(page_size, int(n) - c * page_size))
    cum = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    cache = Grouped(rows, scales, tables, lens, cum=cum).groups(starts, prefix)
    return cache, starts, rng.normal(size=(int(cum[-1]), heads, 512)), rng


def on_gpu(cache):
    return (torch.from_numpy(cache.rows).to(DEV), torch.from_numpy(cache.scales).to(DEV), i32(cache.tables), i32(cache.lens))


def queries(q):
    t = torch.from_numpy(np.ascontiguousarray(q, dtype=np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.to(torch.float64).numpy()


def widened(tables, tokens, heads):
    """The tables with as many more columns (no pages) as make the call long enough, by what it knows of the lengths, to
    compute shared prefixes once for all: shorter ones take each token by itself."""
    empty = -(-heads // 64) - heads / 64                   # of a token's blocks of 64 rows: what sharing may save
    columns = int(7 * 152 * 128 / 8 / (tokens * empty)) + 1 if empty else 3
    return np.concatenate([tables, np.full((tables.shape[0], columns), -77, dtype=np.int32)], axis=1)


def run(cache, *args, **kw):
    """The results of the call as it is, and on widened tables."""
    q, tables = args[2], cache.tables
    first = run_one(cache, *args, **kw)
    try:
        cache.tables = widened(tables, q.shape[0], q.shape[1])
        return first, run_one(cache, *args, **kw)
    finally:
        cache.tables = tables


def run_one(cache, starts, prefix, q, *, sinks=None, bmm1=SCALE, bmm2=1.0, flag=0, uniform=False, cum=None, stream=None):
    qt = q if isinstance(q, torch.Tensor) else queries(q)[0]
    g = on_gpu(cache)
    cum = None if uniform else i32(cache.cum) if cum is None else cum
    s, p = i32(starts), i32(prefix)
    ws = torch.full((C.prefix_workspace_size(qt, *g, group_starts=s, cum_seq_lens_q=cum),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full(qt.shape, math.nan, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(qt.shape[:2], math.nan, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    C.prefix_attention(qt, *g, ws, group_starts=s, prefix_lens=p, cum_seq_lens_q=cum, bmm1_scale=bmm1, bmm2_scale=bmm2,
                       sinks=None if sinks is None else torch.from_numpy(sinks.astype(np.float32)).to(DEV),
                       out=out, out_lse=lse, error_word=err, stream=stream)
    torch.cuda.synchronize()
    assert int(err.item()) == flag
    return out.to(torch.float64).cpu().numpy(), lse.to(torch.float64).cpu().numpy()


def check(cache, q, results, **kw):
    want = R.window(cache, queries(q)[1], window=1 << 30, bmm1=kw.pop("bmm1", SCALE), **kw)
    for got in results:
        check_one(got, *want)


def check_one(got, out, lse, tol_o, tol_l):
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got[1]), empty) and np.all(got[0][empty] == 0)
    bad = ~(np.abs(got[0] - out) <= tol_o) & ~empty[..., None]
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got[0] - out)[bad][:5], tol_o[bad][:5])
    assert np.all(np.abs(got[1][~empty] - lse[~empty]) <= tol_l[~empty])
    scale = np.sqrt((out[~empty] ** 2).mean())
    assert np.sqrt(((got[0] - out)[~empty] ** 2).mean()) <= 2.0 ** -8 * scale


CASES = [
    # members, prefix, own, heads, page_size, block
    ([4], [200], [1, 40, 7, 64], 16, 64, 16),
    ([4], [513], [3, 1, 130, 65], 8, 64, 16),
    ([3, 1, 2], [130, 77, 0], [1, 2, 3, 9, 5, 200], 12, 16, 8),
    ([2, 3], [64, 255], [1, 1, 2, 2, 1], 1, 8, 8),
    ([9], [300], [1 + i * 13 for i in range(9)], 5, 24, 8),
    ([2, 2], [400, 129], [17, 300, 1, 2], 64, 64, 16),
    ([3], [250], [4, 5, 1], 128, 64, 16),
    ([5], [700], [1, 2, 90, 4, 5], 96, 32, 32),
    ([40], [1000], [1 + i % 7 for i in range(40)], 33, 64, 64),
    ([1], [500], [20], 16, 64, 16),
]


@pytest.mark.parametrize("members,prefix,own,heads,page_size,block", CASES)
def test_decode(members, prefix, own, heads, page_size, block):
    cache, starts, q, rng = make(heads, members, prefix, own, [1] * len(own), heads=heads, page_size=page_size, block=block)
    sinks = rng.normal(size=heads)
    check(cache, q, run(cache, starts, prefix, q, sinks=sinks, bmm2=0.5), sinks=sinks, bmm2=0.5)
    check(cache, q, run(cache, starts, prefix, q, uniform=True))


@pytest.mark.parametrize("heads", [3, 16, 48, 64, 100, 128])
def test_several_tokens_a_request(heads):
    members, prefix = [3, 2, 4], [300, 90, 128]
    q_lens = [4, 0, 2, 1, 3, 1, 1, 5, 2]
    own = [10, 3, 200, 1, 3, 5, 1, 5, 40]
    cache, starts, q, rng = make(heads + 1, members, prefix, own, q_lens + [3, 6], heads=heads, outside=[150, 4])
    sinks = rng.normal(size=heads)
    # (the last request has fewer tokens than it is said to have new ones: two see nothing)
    check(cache, q, run(cache, starts, prefix, q, sinks=sinks), sinks=sinks)


def test_prompt_chunks_behind_a_prefix():
    cache, starts, q, _ = make(5, [3], [260], [150, 20, 131], [150, 20, 131], heads=20)
    check(cache, q, run(cache, starts, [260], q))


@pytest.mark.parametrize("heads", [16, 64])
def test_a_prefix_past_what_all_see_ends_there(heads):
    # the shortest request's first new token stands at 101 + 3 - 2 = 102
    cache, starts, q, _ = make(9, [3], [101], [3, 30, 60], [2, 1, 4], heads=heads, shared=True)
    cache.groups(starts, [103])
    first = run(cache, starts, [103], q)
    check(cache, q, first)
    cache.groups(starts, [5000])
    got = run(cache, starts, [5000], q)
    check(cache, q, got)
    assert cache.prefix.max() == 103
    assert all(np.array_equal(a[0], b[0]) for a, b in zip(first, got))
    cache.groups(starts, [-5])
    check(cache, q, run(cache, starts, [-5], q))


@pytest.mark.parametrize("prefix,heads", [(40000, 16), (9000, 128), (20000, 8)])
def test_long_prefixes_in_many_pieces(prefix, heads):
    cache, starts, q, _ = make(4, [3], [prefix], [1, 300, 2], [1, 1, 1], heads=heads)
    check(cache, q, run(cache, starts, [prefix], q))


def test_long_own_parts_in_many_pieces():
    cache, starts, q, _ = make(14, [2, 2], [70, 64], [9000, 1, 2, 5000], [1, 1, 1, 1], heads=24)
    check(cache, q, run(cache, starts, [70, 64], q))


def test_a_token_of_nothing_but_the_prefix():
    # the new token is the prefix's last row: nothing behind it
    cache, starts, q, _ = make(6, [6], [192], [0] * 6, [1] * 6, heads=16)
    check(cache, q, run(cache, starts, [192], q))


def test_equal_to_the_window_attention_on_shared_pages():
    cache, starts, q, _ = make(8, [8, 8], [640, 320], [1 + i for i in range(16)], [1] * 16, heads=16, shared=True)
    results = run(cache, starts, [640, 320], q)
    g, qt = on_gpu(cache), queries(q)[0]
    prefix = i32([-1, -1])
    C.pages_shared_prefix(g[2], g[3], i32(starts), prefix, page_size=64)
    assert prefix.cpu().tolist() == [640, 320]
    ws = torch.empty(C.window_workspace_size(qt, *g, window=1 << 20), dtype=torch.uint8, device=DEV)
    out, lse = C.window_attention(qt, *g, ws, window=1 << 20, bmm1_scale=SCALE)
    torch.cuda.synchronize()
    # both within 2^-7 of the value (weights and output rounded to BF16) of each other, and of the weighted rows' size
    for got in results:
        limit = 2.0 ** -7 * np.abs(got[0]) + 2.0 ** -8 * np.sqrt((got[0] ** 2).mean(axis=-1, keepdims=True)) * 8
        assert np.all(np.abs(out.double().cpu().numpy() - got[0]) <= limit)
        assert np.all(np.abs(lse.double().cpu().numpy() - got[1]) <= 2.0 ** -15 * np.abs(got[1]))


def test_padded_batches_leave_their_outputs_alone():
    cache, starts, q, rng = make(3, [4], [150], [1, 2, 30, 4], [1, 2, 1, 1], heads=16)
    pad = np.concatenate([rng.normal(size=(2, 16, 512)), q, rng.normal(size=(3, 16, 512))])
    for got in run(cache, starts, [150], pad, cum=i32(cache.cum + 2)):
        assert np.isnan(got[0][:2]).all() and np.isnan(got[0][-3:]).all() and np.isnan(got[1][:2]).all()
        check(cache, q, [(got[0][2:-3], got[1][2:-3])])


def test_strided_queries_and_one_group_per_request():
    cache, _, q, _ = make(2, [1, 1, 1], [40, 50, 60], [5, 6, 7], [2, 1, 3], heads=16)
    wide = torch.full((6, 20, 512), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[:, 2:18] = queries(q)[0]
    check(cache, q, run(cache, np.arange(4), [40, 50, 60], wide[:, 2:18]))
    # groups without requests beside one of one request, and none at all
    got = run(cache, [0, 0, 1, 1, 1], [9, 40, 9, 7], q)
    check(cache.groups([0], []), q, got)
    check(cache, q, run(cache, [0], [], q))


def test_groups_out_of_order_are_flagged_and_share_nothing():
    cache, _, q, _ = make(7, [4], [128], [1, 2, 3, 4], [1] * 4, heads=16, shared=True)
    cache.groups([0], [])
    for starts in ([2, 0, 4], [0, 5], [-1, 4]):
        check(cache, q, run(cache, starts, [128] * (len(starts) - 1), q, flag=B.DEVERR_PAGE_STATE))


def test_pages_that_are_none_are_masked_and_flagged():
    cache, starts, q, _ = make(11, [4], [320], [10, 20, 5, 40], [1] * 4, heads=16)
    cache.tables[0, 2] = 10 ** 6                          # of the prefix
    cache.tables[3, 5] = -1                               # of a member
    check(cache, q, run(cache, starts, [320], q, flag=B.DEVERR_INDEX_OUT_OF_RANGE))


def test_a_prefix_row_of_nan_reaches_its_group_only():
    cache, starts, q, _ = make(12, [3, 3], [200, 200], [1, 2, 3, 1, 2, 3], [1] * 6, heads=16)
    cache.rows[cache.tables[0, 1], 3] = 0x7F
    out, lse, tol_o, tol_l = R.window(cache, queries(q)[1], window=1 << 30, bmm1=SCALE)
    for got in run(cache, starts, [200, 200], q):
        assert np.isnan(got[0][:3]).all() and np.isnan(got[1][:3]).all()
        assert np.all(np.abs(got[0] - out)[3:] <= tol_o[3:]) and np.all(np.abs(got[1] - lse)[3:] <= tol_l[3:])


@pytest.mark.parametrize("wide", [False, True])
def test_deterministic_captured_and_on_another_stream(wide):
    prefix, q_lens = [900, 300], [1, 2, 1, 1, 3, 1, 1, 1]
    cache, starts, q, rng = make(13, [4, 4], prefix, [1, 9, 3, 4, 50, 6, 7, 8], q_lens, heads=16)
    if wide:
        cache.tables = widened(cache.tables, q.shape[0], 16)
    g, qt, s, p, cum = on_gpu(cache), queries(q)[0], i32(starts), i32(prefix), i32(cache.cum)
    ws = torch.empty(C.prefix_workspace_size(qt, *g, group_starts=s, cum_seq_lens_q=cum), dtype=torch.uint8, device=DEV)
    call = lambda **kw: C.prefix_attention(qt, *g, ws, group_starts=s, prefix_lens=p, cum_seq_lens_q=cum, bmm1_scale=SCALE, **kw)
    first = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = call(stream=side.cuda_stream)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:                                   # two graphs that share a workspace
        with torch.cuda.graph(graph, stream=side):
            outs.append(call())
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    for got in [other] + outs:
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    # a replay takes the lengths and the prefix as they are then
    p.copy_(i32([64, 17]))
    cache.tables[1:4, :1] = cache.tables[0, :1]
    cache.tables[1:4, 1:14] = cache.tables[0, 1:14]
    cache.tables[5:8, :4] = cache.tables[4, :4]
    g[2].copy_(i32(cache.tables))
    graphs[0].replay()
    torch.cuda.synchronize()
    cache.groups(starts, [64, 17])
    check(cache, q, [[t.double().cpu().numpy() for t in outs[0]]])


@pytest.mark.parametrize("wide", [False, True])
def test_two_calls_at_once_on_two_streams(wide):
    prefix, q_lens = [700, 130], [1, 1, 2, 1, 1, 5]
    calls, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in (31, 32):
        cache, starts, q, rng = make(seed, [3, 3], prefix, [1, 90, 3, 4, 50, 6], q_lens, heads=16)
        if wide:
            cache.tables = widened(cache.tables, q.shape[0], 16)
        g, qt, s, p, cum = on_gpu(cache), queries(q)[0], i32(starts), i32(prefix), i32(cache.cum)
        ws = torch.empty(C.prefix_workspace_size(qt, *g, group_starts=s, cum_seq_lens_q=cum), dtype=torch.uint8, device=DEV)
        kw = dict(group_starts=s, prefix_lens=p, cum_seq_lens_q=cum, bmm1_scale=SCALE)
        calls.append(((qt, *g, ws), kw, [t.clone() for t in C.prefix_attention(qt, *g, ws, **kw)],
                      torch.empty_like(qt), torch.empty(qt.shape[:2], device=DEV)))
    torch.cuda.synchronize()
    for _ in range(10):
        for (args, kw, _, out, lse), stream in zip(calls, streams):
            C.prefix_attention(*args, **kw, out=out, out_lse=lse, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    for _, _, first, out, lse in calls:
        assert torch.equal(first[0], out) and torch.equal(first[1], lse)


@pytest.mark.parametrize("heads", [16, 64])
def test_requests_without_tokens_lead_no_group(heads):
    """The group's first request has ended: its table is empty, its prefix is the next one's."""
    cache, starts, q, _ = make(17, [4, 3], [200, 130], [1, 2, 9, 4, 1, 2, 3], [0, 1, 1, 1, 0, 0, 1], heads=heads, shared=True)
    for b in (0, 4, 5):
        cache.tables[b], cache.lens[b] = -1, 0
    cache.groups(starts, [200, 130])
    check(cache, q, run(cache, starts, [200, 130], q))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("cum", [[0, 3, 1, 4], [2, 0, 9, 4], [0, 4, 4, -3]])
def test_offsets_that_fall_stay_in_range(cum, wide):
    cache, starts, q, _ = make(18, [3], [70], [2, 3, 4], [1, 2, 1], heads=16, shared=True)
    if wide:
        cache.tables = widened(cache.tables, 4, 16)
    qt = queries(q)[0]
    g = on_gpu(cache)
    out, lse = torch.full((6, 16, 512), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((6, 16), 7.0, device=DEV)
    ws = torch.empty(C.prefix_workspace_size(qt, *g, group_starts=i32(starts), cum_seq_lens_q=i32(cum)), dtype=torch.uint8, device=DEV)
    guard = torch.full((4096,), 99, dtype=torch.uint8, device=DEV)
    C.prefix_attention(qt, *g, ws, group_starts=i32(starts), prefix_lens=i32([70]), cum_seq_lens_q=i32(cum), bmm1_scale=SCALE,
                       out=out[1:5], out_lse=lse[1:5])
    torch.cuda.synchronize()
    assert bool((out[0] == 7).all()) and bool((out[5] == 7).all()) and bool((lse[0] == 7).all()) and bool((lse[5] == 7).all())
    assert bool((guard == 99).all())


def test_more_groups_than_the_plan_keeps_near():
    n = 600
    cache, starts, q, _ = make(19, [2] * n, [24] * n, [1, 2] * n, [1] * (2 * n), heads=3, page_size=8, block=8)
    check(cache, q, run(cache, starts, [24] * n, q))


def test_many_tokens():
    """More tokens than the plan's threads, of many groups."""
    n = 1300
    cache, starts, q, _ = make(15, [5] * (n // 5), [40] * (n // 5), [1] * n, [1] * n, heads=2, page_size=8, block=8)
    check(cache, q, run(cache, starts, [40] * (n // 5), q))


def test_scales_on_the_device_and_an_empty_batch():
    cache, starts, q, _ = make(16, [4], [128], [1, 2, 3, 4], [1] * 4, heads=16)
    one, two = torch.tensor([SCALE], device=DEV), torch.tensor([0.25], device=DEV)
    check(cache, q, run(cache, starts, [128], q, bmm1=one, bmm2=two), bmm2=0.25)
    g = on_gpu(cache)
    out, lse = C.prefix_attention(torch.empty(0, 16, 512, dtype=torch.bfloat16, device=DEV), *g, None, group_starts=i32(starts),
                                  prefix_lens=i32([128]))
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
