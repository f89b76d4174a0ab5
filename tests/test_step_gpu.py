"""A step's calls beside the attention on the GPU: beam selection against 64-bit
scores, reordering, shared prefixes and slot maps against one-entry-at-a-time
references, and all of them in a search over the paged cache."""
import math

import numpy as np
import pytest
import torch

import step_reference as S
from sparse_mla_decode_token_gb300 import binding as B
from sparse_mla_decode_token_gb300 import cache as C
from sparse_mla_decode_token_gb300 import search, slots

pytestmark = pytest.mark.gpu
DEV = "cuda"
BEAM_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_decode_token_gb300 import build
    build.build()
    B.lib()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


# ----------------------------------------------------------------- beam selection

def select(logits, scores, keep, finished=None, end=0, flag=0, stream=None):
    """A call into outputs and a workspace full of junk."""
    ws = torch.full((search.beam_workspace_size(logits, scores, num_out=keep),), 0xFF, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = search.BeamChoice(torch.full((scores.shape[0], keep), math.nan, device=DEV),
                            *(torch.full((scores.shape[0], keep), -77, dtype=torch.int32, device=DEV) for _ in range(2)))
    search.beam_select(logits, scores, ws, num_out=keep, finished=finished, end_token=end, out=out, error_word=err,
                       stream=stream)
    torch.cuda.synchronize()
    assert int(err.item()) == flag
    return [t.cpu().numpy() for t in out]


def tolerance(score):
    """e^x by 2^-22, its argument's rounding by 2^-24 at the most weight, under 64 roundings of sums (2^-18 in all), the
    result rounded to fp32."""
    return 2.0 ** -18 + 2.0 ** -23 * np.abs(np.where(np.isfinite(score), score, 0))


def check(got, logits, scores, keep, finished=None, end=0):
    x = logits.to(torch.float64).cpu().numpy()
    s = scores.cpu().numpy()
    f = None if finished is None else finished.cpu().numpy()
    total = S.beam_scores(x, s, f, end)
    best, _, _ = S.beam_best(total, keep)
    score, rows, tokens = got
    batch, beams = s.shape
    assert np.array_equal(np.isneginf(score), np.isneginf(best))
    fin = np.isfinite(best)
    assert np.all(np.abs(score[fin].astype(np.float64) - best[fin]) <= tolerance(best[fin]))
    assert np.all(rows[~fin] == -1) and np.all(tokens[~fin] == -1)
    for b in range(batch):
        n = int(fin[b].sum())
        pairs = list(zip(rows[b, :n].tolist(), tokens[b, :n].tolist()))
        assert len(set(pairs)) == n
        mine = np.array([total[b, r - b * beams, t] for r, t in pairs])
        assert np.all(np.isfinite(mine)) and np.all(np.abs(mine - best[b, :n]) <= 2 * tolerance(best[b, :n]))
        # of one beam, whose continuations differ by their logits alone: exactly, ties to the lowest token
        for r in set(rows[b, :n].tolist()):
            if f is not None and f[b, r - b * beams]:
                continue
            of = [t for q, t in pairs if q == r]
            order = np.argsort(-x[r], kind="stable")
            assert of == order[:len(of)].tolist()


def likely(g, n, vocab, dtype):
    x = torch.randn(n, vocab, generator=g, device=DEV) * 2
    at = torch.randint(0, vocab, (n, 24), generator=g, device=DEV)
    return x.scatter_add_(1, at, torch.rand(at.shape, generator=g, device=DEV) * 10).to(BEAM_DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("batch,beams,vocab,keep", [
    (1, 1, 1, 1), (1, 1, 5, 8), (3, 2, 255, 2), (2, 4, 257, 8), (1, 3, 1021, 64), (5, 8, 4096, 16), (2, 64, 777, 64),
    (1, 7, 50021, 33), (40, 1, 600, 1), (2, 32, 33001, 64),
])
def test_beam_select(batch, beams, vocab, keep, dtype):
    g = torch.Generator(device=DEV).manual_seed(vocab + beams)
    logits = likely(g, batch * beams, vocab, dtype)
    scores = -torch.rand(batch, beams, generator=g, device=DEV) * 20
    check(select(logits, scores, keep), logits, scores, keep)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 0), (3, 1), (7, 9)])
def test_beam_rows_of_any_stride_and_alignment(dtype, offset, pad):
    g = torch.Generator(device=DEV).manual_seed(7)
    batch, beams, vocab, keep = 2, 3, 2043, 5
    stride = vocab + pad
    # what lies between the rows, before and behind them is larger than anything in them
    memory = torch.full((offset + batch * beams * stride + 8,), 1000.0, dtype=BEAM_DTYPES[dtype], device=DEV)
    logits = memory[offset:offset + batch * beams * stride].view(batch * beams, stride)[:, :vocab]
    logits.copy_(likely(g, batch * beams, vocab, dtype))
    scores = -torch.rand(batch, beams, generator=g, device=DEV)
    check(select(logits, scores, keep), logits, scores, keep)


def test_beam_ties_go_to_the_lowest_beam_and_token():
    # equal logits everywhere: all continuations of all beams of equal score
    for vocab in (3, 256, 4096, 40000):
        logits, scores = torch.zeros(4, vocab, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 4, device=DEV)
        score, rows, tokens = select(logits, scores, 8)
        want = [(i // vocab, i % vocab) for i in range(8)]
        assert list(zip(rows[0].tolist(), tokens[0].tolist())) == want
        assert np.allclose(score, -math.log(vocab), rtol=0, atol=2.0 ** -18)
    # the same rows and scores twice, few different values: ties within and between beams
    g = torch.Generator(device=DEV).manual_seed(3)
    row = torch.randint(-3, 4, (1, 2048), generator=g, device=DEV).to(torch.bfloat16)
    logits, scores = row.expand(5, 2048).contiguous(), torch.tensor([[-1.0, -2, -1, -2, -1]], device=DEV)
    score, rows, tokens = select(logits, scores, 64)
    total = S.beam_scores(logits.double().cpu().numpy(), scores.cpu().numpy())
    best, r, t = S.beam_best(total, 64)
    assert np.array_equal(rows, r) and np.array_equal(tokens, t)


def test_beam_masks_and_missing_continuations():
    g = torch.Generator(device=DEV).manual_seed(11)
    for dtype in ("bf16", "fp16", "fp32"):
        lowest = torch.finfo(BEAM_DTYPES[dtype]).min
        logits = likely(g, 12, 3001, dtype)
        scores = -torch.rand(3, 4, generator=g, device=DEV)
        keep = torch.zeros(3001, dtype=torch.bool, device=DEV)
        keep[[0, 17, 2999]] = True
        logits[0:4] = logits[0:4].masked_fill(~keep, -math.inf)      # three tokens a beam
        logits[4:6] = logits[4:6].masked_fill(~keep, lowest)
        logits[5] = -math.inf                                        # a beam of nothing
        logits[6] = lowest                                           # all at the lowest value: uniform
        scores[2] = torch.tensor([0.0, -math.inf, -math.inf, -math.inf])   # a search's first step
        got = select(logits, scores, 16)
        check(got, logits, scores, 16)
        assert np.isneginf(got[0][0, 12:]).all() and np.isfinite(got[0][0, :12]).all()
        assert set(got[1][2].tolist()) == {8}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_beam_finished(dtype):
    g = torch.Generator(device=DEV).manual_seed(5)
    logits, scores = likely(g, 24, 1500, dtype), -torch.rand(3, 8, generator=g, device=DEV) * 8
    finished = torch.rand(3, 8, generator=g, device=DEV) < 0.5
    finished[1], finished[2] = True, False
    logits[8:16] = math.nan                                          # (a finished beam's logits do not count)
    got = select(logits, scores, 12, finished, end=1499)
    check(got, logits, scores, 12, finished, 1499)
    assert np.isfinite(got[0][1]).sum() == 8 and np.all(got[2][1, :8] == 1499)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_beam_logits_that_are_no_logits(bad):
    g = torch.Generator(device=DEV).manual_seed(6)
    logits, scores = likely(g, 8, 5000, "bf16"), -torch.rand(2, 4, generator=g, device=DEV)
    logits[1, 4321] = bad
    got = select(logits, scores, 8, flag=B.DEVERR_BAD_LOGITS)
    check(got, logits, scores, 8)
    assert not (got[1] == 1).any()
    scores[1, 2] = bad
    got = select(logits, scores, 8, flag=B.DEVERR_BAD_LOGITS)
    check(got, logits, scores, 8)
    assert not (got[1] == 6).any()


def test_beam_more_blocks_than_are_ranked_at_a_time():
    g = torch.Generator(device=DEV).manual_seed(8)
    logits = torch.randn(64, 150001, generator=g, device=DEV)
    scores = -torch.rand(1, 64, generator=g, device=DEV) * 3
    logits[63, 150000] = 30.0                                        # the best of all is the last
    got = select(logits, scores, 64)
    assert (got[1][0, 0], got[2][0, 0]) == (63, 150000)
    check(got, logits, scores, 64)
    # the best blocks all in one group of those that are ranked: a beam's tokens a multiple of the group's stride apart
    logits = torch.zeros(8, 150000, device=DEV)
    logits[:, ::128 * 256] = 5.0
    logits[3, ::128] = torch.linspace(1, 4, 1172, device=DEV)
    scores = torch.zeros(1, 8, device=DEV)
    check(select(logits, scores, 64), logits, scores, 64)


def test_beam_rising_and_falling_logits():
    for order in (1, -1):
        logits = (torch.arange(40000, device=DEV, dtype=torch.float32) * (order / 1000.0)).repeat(2, 1)
        scores = torch.tensor([[-0.5, -0.25]], device=DEV)
        check(select(logits, scores, 32), logits, scores, 32)


def test_beam_scores_in_place_and_many_requests():
    g = torch.Generator(device=DEV).manual_seed(12)
    logits, scores = likely(g, 3000, 700, "fp16"), -torch.rand(1500, 2, generator=g, device=DEV)
    before = scores.clone()
    ws = torch.empty(search.beam_workspace_size(logits, scores), dtype=torch.uint8, device=DEV)
    rest = [torch.empty(1500, 2, dtype=torch.int32, device=DEV) for _ in range(2)]
    best = search.beam_select(logits, scores, ws, out=search.BeamChoice(scores, *rest))
    torch.cuda.synchronize()
    assert best.scores is scores
    check([t.cpu().numpy() for t in best], logits, before, 2)


def test_beam_deterministic_and_captured_on_a_stream():
    g = torch.Generator(device=DEV).manual_seed(9)
    logits, scores = likely(g, 32, 20011, "bf16"), -torch.rand(4, 8, generator=g, device=DEV)
    ws = torch.empty(search.beam_workspace_size(logits, scores, num_out=16), dtype=torch.uint8, device=DEV)
    first = [t.clone() for t in search.beam_select(logits, scores, ws, num_out=16)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        search.beam_select(logits, scores, ws, num_out=16)
        with torch.cuda.graph(graph, stream=side):
            out = search.beam_select(logits, scores, ws, num_out=16)
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    logits.copy_(likely(g, 32, 20011, "bf16"))                       # the replay reads what is there then
    graph.replay()
    torch.cuda.synchronize()
    check([t.cpu().numpy() for t in out], logits, scores, 16)
    other = search.beam_select(logits, scores, ws, num_out=16, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, out))


def test_beam_two_calls_at_once_on_two_streams():
    g = torch.Generator(device=DEV).manual_seed(77)
    calls, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for dtype in ("bf16", "fp32"):
        logits, scores = likely(g, 40, 32003, dtype), -torch.rand(5, 8, generator=g, device=DEV)
        ws = torch.empty(search.beam_workspace_size(logits, scores, num_out=16), dtype=torch.uint8, device=DEV)
        first = [t.clone() for t in search.beam_select(logits, scores, ws, num_out=16)]
        calls.append((logits, scores, ws, first, search.BeamChoice(*(torch.empty_like(t) for t in first))))
    torch.cuda.synchronize()
    for _ in range(10):
        for (logits, scores, ws, _, out), stream in zip(calls, streams):
            search.beam_select(logits, scores, ws, num_out=16, out=out, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    for _, _, _, first, out in calls:
        assert all(torch.equal(a, b) for a, b in zip(first, out))


# ------------------------------------------------------- reordering, shared prefix

def beams_state(rng, groups, beams, width, page_size, pages):
    n = groups * beams
    tables = np.full((n, width), -1, dtype=np.int32)
    free = list(rng.permutation(pages))
    lens = np.zeros(n, dtype=np.int32)
    for g in range(groups):
        prompt = int(rng.integers(0, width * page_size // 2 + 1))
        shared = [free.pop() for _ in range(prompt // page_size)]
        for b in range(g * beams, (g + 1) * beams):
            lens[b] = min(prompt + int(rng.integers(0, width * page_size // 4 + 1)), width * page_size)
            own = [free.pop() for _ in range(-(-int(lens[b]) // page_size) - len(shared))]
            tables[b, :len(shared) + len(own)] = shared + own
    refs = np.bincount(tables[tables >= 0], minlength=pages).astype(np.int32)
    return tables, refs, lens


def parents_of(rng, groups, beams):
    p = np.concatenate([g * beams + rng.integers(0, beams, beams) for g in range(groups)]).astype(np.int32)
    p[rng.random(p.size) < 0.1] = -1
    return p


@pytest.mark.parametrize("groups,beams,width,page_size", [
    (1, 1, 1, 1), (2, 4, 3, 64), (5, 3, 17, 16), (8, 16, 130, 64), (16, 8, 1100, 8), (300, 2, 40, 64),
])
def test_reorder_and_shared_prefix(groups, beams, width, page_size):
    rng = np.random.default_rng(groups * 7 + beams)
    pages = groups * (beams + 1) * width + 5
    tables, refs, lens = beams_state(rng, groups, beams, width, page_size, pages)
    starts = np.arange(groups + 1) * beams
    n = groups * beams
    wide = torch.full((n, width + 3), -55, dtype=torch.int32, device=DEV)
    wide[:, :width] = i32(tables)
    for step in range(3):
        parents = parents_of(rng, groups, beams)
        if step == 2:
            parents = rng.integers(-1, n, n).astype(np.int32)         # any request of any other
        t, r, l = wide[:, :width], i32(refs), i32(lens)
        out_lens = torch.full((n,), -9, dtype=torch.int32, device=DEV)
        prefix = torch.full((groups,), -9, dtype=torch.int32, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = torch.full((C.reorder_workspace_size(t),), 0xFF, dtype=torch.uint8, device=DEV)
        C.pages_reorder(t, r, l, i32(parents), out_lens, ws, page_size=page_size, error_word=err)
        C.pages_shared_prefix(t, out_lens, i32(starts), prefix, page_size=page_size, error_word=err)
        torch.cuda.synchronize()
        tables, refs, lens, flag = S.reorder(tables, refs, lens, parents, page_size)
        assert int(err.item()) == 0 and not flag
        assert np.array_equal(t.cpu().numpy(), tables) and np.array_equal(r.cpu().numpy(), refs)
        assert np.array_equal(out_lens.cpu().numpy(), lens) and np.array_equal(l.cpu().numpy() >= 0, lens >= 0)
        assert np.array_equal(prefix.cpu().numpy(), S.shared_prefix(tables, lens, starts, page_size))
        assert np.all(wide[:, width:].cpu().numpy() == -55)


def test_reorder_flags_what_cannot_be():
    tables, refs = np.array([[0, 1], [2, 9], [3, -1]], dtype=np.int32), np.array([1, 1, 0, 1], dtype=np.int32)
    t, r, out_lens = i32(tables), i32(refs), i32([-1, -1, -1])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(C.reorder_workspace_size(t), dtype=torch.uint8, device=DEV)
    # request 0 becomes 1, whose second page is none of the pool's; 1 becomes 2 and gives up a page that counts 0
    C.pages_reorder(t, r, i32([4, 4, 1]), i32([1, 2, 7]), out_lens, ws, page_size=2, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == B.DEVERR_PAGE_STATE
    assert t.cpu().tolist() == [[2, 9], [3, -1], [3, -1]] and out_lens.cpu().tolist() == [4, 1, 1]
    assert r.cpu().tolist() == [0, 0, 0, 2]
    err.zero_()
    prefix = i32([7, 7])
    C.pages_shared_prefix(t, i32([5, -3, 2]), i32([0, 2, 9]), prefix, page_size=2, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == B.DEVERR_PAGE_STATE and prefix.cpu().tolist() == [4, 2]


def test_shared_prefix_of_empty_and_odd_groups():
    t = i32([[1, 2, 3], [1, 2, 4], [5, -1, -1], [1, 2, 3], [-1, -1, -1]])
    lens, prefix = i32([12, 11, 3, 12, 0]), i32([-9] * 5)
    C.pages_shared_prefix(t, lens, i32([0, 2, 2, 3, 4, 5]), prefix, page_size=4)
    torch.cuda.synchronize()
    assert prefix.cpu().tolist() == [8, 0, 0, 12, 0]
    one = i32([-9])
    C.pages_shared_prefix(t, lens, i32([-4, 99]), one, page_size=4)
    torch.cuda.synchronize()
    assert one.item() == 0
    C.pages_shared_prefix(t[:4], i32([12, 12, 0, 12]), i32([0, 4]), one, page_size=4)     # one without tokens does not count
    torch.cuda.synchronize()
    assert one.item() == 8
    C.pages_shared_prefix(i32([[1, -1, 3], [9, 9, 9]]), i32([12, 0]), i32([0, 2]), one, page_size=4)   # an entry of none ends it
    torch.cuda.synchronize()
    assert one.item() == 4


# ----------------------------------------------------------------------- slot maps

@pytest.mark.parametrize("batch,q_max,page_size,pad", [
    (1, 1, 64, 0), (3, 5, 16, 7), (128, 1, 64, 8), (40, 60, 8, 100), (1500, 3, 64, 1), (2, 5000, 100, 0), (5, 0, 64, 3),
])
def test_token_slots(batch, q_max, page_size, pad):
    rng = np.random.default_rng(batch + q_max)
    lens = rng.integers(0, 500, batch)
    new = lens + rng.integers(0, q_max + 1, batch)
    gone = rng.random(batch) < 0.2
    new[gone] = rng.integers(0, 3, gone.sum())                       # requests that end or are cut
    width = -(-int(max(new.max(), 1)) // page_size)
    tables = rng.permutation(batch * width).reshape(batch, width).astype(np.int32)
    tokens = int(np.maximum(new - lens, 0).sum()) + pad
    want = S.token_slots(lens, new, tokens, tables, page_size)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = slots.token_slots(i32(lens), i32(new), i32(tables), max_tokens=tokens, page_size=page_size, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for a, b in zip(got, want):
        assert np.array_equal(a.cpu().numpy(), b)
    assert got.slots.dtype == torch.int64
    plain = slots.token_slots(i32(lens), i32(new), max_tokens=tokens)
    assert plain.slots is None and torch.equal(plain.positions, got.positions)


def test_token_slots_flags():
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tables = i32([[3, -1], [4, 5]])
    got = slots.token_slots(i32([3, 6]), i32([6, 10]), tables, max_tokens=7, page_size=4, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == B.DEVERR_INDEX_OUT_OF_RANGE            # an entry of -1; positions past the table
    assert got.slots.cpu().tolist() == [15, -1, -1, 22, 23, -1, -1]
    err.zero_()
    got = slots.token_slots(i32([3, 2]), i32([4, 9]), tables, max_tokens=4, page_size=4, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == B.DEVERR_TOO_MANY_TOKENS and got.cum_seq_lens_q.cpu().tolist() == [0, 1, 8]
    assert got.positions.cpu().tolist() == [3, 2, 3, 4]
    err.zero_()
    got = slots.token_slots(i32([-2, 0]), i32([2, -1]), tables, max_tokens=3, page_size=4, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == B.DEVERR_PAGE_STATE and got.slots.cpu().tolist() == [12, 13, -1]
    err.zero_()
    big = 2 ** 31 - 1
    got = slots.token_slots(i32([0, 0, 0]), i32([big, big, big]), max_tokens=2, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == B.DEVERR_TOO_MANY_TOKENS and got.cum_seq_lens_q.cpu().tolist() == [0, big, big, big]
    empty = slots.token_slots(i32([]), i32([]), max_tokens=3)
    torch.cuda.synchronize()
    assert empty.cum_seq_lens_q.cpu().tolist() == [0] and empty.requests.cpu().tolist() == [-1] * 3


def test_lengths_of_the_least_number_are_no_tokens():
    least = -2**31
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = slots.token_slots(i32([5, least, 3]), i32([least, 2, 5]), i32([[1], [2], [3]]), max_tokens=6, page_size=8,
                            error_word=err)
    table, topk = slots.sparse_slots(i32([least, 3]), i32([[4], [5]]), 6, page_size=8, cum_seq_lens_q=i32([0, 3, 6]))
    torch.cuda.synchronize()
    assert int(err.item()) == B.DEVERR_PAGE_STATE and got.cum_seq_lens_q.cpu().tolist() == [0, 0, 2, 4]
    assert got.requests.cpu().tolist() == [1, 1, 2, 2, -1, -1] and got.positions.cpu().tolist() == [0, 1, 3, 4, -1, -1]
    assert got.slots.cpu().tolist() == [16, 17, 27, 28, -1, -1]
    assert topk.cpu().tolist() == [0, 0, 0, 128, 128, 128] and bool((table[:3] == -1).all())
    assert table[5, :4].cpu().tolist() == [40, 41, 42, -1]


def test_token_slots_past_32_bits():
    got = slots.token_slots(i32([70000]), i32([70003]), i32([[0, 2 ** 31 - 1]]), max_tokens=3, page_size=65536)
    torch.cuda.synchronize()
    assert got.slots.cpu().tolist() == [(2 ** 31 - 1) * 65536 + 4464 + i for i in range(3)]


@pytest.mark.parametrize("batch,q_max,keep,page_size,ratio,pad", [
    (1, 1, 0, 64, 1, 0), (3, 4, 16, 64, 4, 2), (2, 200, 33, 16, 4, 5), (64, 2, 2048, 64, 4, 1), (5, 3, 7, 100, 128, 0),
    (4, 1, 64, 1, 1, 3),
])
def test_sparse_slots(batch, q_max, keep, page_size, ratio, pad):
    rng = np.random.default_rng(batch * 3 + keep)
    q = rng.integers(1, q_max + 1, batch)
    lens = q + rng.integers(0, 2000, batch)
    lens[0] = q[0]                                                   # a request from its first token on
    cum = np.concatenate([[0], np.cumsum(q)])
    tokens = int(cum[-1]) + pad
    width, comp_width = -(-int(lens.max()) // page_size), -(-int(lens.max() // ratio + 1) // page_size)
    swa = rng.permutation(batch * width).reshape(batch, width).astype(np.int32)
    comp = rng.permutation(batch * comp_width).reshape(batch, comp_width).astype(np.int32)
    selected = rng.integers(-3, lens.max() // ratio + 2, (tokens, keep)).astype(np.int32)
    kw = dict(page_size=page_size, cum_seq_lens_q=i32(cum), compressed_tables=i32(comp), compressed_page_size=page_size,
              compress_ratio=ratio)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for how in ("selected", "first", "strided"):
        if how == "first":
            want = S.sparse_slots(lens, cum, tokens, swa, page_size, comp, page_size, ratio, keep=keep)
            got = slots.sparse_slots(i32(lens), i32(swa), tokens, num_selected=keep, error_word=err, **kw)
        else:
            want = S.sparse_slots(lens, cum, tokens, swa, page_size, comp, page_size, ratio, selected)
            if how == "selected":
                got = slots.sparse_slots(i32(lens), i32(swa), tokens, selected=i32(selected), error_word=err, **kw)
            else:
                wide = torch.full((tokens, 128 + keep + 5), -55, dtype=torch.int32, device=DEV)
                picks = i32(np.concatenate([selected, selected], axis=1))[:, :keep]
                got = slots.sparse_slots(i32(lens), i32(swa), tokens, selected=picks, sparse_indices=wide[:, :128 + keep],
                                         error_word=err, **kw)
                torch.cuda.synchronize()
                assert bool((wide[:, 128 + keep:] == -55).all())
        torch.cuda.synchronize()
        assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
    assert int(err.item()) == 0


@pytest.mark.parametrize("pad,keep,tokens", [(0, 512, 40), (0, 1040, 3), (3, 37, 300)])
def test_sparse_slots_of_a_selection_in_place(pad, keep, tokens):
    rng = np.random.default_rng(17)
    lens, swa = rng.integers(tokens, 900, 1).astype(np.int32), rng.permutation(20).astype(np.int32)[None]
    comp = rng.permutation(40).astype(np.int32)[None]
    picks = rng.integers(-1, 300, (tokens, keep)).astype(np.int32)
    kw = dict(page_size=64, compressed_tables=i32(comp), compressed_page_size=16, compress_ratio=4)
    want = slots.sparse_slots(i32(lens), i32(swa), tokens, selected=i32(picks), **kw)
    table = torch.full((tokens, 128 + keep + pad), -7, dtype=torch.int32, device=DEV)
    table[:, 128:128 + keep] = i32(picks)
    got = slots.sparse_slots(i32(lens), i32(swa), tokens, selected=table[:, 128:128 + keep],
                             sparse_indices=table[:, :128 + keep], **kw)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and bool((table[:, 128 + keep:] == -7).all())


def test_sparse_slots_flags_and_uniform_batches():
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    swa, comp = i32([[3, -1], [2 ** 30, 1]]), i32([[0], [1]])
    got, topk = slots.sparse_slots(i32([3, 9]), swa, 4, page_size=4, selected=i32([[0, 5], [5, 0], [9, 9], [7, -1]]),
                                   compressed_tables=comp, compressed_page_size=4, compress_ratio=1, error_word=err)
    torch.cuda.synchronize()
    want = S.sparse_slots([3, 9], [0, 2, 4], 4, swa.cpu().numpy(), 4, comp.cpu().numpy(), 4, 1,
                          np.array([[0, 5], [5, 0], [9, 9], [7, -1]]))
    assert np.array_equal(got.cpu().numpy(), want[0]) and np.array_equal(topk.cpu().numpy(), want[1])
    assert int(err.item()) == B.DEVERR_INDEX_OUT_OF_RANGE
    # a request of fewer tokens than it is said to have new ones
    got, topk = slots.sparse_slots(i32([1]), i32([[0]]), 3, page_size=4)
    torch.cuda.synchronize()
    assert topk.cpu().tolist() == [0, 0, 128] and bool((got[:2] == -1).all()) and got[2, :2].cpu().tolist() == [0, -1]


def test_sparse_slots_feed_the_sparse_decode():
    """The index table as the decode takes it: the same output as for rows gathered by hand."""
    g = torch.Generator(device=DEV).manual_seed(2)
    page, batch, keep, ratio = 64, 3, 64, 4
    lens, new = [300, 40, 700], [302, 42, 702]
    swa = torch.randperm(batch * 12, generator=g, device=DEV).to(torch.int32).view(batch, 12)
    comp = torch.randperm(batch * 3, generator=g, device=DEV).to(torch.int32).view(batch, 3)
    pool, comp_pool = (torch.randn(n * page, 512, generator=g, device=DEV).to(torch.bfloat16) for n in (batch * 12, batch * 3))
    step = slots.token_slots(i32(lens), i32(new), swa, max_tokens=6, page_size=page)
    picks = torch.randint(-1, 170, (6, keep), generator=g, device=DEV, dtype=torch.int32)
    indices, topk = slots.sparse_slots(i32(new), swa, 6, page_size=page, cum_seq_lens_q=step.cum_seq_lens_q, selected=picks,
                                       compressed_tables=comp, compressed_page_size=page, compress_ratio=ratio)
    q = torch.randn(6, 64, 512, generator=g, device=DEV).to(torch.bfloat16)
    ws = torch.empty(B.workspace_size(q, indices, i32(new)) + 256, dtype=torch.uint8, device=DEV)
    out, lse = B.sparse_mla_decode(q, pool, ws, indices, comp_pool, topk, i32(new), cum_seq_lens_q=step.cum_seq_lens_q,
                                   bmm1_scale=512 ** -0.5)
    torch.cuda.synchronize()
    t = 0
    for b in range(batch):
        for pos in range(lens[b], new[b]):
            j = torch.arange(max(0, pos - 127), pos + 1, device=DEV)
            rows = [pool[swa[b, j // page].long() * page + j % page]]
            c = picks[t].long()
            c = c[(c >= 0) & (c < (pos + 1) // ratio)]
            rows.append(comp_pool[comp[b, c // page].long() * page + c % page])
            kv = torch.cat(rows).double()
            x = q[t].double() @ kv.T * 512 ** -0.5
            assert torch.allclose(torch.softmax(x, 1) @ kv, out[t].double(), atol=2e-2, rtol=0)
            assert torch.allclose(torch.logsumexp(x, 1) / math.log(2), lse[t].double(), atol=1e-3, rtol=0)
            t += 1


def test_calls_on_another_stream_and_captured():
    rng = np.random.default_rng(4)
    tables, refs, lens = beams_state(rng, 4, 4, 20, 16, 600)
    parents = parents_of(rng, 4, 4)
    t, r, l, p = i32(tables), i32(refs), i32(lens), i32(parents)
    t0, r0 = t.clone(), r.clone()
    out_lens, prefix, ws = i32(np.zeros(16)), i32(np.zeros(4)), torch.empty(C.reorder_workspace_size(t), dtype=torch.uint8, device=DEV)
    starts, total = i32(np.arange(5) * 4), int(np.maximum(lens, 0).sum())

    def step():
        C.pages_reorder(t, r, l, p, out_lens, ws, page_size=16)
        C.pages_shared_prefix(t, out_lens, starts, prefix, page_size=16)
        s = slots.token_slots(l, out_lens, t, max_tokens=total, page_size=16)
        return s, slots.sparse_slots(out_lens, t, total, page_size=16, cum_seq_lens_q=s.cum_seq_lens_q)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        s, (table, topk) = step()
    for _ in range(2):
        t.copy_(t0)
        r.copy_(r0)
        graph.replay()
    torch.cuda.synchronize()
    want_t, want_r, want_l, _ = S.reorder(tables, refs, lens, parents, 16)
    assert np.array_equal(t.cpu().numpy(), want_t) and np.array_equal(r.cpu().numpy(), want_r)
    assert np.array_equal(prefix.cpu().numpy(), S.shared_prefix(want_t, want_l, np.arange(5) * 4, 16))
    want = S.token_slots(lens, want_l, total, want_t, 16)
    for a, b in zip(s, want):
        assert np.array_equal(a.cpu().numpy(), b)
    want = S.sparse_slots(want_l, want[0], total, want_t, 16)
    assert np.array_equal(table.cpu().numpy(), want[0]) and np.array_equal(topk.cpu().numpy(), want[1])
