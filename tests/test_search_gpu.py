"""A search over the paged latent cache, all calls of a step together: choice, reordering, pages for the new tokens, slot
maps, append, shared prefixes, attention; against what each beam's history says."""
import math

import numpy as np
import pytest
import torch

import cache_reference as R
import step_reference as S
from sparse_mla_decode_token_gb300 import binding as B
from sparse_mla_decode_token_gb300 import cache as C
from sparse_mla_decode_token_gb300 import search, slots

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE, BLOCK, PAGES, WIDTH = 32, 16, 400, 16
VOCAB, HEADS = 900, 16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_decode_token_gb300 import build
    build.build()
    B.lib()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Search:
    """Device state of a few requests with some beams each, and the calls of a step on it."""

    def __init__(self, requests, beams, seed):
        n = self.n = requests * beams
        self.requests, self.beams = requests, beams
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.rows = torch.zeros(PAGES, PAGE, 512, dtype=torch.float8_e4m3fn, device=DEV)
        self.cscales = torch.ones(PAGES, PAGE // BLOCK, device=DEV)
        self.tables = torch.full((n, WIDTH), -1, dtype=torch.int32, device=DEV)
        self.counts, self.err = i32(np.zeros(PAGES)), i32([0])
        self.lens, self.chosen, self.grown = i32(np.zeros(n)), i32(np.zeros(n)), i32(np.zeros(n))
        self.starts, self.prefix = i32(np.arange(requests + 1) * beams), i32(np.zeros(requests))
        self.pages_ws = torch.empty(C.pages_workspace_size(self.tables, self.counts, PAGE), dtype=torch.uint8, device=DEV)
        self.reorder_ws = torch.empty(C.reorder_workspace_size(self.tables), dtype=torch.uint8, device=DEV)
        self.moves = C.new_moves(n, DEV)
        self.scores = torch.full((requests, beams), -math.inf, device=DEV)
        self.scores[:, 0] = 0.0                            # a search's first step has one beam
        self.embed = torch.randn(VOCAB, 512, generator=self.gen, device=DEV).to(torch.bfloat16)
        self.logits = torch.empty(n, VOCAB, dtype=torch.bfloat16, device=DEV)
        self.q = torch.empty(n, HEADS, 512, dtype=torch.bfloat16, device=DEV)
        self.beam_ws = torch.empty(search.beam_workspace_size(self.logits, self.scores), dtype=torch.uint8, device=DEV)
        self.prefix_ws = torch.empty(C.prefix_workspace_size(self.q, self.rows, self.cscales, self.tables, self.lens,
                                                             group_starts=self.starts, cum_seq_lens_q=i32(np.zeros(n + 1))),
                                     dtype=torch.uint8, device=DEV)

    def prompts(self, lens):
        """Prompts into each request's first beam."""
        new = np.zeros(self.n, dtype=np.int32)
        new[::self.beams] = lens
        x = torch.randn(int(new.sum()), 512, generator=self.gen, device=DEV).to(torch.bfloat16)
        self.grown.copy_(i32(new))
        C.pages_resize(self.tables, self.counts, self.lens, self.grown, self.pages_ws, page_size=PAGE, moves=self.moves,
                       error_word=self.err)
        step = slots.token_slots(self.lens, self.grown, self.tables, max_tokens=x.shape[0], page_size=PAGE, error_word=self.err)
        C.append(x, self.rows, self.cscales, self.tables, self.grown, cum_seq_lens_q=step.cum_seq_lens_q, error_word=self.err)
        self.lens.copy_(self.grown)
        return np.split(x.float().cpu().numpy(), np.cumsum(lens)[:-1])

    def step(self):
        best = search.beam_select(self.logits, self.scores, self.beam_ws, error_word=self.err)
        C.pages_reorder(self.tables, self.counts, self.lens, best.parents, self.chosen, self.reorder_ws, page_size=PAGE,
                        error_word=self.err)
        torch.add(self.chosen, (self.chosen > 0).int(), out=self.grown)
        C.pages_resize(self.tables, self.counts, self.chosen, self.grown, self.pages_ws, page_size=PAGE, moves=self.moves,
                       error_word=self.err)
        C.pages_copy([self.rows, self.cscales], self.moves, error_word=self.err)
        slot = slots.token_slots(self.chosen, self.grown, self.tables, max_tokens=self.n, page_size=PAGE, error_word=self.err)
        tokens = best.tokens.view(-1)[slot.requests.clamp(min=0)].clamp(min=0)
        C.append(self.embed[tokens], self.rows, self.cscales, self.tables, self.grown, cum_seq_lens_q=slot.cum_seq_lens_q,
                 error_word=self.err)
        C.pages_shared_prefix(self.tables, self.grown, self.starts, self.prefix, page_size=PAGE, error_word=self.err)
        out = C.prefix_attention(self.q, self.rows, self.cscales, self.tables, self.grown, self.prefix_ws,
                                 group_starts=self.starts, prefix_lens=self.prefix, cum_seq_lens_q=slot.cum_seq_lens_q,
                                 bmm1_scale=0.05, error_word=self.err)
        self.lens.copy_(self.grown)
        self.scores.copy_(best.scores)
        return best, slot, out


@pytest.mark.parametrize("captured", [False, True])
def test_search(captured):
    requests, beams = 3, 4
    s = Search(requests, beams, 7)
    history = [[] for _ in range(s.n)]
    for r, x in enumerate(s.prompts([70, 33, 160])):
        history[r * beams] = list(x)
    rng = np.random.default_rng(3)
    embed = s.embed.float().cpu().numpy()
    fill = lambda: (s.logits.copy_(torch.randn(s.n, VOCAB, generator=s.gen, device=DEV) * 3),
                    s.q.copy_(torch.randn(s.n, HEADS, 512, generator=s.gen, device=DEV)))
    run, graph = s.step, None
    for k in range(9):
        fill()
        scores, logits = s.scores.cpu().numpy(), s.logits.double().cpu().numpy()
        if captured and k == 2:                            # the rest of the search from one graph
            graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=side):
                results = s.step()
            run = lambda: (graph.replay(), results)[1]
        best, slot, (out, lse) = run()
        torch.cuda.synchronize()
        assert int(s.err.item()) == 0
        want = S.beam_best(S.beam_scores(logits, scores), beams)
        assert np.array_equal(best.parents.cpu().numpy(), want[1]) and np.array_equal(best.tokens.cpu().numpy(), want[2])
        parents, tokens = want[1].reshape(-1), want[2].reshape(-1)
        history = [history[p] + [embed[t]] if p >= 0 else [] for p, t in zip(parents, tokens)]
        lens, tables = s.lens.cpu().numpy(), s.tables.cpu().numpy()
        assert lens.tolist() == [len(h) for h in history]
        assert np.array_equal(s.counts.cpu().numpy(), np.bincount(tables[tables >= 0], minlength=PAGES))
        assert np.array_equal(s.prefix.cpu().numpy(), S.shared_prefix(tables, lens, np.arange(requests + 1) * beams, PAGE))
        live = [b for b in range(s.n) if lens[b] > 0]
        cum = np.concatenate([[0], np.cumsum(lens > 0)])
        assert np.array_equal(slot.cum_seq_lens_q.cpu().numpy(), cum)
        assert slot.requests.cpu().tolist() == live + [-1] * (s.n - len(live))
        cache = R.Cache(s.rows.view(torch.uint8).cpu().numpy(), s.cscales.cpu().numpy(), tables, lens, cum=cum)
        for b in live:
            # E4M3 within 2^-4 of the value, twice where a block's scale grew; its subnormals by 2^-10 of the scale
            held = np.stack([cache.row(b, j) for j in range(lens[b])])
            x = np.stack(history[b])
            step = max(cache.scales[cache.page(b, j), j % PAGE // BLOCK] for j in range(lens[b])) * 2.0 ** -9
            assert np.all(np.abs(held - x) <= 2.0 ** -3 * np.abs(x) + step)
        o, l, tol_o, tol_l = R.window(cache, s.q.double().cpu().numpy()[:len(live)], window=1 << 30, bmm1=0.05)
        n = len(live)
        assert np.all(np.abs(out.double().cpu().numpy()[:n] - o) <= tol_o) and np.all(np.abs(lse.double().cpu().numpy()[:n] - l) <= tol_l)
    assert len(set(parents.tolist())) > 1 and s.prefix.cpu().numpy().min() > 0
