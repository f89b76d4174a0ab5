"""The search step of the README as it stands there, run on beams of which one request has fewer continuations than
places."""
import math
import os
import re

import numpy as np
import pytest
import torch

from sparse_mla_decode_token_gb300 import cache as C
from test_search_gpu import DEV, HEADS, VOCAB, Search, built, i32  # noqa: F401  (built: the library, once a module)

pytestmark = pytest.mark.gpu


def search_step():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    return re.search(r"^A step of a search on it.*?```python\n(.*?)```", text, re.S | re.M).group(1).replace("page_size=64", "page_size=32")


def test_the_search_step():
    requests, beams, eos = 2, 4, VOCAB - 1
    s = Search(requests, beams, 5)
    s.prompts([70, 100])
    embed = torch.randn(VOCAB, 512, generator=s.gen, device=DEV).to(torch.bfloat16)
    modelled = []

    def model(tokens, positions):
        modelled.append((tokens.clone(), positions.clone()))
        return embed[tokens.clamp(min=0)], torch.randn(s.n, HEADS, 512, generator=s.gen, device=DEV).to(torch.bfloat16)

    swa = i32(np.arange(s.n * 16).reshape(s.n, 16))
    space = dict(torch=torch, cache=C, model=model, beam_ws=s.beam_ws, eos=eos, tables=s.tables, counts=s.counts, lens=s.lens,
                 chosen_lens=s.chosen, reorder_ws=s.reorder_ws, new_lens=s.grown, ws=s.pages_ws, moves=s.moves, rows=s.rows,
                 scales=s.cscales, T=s.n, group_starts=s.starts, prefix_lens=s.prefix, prefix_ws=s.prefix_ws, scale=0.05,
                 swa_tables=swa, comp_tables=swa, picks=i32(np.zeros((s.n, 4))), scores=s.scores,
                 done=torch.zeros(requests, beams, dtype=torch.bool, device=DEV))
    source = search_step()
    for k in range(3):
        logits = torch.randn(s.n, VOCAB, generator=s.gen, device=DEV) * 3
        logits[:, eos] = -math.inf
        if k == 0:
            logits[beams, 2:] = -math.inf                  # the second request's first beam has two continuations
        elif k == 1:
            logits[beams:, 1:] = -math.inf                 # and each of those one
        space["logits"] = logits.to(torch.bfloat16)
        exec(source, space)
        torch.cuda.synchronize()
        live = [4, 2] if k < 2 else [4, 4]
        lens = s.grown.view(requests, beams).cpu().tolist()
        assert lens == [[71 + k] * 4, [101 + k] * live[1] + [0] * (4 - live[1])]
        assert s.prefix.cpu().tolist() == [64, 96]         # the prompts' whole pages: empty places do not end them
        tokens, positions = modelled[-1]
        best, n = space["best"], sum(live)
        of = [b for b in range(s.n) if s.grown[b] > 0]
        assert torch.equal(tokens[:n], best.tokens.view(-1)[of]) and bool((tokens[:n] >= 0).all())
        assert positions[:n].cpu().tolist() == [int(s.grown[b]) - 1 for b in of] and bool((positions[n:] == -1).all())
        out, lse = space["out"], space["lse"]
        assert bool(out[:n].isfinite().all()) and bool(lse[:n].isfinite().all())
        assert space["topk"][:n].min() >= 128 and bool((space["topk"][n:] == 0).all())
        tables = s.tables.cpu().numpy()
        assert np.array_equal(s.counts.cpu().numpy(), np.bincount(tables[tables >= 0], minlength=s.counts.numel()))
        space["scores"] = best.scores
        s.lens.copy_(s.grown)
