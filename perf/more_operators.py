"""Cases of a search or sampling step: what a server does around the decode when
requests share a prompt.

* ``prefix``: attention of a batch whose groups share a long prefix of the paged
  latent cache (E4M3 rows, one fp32 scale per block of tokens);
* ``beam``: the best continuations over a request's beams and the vocabulary;
* ``reorder``: page tables and counts after such a choice, and how much of a
  prefix the beams then share;
* ``slots``: a step's offsets, positions and physical slots from request
  lengths, and the index tables of the sparse decode.

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through the package's public calls.
"""
import math

import torch

own = False

PAGE = 64          # tokens per page
BLOCK = 16         # tokens that share a scale
DIM = 512          # latent row
WINDOW = 128       # sliding-window columns of an index table
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # four samples of one short prompt, a rank with 16 heads
        dict(name="prefix tiny", kind="prefix", groups=1, members=4, q_max=1, heads=16, prefix_min=500, prefix_max=520,
             own_max=64),
        # eight samples of each of eight prompts, a rank with 16 heads
        dict(name="prefix samples", kind="prefix", groups=8, members=8, q_max=1, heads=16, prefix_min=4096, prefix_max=8192,
             own_max=512),
        # wide searches over four long documents, a rank with 8 heads
        dict(name="prefix search", kind="prefix", groups=4, members=32, q_max=1, heads=8, prefix_min=16000, prefix_max=16384,
             own_max=256),
        # speculative decode behind a system prompt, all 128 heads, 1 to 4 tokens a request
        dict(name="prefix varlen", kind="prefix", groups=16, members=4, q_max=4, heads=128, prefix_min=1000, prefix_max=2048,
             own_max=512),
        # one user's search with four beams over a small vocabulary
        dict(name="beam tiny", kind="beam", batch=1, beams=4, vocab=32000, dtype="bf16", keep=4),
        # a decode batch of searches, twice as many kept as there are beams
        dict(name="beam decode", kind="beam", batch=64, beams=8, vocab=128000, dtype="bf16", keep=16),
        # few wide searches, fp32 logits, an odd vocabulary
        dict(name="beam wide", kind="beam", batch=8, beams=32, vocab=151001, dtype="fp32", keep=64),
        # a small server's beams change places
        dict(name="reorder small", kind="reorder", groups=4, beams=4, max_pages=64, pages=1024),
        # a thousand beams over tables of a thousand pages
        dict(name="reorder server", kind="reorder", groups=64, beams=16, max_pages=1024, pages=327680),
        # one token of each request of a decode batch, 2048 selected rows each
        dict(name="slots decode", kind="slots", batch=128, q_max=1, ctx_min=4096, ctx_max=32768, selected=2048, ratio=4),
        # chunks of prompts, 512 selected rows a token
        dict(name="slots prompts", kind="slots", batch=8, q_max=1536, ctx_min=1536, ctx_max=9000, selected=512, ratio=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prefix", "prefix", "prefix", "beam", "beam", "reorder", "slots"])
    if kind == "prefix":
        groups, members, heads = _log(rng, 1, 16), _log(rng, 1, 48), rng.choice([8, 16, 32, 64, 128, rng.randint(1, 128)])
        q_max = rng.choice([1, 1, 1, 2, 3, 4])
        # tokens x heads x rows stays at or under the largest listed case's, the rows of all tokens at what their plain form can hold
        most = min((160 * 128 * 1536) // heads, 1 << 22) // (groups * members * q_max)
        prefix_max = _log(rng, 1, max(2, min(16384, most)))
        return dict(kind=kind, groups=groups, members=members, q_max=q_max, heads=heads,
                    prefix_min=max(1, prefix_max // rng.randint(1, 4)), prefix_max=prefix_max,
                    own_max=q_max + _log(rng, 1, max(1, min(512, most))))
    if kind == "beam":
        batch, beams, vocab = _log(rng, 1, 64), _log(rng, 1, 32), _log(rng, 500, 152000)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        while batch * beams * vocab * (2 if dtype == "fp32" else 1) > 64 * 8 * 128000:
            batch = (batch + 1) // 2
            vocab = vocab * 2 // 3
        return dict(kind=kind, batch=batch, beams=beams, vocab=vocab, dtype=dtype, keep=min(64, beams * rng.choice([1, 2])))
    if kind == "reorder":
        groups, beams, max_pages = _log(rng, 1, 64), _log(rng, 1, 16), _log(rng, 4, 1024)
        return dict(kind=kind, groups=groups, beams=beams, max_pages=max_pages,
                    pages=groups * (beams + 1) * max_pages + rng.randint(1, 1000))
    batch = _log(rng, 1, 256)
    q_max = _log(rng, 1, max(1, 12288 // batch))
    ctx_min = q_max + _log(rng, 1, 4096)
    return dict(kind=kind, batch=batch, q_max=q_max, ctx_min=ctx_min, ctx_max=ctx_min + _log(rng, 1, 16384),
                selected=_log(rng, 16, max(16, min(2048, 6000000 // (batch * q_max)))), ratio=rng.choice([1, 4, 4, 128]))


# ------------------------------------------------------------------ the inputs

def _lengths(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int64)


def _spread(g, n, lo, hi):
    """n numbers over lo .. hi, the same ones for every seed, in an order of the seed's."""
    return lo + (torch.arange(1, n + 1) * 40503 % (hi - lo + 1))[torch.randperm(n, generator=g)]


def _i32(t):
    return t.to(torch.int32).cuda()


def _cum(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])


def _shared_tables(g, lens, shared, first, max_pages, pages):
    """Random distinct pages for each request's tokens; the first ``shared`` columns are the ones of its group's first
    request; -1 behind the last."""
    columns = torch.arange(max_pages)[None, :]
    held = columns < ((lens + PAGE - 1) // PAGE)[:, None]
    theirs = held & (columns < shared[:, None]) & (torch.arange(lens.numel()) != first)[:, None]
    tables = torch.full((lens.numel(), max_pages), -1, dtype=torch.int64)
    mine = held & ~theirs
    tables[mine] = torch.randperm(pages, generator=g)[: int(mine.sum())]
    return torch.where(theirs, tables[first], tables)


def _filled_cache(gd, pages):
    """Pages as they stand in a running server: unit normal rows, each token with a magnitude of its own; block scales are
    powers of two that fit the block's largest value."""
    rows = torch.empty((pages, PAGE, DIM), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((pages, PAGE // BLOCK), dtype=torch.float32, device="cuda")
    for p in range(0, pages, 2048):
        n = min(2048, pages - p)
        x = torch.randn((n, PAGE // BLOCK, BLOCK, DIM), generator=gd, device="cuda")
        x = x * torch.exp2(torch.randn((n, PAGE // BLOCK, BLOCK, 1), generator=gd, device="cuda") * 0.5)
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448.0)))
        rows[p:p + n] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(n, PAGE, DIM)
        scales[p:p + n] = s
    return rows, scales


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    {"prefix": _prepare_prefix, "beam": _prepare_beam, "reorder": _prepare_reorder, "slots": _prepare_slots}[case["kind"]](s, g, gd)
    return s


def _prepare_prefix(s, g, gd):
    groups, members = s["groups"], s["members"]
    n = groups * members
    prefix = _spread(g, groups, s["prefix_min"], s["prefix_max"])
    q_lens = _spread(g, n, 1, s["q_max"])
    own_tokens = torch.maximum(_spread(g, n, 1, s["own_max"]), q_lens)
    group = torch.arange(n) // members
    lens = prefix[group] + own_tokens
    max_pages = -(-int(s["prefix_max"] + s["own_max"]) // PAGE)
    shared = prefix[group] // PAGE
    pages = groups * (-(-s["prefix_max"] // PAGE)) + n * (s["own_max"] // PAGE + 2)
    s["tables"] = _i32(_shared_tables(g, lens, shared, group * members, max_pages, pages))
    s["seq_lens"], s["prefix"] = _i32(lens), _i32(prefix)
    s["starts"] = _i32(torch.arange(groups + 1) * members)
    s["cum"] = _i32(_cum(q_lens))
    s["tokens"], s["ctx"] = int(q_lens.sum()), int(lens.max())
    s["rows"], s["scales"] = _filled_cache(gd, pages)
    s["q"] = torch.randn((s["tokens"], s["heads"], DIM), generator=gd, device="cuda").to(torch.bfloat16)
    s["sinks"] = torch.randn((s["heads"],), generator=gd, device="cuda")
    s["scale"] = 1.0 / math.sqrt(DIM)
    if own:
        from sparse_mla_decode_token_gb300 import cache
        s["workspace"] = torch.empty(cache.prefix_workspace_size(s["q"], s["rows"], s["scales"], s["tables"], s["seq_lens"],
                                                                 group_starts=s["starts"], cum_seq_lens_q=s["cum"]),
                                     dtype=torch.uint8, device="cuda")


def _prepare_beam(s, g, gd):
    batch, beams, vocab = s["batch"], s["beams"], s["vocab"]
    # a few likely tokens a beam over a broad rest, as a language model's logits are
    x = torch.randn((batch * beams, vocab), generator=gd, device="cuda") * 2.0
    likely = torch.randint(0, vocab, (batch * beams, 40), generator=gd, device="cuda")
    x.scatter_add_(1, likely, torch.rand(likely.shape, generator=gd, device="cuda") * 12.0)
    s["logits"] = x.to(DTYPES[s["dtype"]])
    s["scores"] = -torch.rand((batch, beams), generator=gd, device="cuda").mul_(30.0).cumsum(1) / beams
    s["finished"] = torch.rand((batch, beams), generator=gd, device="cuda") < 0.1
    s["end"] = vocab - 1
    if own:
        from sparse_mla_decode_token_gb300 import search
        s["workspace"] = torch.empty(search.beam_workspace_size(s["logits"], s["scores"], num_out=s["keep"]),
                                     dtype=torch.uint8, device="cuda")


def _prepare_reorder(s, g, gd):
    groups, beams, width = s["groups"], s["beams"], s["max_pages"]
    n = groups * beams
    group = torch.arange(n) // beams
    prompt = _spread(g, groups, max(1, width * PAGE // 4), max(1, width * PAGE * 3 // 4))
    lens = (prompt + _spread(g, groups, 1, width * PAGE // 4))[group]
    # beams share their prompt's whole pages
    s["tables0"] = _i32(_shared_tables(g, lens, (prompt // PAGE)[group], group * beams, width, s["pages"]))
    s["lens"] = _i32(lens)
    flat = s["tables0"][s["tables0"] >= 0].long()
    s["refs0"] = torch.bincount(flat, minlength=s["pages"]).to(torch.int32)
    s["tables"], s["refs"] = s["tables0"].clone(), s["refs0"].clone()
    # the chosen beams' parents; one place in 32 has no continuation and ends
    parent = group * beams + torch.randint(0, beams, (n,), generator=g)
    parent[torch.rand(n, generator=g) < 1 / 32] = -1
    s["parents"] = _i32(parent)
    s["starts"] = _i32(torch.arange(groups + 1) * beams)
    s["out_lens"], s["out_prefix"] = _i32(torch.zeros(n)), _i32(torch.zeros(groups))
    if own:
        from sparse_mla_decode_token_gb300 import cache
        s["workspace"] = torch.empty(cache.reorder_workspace_size(s["tables"]), dtype=torch.uint8, device="cuda")


def _prepare_slots(s, g, gd):
    n, ratio = s["batch"], s["ratio"]
    q_lens = _spread(g, n, 1 if s["q_max"] <= 4 else -(-s["q_max"] // 3), s["q_max"])
    lens = torch.maximum(_lengths(g, n, s["ctx_min"], s["ctx_max"]), q_lens)
    tokens = int(q_lens.sum())
    s["tokens"] = tokens + tokens % 8                  # the batch padded to a size that was captured once
    s["lens"], s["new_lens"] = _i32(lens - q_lens), _i32(lens)
    width = -(-max(s["ctx_max"], s["q_max"]) // PAGE)
    comp_width = -(-max(1, s["ctx_max"] // ratio) // PAGE)
    none = torch.zeros(n, dtype=torch.int64)
    s["tables"] = _i32(_shared_tables(g, lens, none, torch.arange(n), width, n * width))
    s["comp_tables"] = _i32(_shared_tables(g, lens // ratio, none, torch.arange(n), comp_width, n * comp_width))
    # compressed positions that an indexer chose, in any order, -1 behind the last
    limit = torch.ones(s["tokens"], dtype=torch.int64)
    b = torch.repeat_interleave(torch.arange(n), q_lens)
    pos = torch.arange(tokens) - _cum(q_lens)[b] + (lens - q_lens)[b]
    limit[:tokens] = (pos + 1) // ratio
    limit = limit.cuda()
    pick = (torch.rand((s["tokens"], s["selected"]), generator=gd, device="cuda", dtype=torch.float64) * limit[:, None]).long()
    count = torch.randint(0, s["selected"] + 1, (s["tokens"],), generator=gd, device="cuda").minimum(limit)
    s["picks"] = torch.where(torch.arange(s["selected"], device="cuda")[None, :] < count[:, None], pick,
                             torch.full_like(pick, -1)).to(torch.int32)


# -------------------------------------------------------------- the plain forms

def _prefix(s):
    t = torch.arange(s["tokens"], device="cuda")
    cum, lens, starts = s["cum"].long(), s["seq_lens"].long(), s["starts"].long()
    b = torch.searchsorted(cum, t, right=True) - 1
    pos = lens[b] - (cum[b + 1] - cum[b]) + (t - cum[b])
    group = torch.searchsorted(starts, b, right=True) - 1
    j = torch.arange(s["ctx"], device="cuda")[None, :]
    of = torch.where(j < s["prefix"].long()[group][:, None], starts[group][:, None], b[:, None])
    seen = j <= pos[:, None]
    at = j.minimum(pos[:, None])
    page = s["tables"][of, at // PAGE].long()
    kv = s["rows"][page, at % PAGE].float() * s["scales"][page, at % PAGE // BLOCK][..., None]
    logits = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * s["scale"]          # [T, H, ctx]
    logits = logits.masked_fill(~seen[:, None, :], -math.inf)
    m = logits.amax(dim=2, keepdim=True)
    p = torch.exp(logits - m)
    total = p.sum(dim=2, keepdim=True)
    out = torch.matmul(p, kv) / (total + torch.exp(s["sinks"][None, :, None] - m))
    lse = (m + torch.log(total)).squeeze(2) / math.log(2.0)
    return out.to(torch.bfloat16), lse


def _beam(s):
    batch, beams, vocab, keep = s["batch"], s["beams"], s["vocab"], s["keep"]
    x = s["logits"].double()
    m = x.amax(dim=1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(dim=1, keepdim=True))
    done = s["finished"].view(-1, 1)
    total = (x - lse) + s["scores"].double().view(-1, 1)
    total = total.masked_fill(done, -math.inf)
    total[:, s["end"]] = torch.where(done[:, 0], s["scores"].double().view(-1), total[:, s["end"]])
    best, at = torch.sort(total.view(batch, beams * vocab), dim=1, descending=True, stable=True)
    best, at = best[:, :keep], at[:, :keep]
    parents = at // vocab + beams * torch.arange(batch, device="cuda")[:, None]
    none = best == -math.inf
    return (best.float(), parents.masked_fill(none, -1).to(torch.int32), (at % vocab).masked_fill(none, -1).to(torch.int32))


def _reorder(s):
    parent, lens, width = s["parents"].long(), s["lens"].long(), s["max_pages"]
    columns = torch.arange(width, device="cuda")[None, :]
    held = columns < ((lens + PAGE - 1) // PAGE)[:, None]
    gone = s["tables"][held].long()
    s["refs"].index_add_(0, gone, -torch.ones_like(gone, dtype=torch.int32))
    p = parent.clamp(min=0)
    s["out_lens"].copy_(torch.where(parent >= 0, lens[p], torch.zeros_like(p)))
    use = held[p] & (parent >= 0)[:, None]
    s["tables"].copy_(torch.where(use, s["tables"][p], torch.full_like(s["tables"], -1)))
    got = s["tables"][use].long()
    s["refs"].index_add_(0, got, torch.ones_like(got, dtype=torch.int32))
    # tokens of the leading pages that all the group's requests with tokens hold
    rows = s["tables"].view(s["groups"], s["beams"], width)
    n = s["out_lens"].long().view(s["groups"], s["beams"])
    live = n > 0
    lead = live.to(torch.int32).argmax(dim=1)
    first = rows.gather(1, lead[:, None, None].expand(-1, 1, width))
    same = ((rows == first) | ~live[:, :, None]).all(dim=1)
    full = torch.where(live, n, torch.full_like(n, width * PAGE)).amin(dim=1) // PAGE
    same &= columns < full[:, None]
    columns_shared = same.to(torch.int64).cumprod(dim=1).sum(dim=1)
    s["out_prefix"].copy_(torch.where(live.any(dim=1), columns_shared * PAGE, torch.zeros_like(full)))


def _slots(s):
    tokens, n = s["tokens"], s["batch"]
    old, new = s["lens"].long(), s["new_lens"].long()
    cum = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), (new - old).clamp(min=0).cumsum(0)])
    t = torch.arange(tokens, device="cuda")
    real = t < cum[-1]
    b = (torch.searchsorted(cum, t, right=True) - 1).clamp(max=n - 1)
    pos = old[b] + t - cum[b]
    at = pos.clamp(min=0, max=s["tables"].shape[1] * PAGE - 1)
    slot = s["tables"][b, at // PAGE].long() * PAGE + at % PAGE
    none = torch.full_like(t, -1)
    request, position, slot = torch.where(real, b, none), torch.where(real, pos, none), torch.where(real, slot, none)
    # the index table: the last 128 tokens' rows, then the selected compressed rows
    lo = (pos - WINDOW + 1).clamp(min=0)
    j = lo[:, None] + torch.arange(WINDOW, device="cuda")[None, :]
    seen = real[:, None] & (j <= pos[:, None])
    j = j.minimum(at[:, None])
    window = torch.where(seen, s["tables"][b[:, None], j // PAGE].long() * PAGE + j % PAGE, torch.full_like(j, -1))
    c = s["picks"].long()
    ok = real[:, None] & (c >= 0) & (c < ((pos + 1) // s["ratio"])[:, None])
    c = torch.where(ok, c, torch.zeros_like(c))
    rows = s["comp_tables"][b[:, None], c // PAGE].long() * PAGE + c % PAGE
    rows = torch.where(ok, rows, torch.full_like(rows, -1))
    last = torch.where(ok, torch.arange(1, s["selected"] + 1, device="cuda")[None, :], torch.zeros_like(c)).amax(dim=1)
    topk = torch.where(real, WINDOW + last, torch.zeros_like(last))
    return (cum.to(torch.int32), request.to(torch.int32), position.to(torch.int32), slot,
            torch.cat([window, rows], dim=1).to(torch.int32), topk.to(torch.int32))


# ------------------------------------------------------------------------ a pass

def run(s):
    kind = s["kind"]
    if kind == "prefix":
        if own:
            from sparse_mla_decode_token_gb300 import cache
            return cache.prefix_attention(s["q"], s["rows"], s["scales"], s["tables"], s["seq_lens"], s["workspace"],
                                          group_starts=s["starts"], prefix_lens=s["prefix"], cum_seq_lens_q=s["cum"],
                                          sinks=s["sinks"], bmm1_scale=s["scale"])
        return _prefix(s)
    if kind == "beam":
        if own:
            from sparse_mla_decode_token_gb300 import search
            return search.beam_select(s["logits"], s["scores"], s["workspace"], num_out=s["keep"], finished=s["finished"],
                                      end_token=s["end"])
        return _beam(s)
    if kind == "reorder":
        # the tables as they were before the pass
        s["tables"].copy_(s["tables0"])
        s["refs"].copy_(s["refs0"])
        if own:
            from sparse_mla_decode_token_gb300 import cache
            cache.pages_reorder(s["tables"], s["refs"], s["lens"], s["parents"], s["out_lens"], s["workspace"], page_size=PAGE)
            cache.pages_shared_prefix(s["tables"], s["out_lens"], s["starts"], s["out_prefix"], page_size=PAGE)
        else:
            _reorder(s)
        return s["tables"], s["refs"], s["out_lens"], s["out_prefix"]
    if own:
        from sparse_mla_decode_token_gb300 import slots
        step = slots.token_slots(s["lens"], s["new_lens"], s["tables"], max_tokens=s["tokens"], page_size=PAGE)
        table, topk = slots.sparse_slots(s["new_lens"], s["tables"], s["tokens"], page_size=PAGE, cum_seq_lens_q=step.cum_seq_lens_q,
                                         selected=s["picks"], compressed_tables=s["comp_tables"], compressed_page_size=PAGE,
                                         compress_ratio=s["ratio"])
        return (*step, table, topk)
    return _slots(s)


# ------------------------------------------------------------------- floor, exact

def _mean_spread(n, lo, hi):
    return sum(lo + i * 40503 % (hi - lo + 1) for i in range(1, n + 1)) / n


def work(case):
    kind = case["kind"]
    if kind == "prefix":
        n = case["groups"] * case["members"]
        prefix = _mean_spread(case["groups"], case["prefix_min"], case["prefix_max"])
        mine, q = _mean_spread(n, 1, case["own_max"]), _mean_spread(n, 1, case["q_max"])
        tokens, h = n * q, case["heads"]
        return {"bytes": (case["groups"] * prefix + n * mine) * (DIM + 4 / BLOCK) + tokens * h * (4 * DIM + 4),
                "flops": 4.0 * tokens * h * (prefix + mine) * DIM}
    if kind == "beam":
        n = case["batch"] * case["beams"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 0.9 * n * case["vocab"] * size + n * 5 + case["batch"] * case["keep"] * 12,
                "flops": 3.0 * 0.9 * n * case["vocab"]}
    if kind == "reorder":
        n = case["groups"] * case["beams"]
        # entries held (read in the old rows and for the shared prefix), those of the beams' own pages written and counted
        held, mine = n * case["max_pages"] * 0.625, n * case["max_pages"] * 0.125
        return {"bytes": 8 * held + 12 * mine + 12 * n, "flops": 0}
    tokens = case["batch"] * _mean_spread(case["batch"], 1 if case["q_max"] <= 4 else -(-case["q_max"] // 3), case["q_max"])
    per = 4 * (WINDOW + case["selected"]) + 4 * case["selected"] + 20
    return {"bytes": tokens * per + case["batch"] * 4 * (3 + (case["q_max"] + WINDOW) / PAGE), "flops": 0}


def exact(case, seed):
    """The definitions in 64 bits; whole numbers (tables, tokens, slots) have no such value."""
    if case["kind"] == "prefix":
        return _exact_prefix(prepare(case, seed))
    if case["kind"] == "beam":
        return _exact_beam(prepare(case, seed))
    return None


def _exact_prefix(s):
    cum, lens, prefix = s["cum"].tolist(), s["seq_lens"].tolist(), s["prefix"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")

    def values(row, lo, hi):
        j = torch.arange(lo, hi, device="cuda")
        page = s["tables"][row].long()[j // PAGE]
        return s["rows"][page, j % PAGE].to(torch.float64) * s["scales"].to(torch.float64)[page, j % PAGE // BLOCK][:, None]

    for g, p in enumerate(prefix):
        first = g * s["members"]
        head = values(first, 0, p)
        for b in range(first, first + s["members"]):
            kv = torch.cat([head, values(b, p, lens[b])])
            for t in range(cum[b], cum[b + 1]):
                n = lens[b] - (cum[b + 1] - 1 - t)                     # rows that the token sees
                x = s["q"][t].to(torch.float64) @ kv[:n].T * s["scale"]
                e = torch.logsumexp(x, dim=1)
                z = torch.logaddexp(e, s["sinks"].to(torch.float64))
                out[t] = torch.exp(x - z[:, None]) @ kv[:n]
                lse[t] = e / math.log(2.0)
    return out, lse


def _exact_beam(s):
    scores = []
    for b in range(s["batch"]):
        best = []
        for i in range(s["beams"]):
            start = s["scores"][b, i].double()
            if bool(s["finished"][b, i]):
                best.append(start[None])
            else:
                x = s["logits"][b * s["beams"] + i].double()
                best.append(torch.topk(x, min(s["keep"], x.numel())).values - torch.logsumexp(x, dim=0) + start)
        best = torch.sort(torch.cat(best), descending=True).values[: s["keep"]]
        scores.append(torch.nn.functional.pad(best, (0, s["keep"] - best.numel()), value=-math.inf))
    return torch.stack(scores), None, None
