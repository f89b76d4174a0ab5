"""Cases of the paged latent cache: what a serving program does around a decode.

Four operators over one paged cache of 512-wide latent rows, held in E4M3 with
one fp32 scale per block of tokens:

* ``window``: attention of BF16 queries (64 or 128 heads sharing the latent
  row) over the last ``window`` tokens of each request and its first few;
* ``append``: new BF16 latent rows quantised into the cache's pages;
* ``resize``: a serving step's page turnover: requests that end give their
  pages back, others take pages for the tokens they are about to write;
* ``fork``: parallel sampling: children share their parent's pages, every
  sequence grows by one token, shared partial pages are copied first;
* ``compact``: live pages moved to the front of the pool, the tables renumbered.

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through the package's public calls.
"""
import math

import torch

own = False

PAGE = 64          # tokens per page
BLOCK = 16         # tokens that share a scale
DIM = 512          # latent row
MAX_CODE = 448.0   # largest E4M3 value
MIN_EXP, MAX_EXP = -64, 64


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one user's chat: two sequences, the sliding-window layer's 128 tokens
        dict(name="window tiny", kind="window", batch=2, q_max=1, heads=64, window=128, first=4, ctx_min=129, ctx_max=2048),
        # a full decode batch over a medium window
        dict(name="window decode", kind="window", batch=128, q_max=1, heads=128, window=2048, first=4, ctx_min=4096,
             ctx_max=8192),
        # speculative decode: 1 to 4 tokens a request, ragged
        dict(name="window varlen", kind="window", batch=64, q_max=4, heads=64, window=1024, first=16, ctx_min=1000,
             ctx_max=6000),
        # chunked prefill: a few hundred new tokens behind ragged prefixes
        dict(name="window prefill", kind="window", batch=4, q_max=768, heads=128, window=512, first=4, ctx_min=800,
             ctx_max=5000),
        # one new token for each request of a decode batch
        dict(name="append decode", kind="append", batch=128, q_max=1, ctx_min=1000, ctx_max=4096),
        # prompts of a prefill batch
        dict(name="append prefill", kind="append", batch=8, q_max=6000, ctx_min=6000, ctx_max=9000),
        # a decode batch's turnover in a pool of 16 thousand pages
        dict(name="resize batch", kind="resize", rows=128, max_pages=128, pages=16384),
        # a large server's turnover: a million pages (16 layers' worth of a shared numbering)
        dict(name="resize server", kind="resize", rows=1024, max_pages=1024, pages=1048576),
        # four samples of each of a few prompts
        dict(name="fork samples", kind="fork", parents=4, children=3, max_pages=64, pages=1024, layers=1),
        # a wide search over many prompts, pages of four layers
        dict(name="fork search", kind="fork", parents=64, children=7, max_pages=64, pages=6144, layers=4),
        # a small pool after a burst of requests ended
        dict(name="compact small", kind="compact", rows=64, max_pages=32, pages=2048, layers=1),
        # half a gigabyte of pages a layer, two layers
        dict(name="compact large", kind="compact", rows=256, max_pages=64, pages=16384, layers=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["window", "window", "window", "append", "append", "resize", "fork", "compact"])
    if kind == "window":
        window, batch, heads = _log(rng, 32, 2048), _log(rng, 1, 128), rng.choice([64, 128])
        # tokens x heads x window stays at or under the largest listed case's
        most = max(1, (128 * 128 * 2048) // (batch * heads * window))
        q_max = _log(rng, 1, min(768, most, max(1, 2048 // batch)))
        ctx_min = _log(rng, max(1, q_max), 4096)
        return dict(kind=kind, batch=batch, q_max=q_max, heads=heads, window=window, first=rng.choice([0, 1, 4, 7, 16, 64]),
                    ctx_min=ctx_min, ctx_max=ctx_min + _log(rng, 1, 4096))
    if kind == "append":
        batch = _log(rng, 1, 256)
        q_max = _log(rng, 1, max(1, 48000 // batch))
        ctx_min = q_max + _log(rng, 1, 1000)
        return dict(kind=kind, batch=batch, q_max=q_max, ctx_min=ctx_min, ctx_max=ctx_min + _log(rng, 1, 2000))
    if kind == "resize":
        rows, max_pages = _log(rng, 1, 1024), _log(rng, 4, 1024)
        return dict(kind=kind, rows=rows, max_pages=max_pages, pages=rows * max_pages + rng.randint(0, 1000))
    if kind == "fork":
        parents, children, max_pages = _log(rng, 1, 64), rng.randint(1, 7), _log(rng, 4, 64)
        return dict(kind=kind, parents=parents, children=children, max_pages=max_pages,
                    pages=parents * max_pages + 2 * parents * (children + 1) + rng.randint(0, 500), layers=rng.randint(1, 4))
    rows, max_pages = _log(rng, 4, 256), _log(rng, 4, 64)
    return dict(kind=kind, rows=rows, max_pages=max_pages, pages=rows * max_pages + rng.randint(0, 300),
                layers=rng.randint(1, 2))


# ------------------------------------------------------------------ the inputs

def _lengths(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int64)


def _q_lens(case, g):
    """New tokens of each request: from 1 (a third of q_max for prompts) to q_max, in an order of the seed's; as many in all for every seed."""
    lo, q, n = 1 if case["q_max"] <= 4 else -(-case["q_max"] // 3), case["q_max"], case["batch"]
    return lo + (torch.arange(1, n + 1) * 40503 % (q - lo + 1))[torch.randperm(n, generator=g)]


def _tables(g, lens, max_pages, num_pages):
    """Random distinct pages for each request's tokens; -1 behind them."""
    n = (lens + PAGE - 1) // PAGE
    used = torch.arange(max_pages)[None, :] < n[:, None]
    tables = torch.full((lens.numel(), max_pages), -1, dtype=torch.int64)
    tables[used] = torch.randperm(num_pages, generator=g)[: int(n.sum())]
    return tables


def _latents(gd, n):
    """Latent rows: unit normal, each token with a magnitude of its own."""
    x = torch.randn((n, DIM), generator=gd, device="cuda")
    return x * torch.exp2(torch.randn((n, 1), generator=gd, device="cuda") * 0.5)


def _filled_cache(gd, pages):
    """Pages as they stand in a running server: block scales are powers of two that fit the block's largest value."""
    rows = torch.empty((pages, PAGE, DIM), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((pages, PAGE // BLOCK), dtype=torch.float32, device="cuda")
    for p in range(0, pages, 2048):
        n = min(2048, pages - p)
        x = _latents(gd, n * PAGE).view(n, PAGE // BLOCK, BLOCK, DIM)
        s = _block_scale(x.abs().amax(dim=(2, 3)))
        rows[p:p + n] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(n, PAGE, DIM)
        scales[p:p + n] = s
    return rows, scales


def _i32(t):
    return t.to(torch.int32).cuda()


def _moves(capacity):
    return (torch.full((capacity,), -1, dtype=torch.int32, device="cuda"),
            torch.full((capacity,), -1, dtype=torch.int32, device="cuda"),
            torch.zeros(1, dtype=torch.int32, device="cuda"))


def _pools(gd, case):
    return [torch.randint(0, 256, (case["pages"], PAGE, DIM), generator=gd, device="cuda", dtype=torch.uint8)
            for _ in range(case["layers"])] + \
           [torch.rand((case["pages"], PAGE // BLOCK), generator=gd, device="cuda") + 0.5 for _ in range(case["layers"])]


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    s = dict(case)
    if kind in ("window", "append"):
        q_lens = _q_lens(case, g)
        ctx = torch.maximum(_lengths(g, case["batch"], case["ctx_min"], case["ctx_max"]), q_lens)
        max_pages = -(-max(case["ctx_max"], case["q_max"]) // PAGE)
        pages = case["batch"] * max_pages + 16
        s["tables"] = _i32(_tables(g, ctx, max_pages, pages))
        s["seq_lens"] = _i32(ctx)
        s["cum"] = _i32(torch.cat([torch.zeros(1, dtype=torch.int64), q_lens.cumsum(0)]))
        s["tokens"] = int(q_lens.sum())
        s["rows"], s["scales"] = _filled_cache(gd, pages)
        if kind == "window":
            s["q"] = torch.randn((s["tokens"], case["heads"], DIM), generator=gd, device="cuda").to(torch.bfloat16)
            s["sinks"] = torch.randn((case["heads"],), generator=gd, device="cuda")
            s["scale"] = 1.0 / math.sqrt(DIM)
            s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        else:
            s["latent"] = _latents(gd, s["tokens"]).to(torch.bfloat16)
    elif kind == "resize":
        rows, cap = case["rows"], case["max_pages"] * PAGE
        s["lens"] = []
        # a request in four has ended (or not yet begun) in each of the two phases; the others grow or are cut by some tokens
        base = _lengths(g, rows, 1, max(1, cap - 8))
        gone = torch.rand((2, rows), generator=g)
        for k in range(2):
            lens = (base + torch.randint(0, 9, (rows,), generator=g)).clamp(max=cap)
            s["lens"].append(torch.where(gone[k] < 0.25, torch.zeros_like(lens), lens))
        s["tables"] = _i32(_tables(g, s["lens"][0], case["max_pages"], case["pages"]))
        s["lens"] = [_i32(x) for x in s["lens"]]
        s["phase"] = 0
        s["refs"] = _ref_counts(s["tables"], case["pages"])
        s["moves"] = _moves(rows)
    elif kind == "fork":
        rows = case["parents"] * (1 + case["children"])
        lens = torch.zeros(rows, dtype=torch.int64)
        lens[: case["parents"]] = _lengths(g, case["parents"], PAGE, case["max_pages"] * PAGE - 2)
        s["tables"] = _i32(_tables(g, lens, case["max_pages"], case["pages"]))
        s["refs"] = _ref_counts(s["tables"], case["pages"])
        parent = torch.full((rows,), -1, dtype=torch.int64)
        parent[case["parents"]:] = torch.arange(rows - case["parents"]) % case["parents"]
        s["parent"] = _i32(parent)
        s["start"], s["forked"] = _i32(lens), _i32(torch.zeros(rows))
        s["lens"] = s["start"].clone()
        s["moves"] = _moves(rows)
        s["pools"] = _pools(gd, case)
    else:
        rows = case["rows"]
        lens = _lengths(g, rows, 1, case["max_pages"] * PAGE)
        tables = _tables(g, lens, case["max_pages"], case["pages"])
        ended = torch.rand(rows, generator=g) < 0.4        # requests that ended since: their pages are holes
        ended[0] = False
        lens[ended] = 0
        tables[ended] = -1
        s["tables0"], s["lens"] = _i32(tables), _i32(lens)
        s["refs0"] = _ref_counts(s["tables0"], case["pages"])
        s["tables"], s["refs"] = s["tables0"].clone(), s["refs0"].clone()
        s["moves"] = _moves(case["pages"] // 2)
        s["pools"] = _pools(gd, case)
    if kind in ("resize", "fork", "compact"):
        s["workspace"] = torch.empty(16 * case["pages"] + 65536, dtype=torch.uint8, device="cuda")
    return s


def _ref_counts(tables, pages):
    flat = tables[tables >= 0].long()
    return torch.bincount(flat, minlength=pages).to(torch.int32)


# -------------------------------------------------------------- the plain forms

def _block_scale(amax):
    """Smallest power of two s with amax <= 448 s, its exponent held to [-64, 64]."""
    f, e = torch.frexp(amax)                       # amax = f 2^e, f in [0.5, 1); 448 = 0.875 2^9
    k = torch.where(f <= 0.875, e - 9, e - 8)
    k = torch.where(amax > 0, k, torch.full_like(k, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)
    return torch.ldexp(torch.ones_like(amax), k)


def _positions(s):
    """Request and right-aligned position of each flattened new token."""
    t = torch.arange(s["tokens"], device="cuda")
    cum = s["cum"].long()
    b = torch.searchsorted(cum, t, right=True) - 1
    pos = s["seq_lens"].long()[b] - (cum[b + 1] - cum[b]) + (t - cum[b])
    return b, pos


def _window(s):
    b, pos = _positions(s)
    first, window = s["first"], s["window"]
    lead = torch.arange(first, device="cuda").expand(pos.numel(), first)
    last = pos[:, None] - window + 1 + torch.arange(window, device="cuda")[None, :]
    at = torch.cat([lead, last], dim=1)                                            # [T, first + window] positions
    ok = torch.cat([lead <= pos[:, None], last >= first], dim=1)
    at = at.clamp(min=0).minimum(pos[:, None].clamp(min=0))
    page = s["tables"][b[:, None], at // PAGE].long()
    kv = s["rows"][page, at % PAGE].float() * s["scales"][page, at % PAGE // BLOCK][..., None]
    logits = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * s["scale"]         # [T, H, first + window]
    logits = logits.masked_fill(~ok[:, None, :], -math.inf)
    m = logits.amax(dim=2, keepdim=True)
    p = torch.exp(logits - m)
    total = p.sum(dim=2, keepdim=True)
    out = torch.matmul(p, kv) / (total + torch.exp(s["sinks"][None, :, None] - m))
    lse = (m + torch.log(total)).squeeze(2) / math.log(2.0)
    return out.to(torch.bfloat16), lse


def _append(s):
    b, pos = _positions(s)
    cum = s["cum"].long()
    start = (s["seq_lens"].long() - (cum[1:] - cum[:-1]))[b]                       # first new position of the request
    page = s["tables"][b, pos // PAGE].long()
    block = page * (PAGE // BLOCK) + pos % PAGE // BLOCK                           # block of each new token
    scales, x = s["scales"].view(-1), s["latent"].float()
    amax = torch.zeros_like(scales).scatter_reduce_(0, block, x.abs().amax(dim=1), "amax")
    had = start > pos // BLOCK * BLOCK                                             # the block holds older tokens
    touched = torch.zeros_like(scales, dtype=torch.bool)
    touched[block] = True
    old = torch.zeros_like(scales)
    old[block[had]] = scales[block[had]]
    new = torch.where(touched, torch.maximum(old, _block_scale(amax)), scales)
    # older rows of the blocks whose scale grew
    lead = had & ((pos == start) | (pos % BLOCK == 0))
    n_old = (start - pos // BLOCK * BLOCK)[lead]
    blk = block[lead]
    mine = torch.arange(BLOCK, device="cuda")[None, :] < n_old[:, None]
    rows = s["rows"].view(-1, BLOCK, DIM)
    codes = rows[blk].float()
    moved = (codes * (old[blk] / new[blk])[:, None, None]).to(torch.float8_e4m3fn)
    keep = ~mine | (old[blk] == new[blk])[:, None]
    rows.view(torch.uint8)[blk] = torch.where(keep[..., None], rows[blk].view(torch.uint8), moved.view(torch.uint8))
    s["rows"].view(torch.uint8)[page, pos % PAGE] = \
        (x / new[block][:, None]).clamp(-MAX_CODE, MAX_CODE).to(torch.float8_e4m3fn).view(torch.uint8)
    scales.copy_(new)


def _resize(tables, refs, old, new, moves):
    rows, width = tables.shape
    old, new = old.long(), new.long()
    c = torch.arange(width, device="cuda")[None, :]
    c_old, c_new = ((old + PAGE - 1) // PAGE)[:, None], ((new + PAGE - 1) // PAGE)[:, None]
    freed = (c >= c_new) & (c < c_old)
    gone = tables[freed].long()
    refs.index_add_(0, gone, -torch.ones_like(gone, dtype=torch.int32))
    tables[freed] = -1
    # a shared page that is about to be written is replaced by a copy
    at = (old // PAGE).clamp(max=width - 1)
    page = tables.gather(1, at[:, None]).squeeze(1).long()
    cow = (new > old) & (old % PAGE > 0) & (refs[page.clamp(min=0)] > 1)
    grown = (c >= c_old) & (c < c_new)
    need = torch.cat([cow[:, None], grown], dim=1)
    free = torch.nonzero(refs == 0).squeeze(1)[: int(need.sum())]
    refs[free] = 1
    got = torch.full((rows, width + 1), -1, dtype=torch.int32, device="cuda")
    got[need] = free.to(torch.int32)                                               # in order of row, then column
    tables.copy_(torch.where(grown, got[:, 1:], tables))
    src, dst = page[cow], got[:, 0][cow]
    refs.index_add_(0, src, -torch.ones_like(src, dtype=torch.int32))
    tables[cow, at[cow]] = dst
    moves[0][: src.numel()] = src.to(torch.int32)
    moves[1][: src.numel()] = dst
    moves[2].fill_(src.numel())


def _fork(tables, refs, lens, parent, new_lens):
    p = parent.long().clamp(min=0)
    child = parent >= 0
    new_lens.copy_(torch.where(child, lens[p], lens))
    n = (lens[p].long() + PAGE - 1) // PAGE
    use = child[:, None] & (torch.arange(tables.shape[1], device="cuda")[None, :] < n[:, None])
    tables.copy_(torch.where(use, tables[p], tables))
    shared = tables[use].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))


def _compact(tables, refs, lens, moves):
    ids = torch.arange(refs.numel(), device="cuda")
    live = refs > 0
    n = live.sum()
    src, dst = torch.nonzero(live & (ids >= n)).squeeze(1), torch.nonzero(~live & (ids < n)).squeeze(1)
    name = ids.clone()
    name[src] = dst
    used = torch.arange(tables.shape[1], device="cuda")[None, :] < ((lens.long() + PAGE - 1) // PAGE)[:, None]
    tables.copy_(torch.where(used, name[tables.long().clamp(min=0)].to(torch.int32), tables))
    refs[dst] = refs[src]
    refs[src] = 0
    moves[0][: src.numel()] = src.to(torch.int32)
    moves[1][: src.numel()] = dst.to(torch.int32)
    moves[2].fill_(src.numel())


def _copy(pools, moves):
    n = int(moves[2])
    src, dst = moves[0][:n].long(), moves[1][:n].long()
    return [pool.index_copy_(0, dst, pool[src]) for pool in pools]


# ------------------------------------------------------------------------ a pass

def run(s):
    kind = s["kind"]
    if own:
        from sparse_mla_decode_token_gb300 import cache
    if kind == "window":
        if own:
            return cache.window_attention(s["q"], s["rows"], s["scales"], s["tables"], s["seq_lens"], s["workspace"],
                                          window=s["window"], first_tokens=s["first"], cum_seq_lens_q=s["cum"],
                                          sinks=s["sinks"], bmm1_scale=s["scale"])
        return _window(s)
    if kind == "append":
        if own:
            cache.append(s["latent"], s["rows"], s["scales"], s["tables"], s["seq_lens"], cum_seq_lens_q=s["cum"])
        else:
            _append(s)
        return s["rows"], s["scales"]
    if kind == "resize":
        old, new = s["lens"][s["phase"]], s["lens"][1 - s["phase"]]
        s["phase"] = 1 - s["phase"]
        if own:
            cache.pages_resize(s["tables"], s["refs"], old, new, s["workspace"], page_size=PAGE, moves=s["moves"])
        else:
            _resize(s["tables"], s["refs"], old, new, s["moves"])
        return s["tables"], s["refs"], s["moves"][2]
    if kind == "fork":
        # the last step's children end (the first time there are none), then every parent is forked and all grow by a token
        if own:
            cache.pages_resize(s["tables"], s["refs"], s["lens"], s["start"], s["workspace"], page_size=PAGE,
                               moves=s["moves"])
            cache.pages_fork(s["tables"], s["refs"], s["start"], s["parent"], s["forked"], page_size=PAGE)
            torch.add(s["forked"], 1, out=s["lens"])
            cache.pages_resize(s["tables"], s["refs"], s["forked"], s["lens"], s["workspace"], page_size=PAGE,
                               moves=s["moves"])
            cache.pages_copy(s["pools"], s["moves"])
        else:
            _resize(s["tables"], s["refs"], s["lens"], s["start"], s["moves"])
            _fork(s["tables"], s["refs"], s["start"], s["parent"], s["forked"])
            torch.add(s["forked"], 1, out=s["lens"])
            _resize(s["tables"], s["refs"], s["forked"], s["lens"], s["moves"])
            _copy(s["pools"], s["moves"])
        return s["tables"], s["refs"], s["lens"], s["moves"][2], s["pools"]
    # the pool as it was before the pass; moving the same pages again leaves the same bytes
    s["tables"].copy_(s["tables0"])
    s["refs"].copy_(s["refs0"])
    if own:
        cache.pages_compact(s["tables"], s["refs"], s["lens"], s["workspace"], page_size=PAGE, moves=s["moves"])
        cache.pages_copy(s["pools"], s["moves"])
    else:
        _compact(s["tables"], s["refs"], s["lens"], s["moves"])
        _copy(s["pools"], s["moves"])
    return s["tables"], s["refs"], s["moves"][2], s["pools"]


# ------------------------------------------------------------------- floor, exact

def _means(case):
    q = (1 + case["q_max"]) / 2 if case["q_max"] <= 4 else (-(-case["q_max"] // 3) + case["q_max"]) / 2
    return case["batch"] * q, q, (case["ctx_min"] + case["ctx_max"]) / 2


def work(case):
    kind = case["kind"]
    if kind == "window":
        tokens, q, ctx = _means(case)
        per = min(case["window"] + case["first"], ctx)                  # rows a token sees
        rows = case["batch"] * min(per + q - 1, ctx)                    # distinct rows of a request's tokens
        return {"bytes": rows * (DIM + 4 / BLOCK) + tokens * case["heads"] * (4 * DIM + 4),
                "flops": 4.0 * tokens * case["heads"] * per * DIM}
    if kind == "append":
        tokens, _, _ = _means(case)
        return {"bytes": tokens * 3 * DIM + (tokens / BLOCK + case["batch"]) * 8, "flops": 2.0 * tokens * DIM}
    if kind == "resize":
        # each count once, the changed table entries, the lengths
        changed = case["rows"] * case["max_pages"] * 0.5 * 0.375
        return {"bytes": 4.0 * case["pages"] + 12 * changed + 8 * case["rows"], "flops": 0}
    page = PAGE * DIM + PAGE // BLOCK * 4
    if kind == "fork":
        rows = case["parents"] * (1 + case["children"])
        shared = case["parents"] * case["children"] * case["max_pages"] / 2
        return {"bytes": 4.0 * case["pages"] + 12 * shared + 2.0 * rows * page * case["layers"], "flops": 0}
    live = case["rows"] * case["max_pages"] / 2 * 0.6
    moved = live * (1 - live / case["pages"])
    return {"bytes": 8.0 * case["pages"] + 8 * live + 2 * moved * page * case["layers"], "flops": 0}


def exact(case, seed):
    """The definitions in 64 bits; whole numbers (tables, counts, copied bytes) have no such value."""
    if case["kind"] == "window":
        return _exact_window(prepare(case, seed))
    if case["kind"] == "append":
        return _exact_append(prepare(case, seed))
    return None


def _exact_window(s):
    cum, lens = s["cum"].tolist(), s["seq_lens"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        lo = max(0, n - (cum[b + 1] - cum[b]) - s["window"] + 1)        # the earliest row a window of this request reaches
        at = [j for j in range(n) if j >= lo or j < s["first"]]
        j = torch.tensor(at, device="cuda")
        page = s["tables"][b].long()[j // PAGE]
        kv = s["rows"][page, j % PAGE].to(torch.float64) * s["scales"].to(torch.float64)[page, j % PAGE // BLOCK][:, None]
        for t0 in range(cum[b], cum[b + 1], 64):
            t1 = min(t0 + 64, cum[b + 1])
            pos = n - cum[b + 1] + torch.arange(t0, t1, device="cuda")
            seen = (j[None, :] <= pos[:, None]) & ((j[None, :] > pos[:, None] - s["window"]) | (j[None, :] < s["first"]))
            x = torch.einsum("thd,jd->thj", s["q"][t0:t1].to(torch.float64), kv) * s["scale"]
            x = torch.where(seen[:, None, :], x, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
            e = torch.logsumexp(x, dim=2)
            z = torch.logaddexp(e, s["sinks"].to(torch.float64)[None, :])
            out[t0:t1] = torch.einsum("thj,jd->thd", torch.exp(x - z[:, :, None]), kv)
            lse[t0:t1] = e / math.log(2.0)
    return out, lse


def _exact_append(s):
    """Codes as the unrounded quotients of the rows and their block's scale."""
    cum, lens, tables = s["cum"].tolist(), s["seq_lens"].tolist(), s["tables"].cpu()
    codes, scales = s["rows"].to(torch.float64), s["scales"].to(torch.float64)
    x = s["latent"].to(torch.float64)
    top = x.abs().amax(dim=1).cpu()
    for b, n in enumerate(lens):
        start = n - (cum[b + 1] - cum[b])
        p = start
        while p < n:
            end = min(n, p // BLOCK * BLOCK + BLOCK)
            page, at, blk = int(tables[b, p // PAGE]), p % PAGE, p % PAGE // BLOCK
            t = cum[b] + p - start
            big = float(top[t:t + end - p].max())
            k = MIN_EXP
            while k < MAX_EXP and big > MAX_CODE * 2.0 ** k:
                k += 1
            new = 2.0 ** k
            if p % BLOCK:
                old = float(scales[page, blk])
                new = max(old, new)
                codes[page, blk * BLOCK:at] *= old / new
            scales[page, blk] = new
            codes[page, at:at + end - p] = x[t:t + end - p] / new
            p = end
    return codes, scales
