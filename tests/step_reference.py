"""Plain references of a step's calls beside the attention: beam selection in 64
bits, reordering of page tables, shared prefixes and slot maps one entry at a
time on the host."""
from __future__ import annotations

import numpy as np


def beam_scores(logits, scores, finished=None, end_token=0):
    """[B, beams, V] scores of every continuation in float64 (-inf where there is none)."""
    batch, beams = scores.shape
    x = np.asarray(logits, dtype=np.float64).reshape(batch, beams, -1)
    s = np.asarray(scores, dtype=np.float64)
    total = np.full(x.shape, -np.inf)
    for b in range(batch):
        for i in range(beams):
            if not np.isfinite(s[b, i]):
                continue
            if finished is not None and finished[b, i]:
                total[b, i, end_token] = s[b, i]
                continue
            row = x[b, i]
            m = row.max()
            if np.isnan(row).any() or m == np.inf or m == -np.inf:
                continue
            total[b, i] = (row - m) + (s[b, i] - np.log(np.exp(row - m).sum()))
    return total


def beam_best(total, keep):
    """The `keep` best of each request, ties to the lowest (beam, token): scores, rows, tokens."""
    batch, beams, vocab = total.shape
    best = np.full((batch, keep), -np.inf)
    rows, tokens = np.full((batch, keep), -1), np.full((batch, keep), -1)
    for b in range(batch):
        flat = total[b].reshape(-1)
        at = np.argsort(-flat, kind="stable")[:keep]
        at = at[flat[at] > -np.inf]
        best[b, :at.size] = flat[at]
        rows[b, :at.size], tokens[b, :at.size] = b * beams + at // vocab, at % vocab
    return best, rows, tokens


def columns(n, width, page_size):
    return -(-min(max(int(n), 0), width * page_size) // page_size)


def reorder(tables, refs, lens, parents, page_size):
    """Tables, counts and lengths after it; flagged if something could not be."""
    width, old = tables.shape[1], tables.copy()
    out, refs, lengths, flag = tables.copy(), refs.copy(), lens.copy(), False
    for b, p in enumerate(parents):
        if p >= len(parents):
            flag, p = True, b
        n_old = columns(lens[b], width, page_size)
        n_new = columns(lens[p], width, page_size) if p >= 0 else 0
        lengths[b] = lens[p] if p >= 0 else 0
        if p == b:
            continue
        for c in range(n_old):
            refs[old[b, c]] -= 1
            out[b, c] = -1
        for c in range(n_new):
            refs[old[p, c]] += 1
            out[b, c] = old[p, c]
    return out, refs, lengths, flag


def shared_prefix(tables, lens, starts, page_size):
    out = []
    for lo, hi in zip(starts[:-1], starts[1:]):
        rows = [b for b in range(max(lo, 0), min(hi, len(lens))) if lens[b] > 0]
        n = 0
        if rows:
            full = min(min(int(lens[b]), tables.shape[1] * page_size) // page_size for b in rows)
            while n < full and tables[rows[0], n] >= 0 and all(tables[b, n] == tables[rows[0], n] for b in rows):
                n += 1
        out.append(n * page_size)
    return np.array(out)


def slot(tables, b, j, page_size, most=2 ** 62):
    c = j // page_size
    page = int(tables[b, c]) if c < tables.shape[1] else -1
    at = page * page_size + j % page_size
    return at if page >= 0 and at <= most else -1


def token_slots(lens, new_lens, max_tokens, tables=None, page_size=1):
    request, position, slots = (np.full(max_tokens, -1, dtype=np.int64) for _ in range(3))
    cum, t = [0], 0
    for b in range(len(lens)):
        old = max(0, int(lens[b]))
        n = max(0, int(new_lens[b]) - old)
        for i in range(n):
            if t + i < max_tokens:
                request[t + i], position[t + i] = b, old + i
                if tables is not None:
                    slots[t + i] = slot(tables, b, old + i, page_size)
        t += n
        cum.append(min(t, 2 ** 31 - 1))
    return np.array(cum), request, position, slots


def sparse_slots(seq_lens, cum, tokens, swa, page_size, comp=None, comp_page=1, ratio=1, selected=None, keep=0):
    keep = selected.shape[1] if selected is not None else keep
    out, topk = np.full((tokens, 128 + keep), -1), np.zeros(tokens, dtype=np.int64)
    for t in range(tokens):
        b = next((b for b in range(len(seq_lens)) if cum[b] <= t < cum[b + 1]), None)
        if b is None:
            continue
        pos = int(seq_lens[b]) - int(cum[b + 1] - cum[b]) + t - int(cum[b])
        if pos < 0:
            continue
        for j, at in enumerate(range(max(0, pos - 127), pos + 1)):
            out[t, j] = slot(swa, b, at, page_size, 2 ** 31 - 1)
        topk[t] = 128
        for k in range(keep):
            c = int(selected[t, k]) if selected is not None else k
            if 0 <= c < (pos + 1) // ratio:
                out[t, 128 + k] = slot(comp, b, c, comp_page, 2 ** 31 - 1)
                if out[t, 128 + k] >= 0:
                    topk[t] = 129 + k
    return out, topk
