"""Plain 64-bit references of the paged latent cache, one step at a time on the
host, and the error bounds that the GPU results are held to."""
from __future__ import annotations

import math

import numpy as np
import torch

DIM = 512


def e4m3(codes):
    """Values of E4M3 codes (uint8 array) in float64."""
    t = torch.from_numpy(np.ascontiguousarray(codes, dtype=np.uint8)).view(torch.float8_e4m3fn)
    return t.to(torch.float64).numpy()


def to_e4m3(x):
    """Codes of float values, rounded to nearest even, saturated; NaN is 0x7f."""
    x = np.asarray(x, dtype=np.float32)
    t = torch.from_numpy(np.clip(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0), -448.0, 448.0))
    c = t.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    c[np.isnan(x)] = 0x7F
    return c


class Cache:
    """rows [pages, page_size, 512] uint8, scales [pages, page_size // block] float32, tables, lens (numpy)."""

    def __init__(self, rows, scales, tables, lens, cum=None, tokens=None):
        self.rows, self.scales, self.tables, self.lens = rows, scales, tables, lens
        self.page_size, self.block = rows.shape[1], rows.shape[1] // scales.shape[1]
        batch = len(lens)
        self.cum = cum if cum is not None else np.arange(batch + 1) * (tokens // batch)

    def page(self, b, j):
        c = j // self.page_size
        page = int(self.tables[b, c]) if c < self.tables.shape[1] else -1
        return page if 0 <= page < self.rows.shape[0] else -1

    def row(self, b, j):
        page, r = self.page(b, j), j % self.page_size
        return e4m3(self.rows[page, r]) * np.float64(abs(self.scales[page, r // self.block]))


def window(cache, q, *, window, first=0, sinks=None, bmm1=1.0, bmm2=1.0):
    """O [T, H, 512], LSE2 [T, H] and how far a kernel may be from each.

    The kernel computes, per row j and head, t_j from products of exact E4M3
    numbers in fp32 (a relative 2^-18 of sum |q||k| covers its 32 accumulation
    steps; q's split is exact but for 2^-17 of the head's largest |q|), weights
    p_j rounded twice to E4M3 (2^-4 * 2^-4, through fp16: 2^-11) with an absolute
    floor of half E4M3's subnormal step, 2^-10 against a largest weight of at
    least 2^4, a sum of products in fp32 (2^-18), and one rounding to BF16 (2^-8).
    """
    T, H = q.shape[:2]
    out, lse = np.zeros((T, H, DIM)), np.full((T, H), -np.inf)
    tol_o, tol_l = np.zeros((T, H, DIM)), np.zeros((T, H))
    for b in range(len(cache.lens)):
        for t in range(int(cache.cum[b]), int(cache.cum[b + 1])):
            pos = int(cache.lens[b]) - int(cache.cum[b + 1] - cache.cum[b]) + (t - int(cache.cum[b]))
            last = min(pos, cache.tables.shape[1] * cache.page_size - 1)
            at = [j for j in range(last + 1) if (j > pos - window or j < first) and cache.page(b, j) >= 0]
            if not at:
                continue
            kv = np.stack([cache.row(b, j) for j in at])
            with np.errstate(invalid="ignore"):
                l = (q[t] @ kv.T) * bmm1
                reach = np.abs(q[t]) @ np.abs(kv).T * abs(bmm1)
                off = 2.0 ** -18 * reach + \
                    2.0 ** -17 * np.abs(q[t]).max(axis=1, keepdims=True) * np.abs(kv).sum(axis=1)[None, :] * abs(bmm1)
                m = l.max(axis=1, keepdims=True)
                p = np.exp(l - m)
                total = p.sum(axis=1)
                z = total if sinks is None else total + np.exp(sinks - m[:, 0])
                out[t] = bmm2 * (p @ kv) / z[:, None]
                lse[t] = (m[:, 0] + np.log(total)) / math.log(2.0)
                rel = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18 + 2 * off
                # the floor counts in weights p_j s_j / s_max of the raw codes: relative to the largest |row scale|
                code = np.stack([e4m3(cache.rows[cache.page(b, j), j % cache.page_size]) for j in at])
                s = np.array([max(abs(cache.scales[cache.page(b, j), j % cache.page_size // cache.block]), 2.0 ** -64)
                              for j in at], dtype=np.float64)
                w = p * s[None, :]
                floor = 2.0 ** -14 * w.max(axis=1)[:, None] * np.abs(code).sum(axis=0)[None, :] / z[:, None]
                mean = ((p * rel) @ np.abs(kv)) / z[:, None]
                # (the normaliser's own error scales the result)
                norm = (p * 2 * off).sum(axis=1) / z + 2.0 ** -18
                tol_o[t] = abs(bmm2) * (mean + floor) + np.abs(out[t]) * (2.0 ** -8 + norm[:, None]) + 2.0 ** -120
                tol_l[t] = 1.4427 * ((p * 2 * off).sum(axis=1) / total + 2.0 ** -18) + 2.0 ** -21 * np.abs(lse[t])
    return out, lse, tol_o, tol_l


def append(cache, latent, flags=None):
    """Quantises latent [T, 512] (float32 values of BF16) into the cache in place."""
    for b in range(len(cache.lens)):
        t0, t1 = int(cache.cum[b]), int(cache.cum[b + 1])
        start = int(cache.lens[b]) - (t1 - t0)
        blocks = sorted({j // cache.block for j in range(max(start, 0), int(cache.lens[b]))}) if t1 > t0 else []
        for blk in blocks:
            j0 = blk * cache.block
            page = cache.page(b, j0)
            if page < 0:
                continue
            new = [j for j in range(j0, j0 + cache.block) if max(start, 0) <= j < int(cache.lens[b])]
            x = latent[[t0 + j - start for j in new]].astype(np.float32)
            finite = np.abs(x[np.isfinite(x)])
            amax = float(finite.max()) if finite.size else 0.0
            k = -64
            while k < 64 and amax > 448.0 * 2.0 ** k:
                k += 1
            s_at = (page, j0 % cache.page_size // cache.block)
            old = np.float32(0)
            if new[0] > j0:
                old = cache.scales[s_at]
                old = old if np.isfinite(old) and old > 0 else np.float32(0)
            stored = cache.scales[s_at] if new[0] > j0 else np.float32(0)
            s = np.float32(max(float(old), 2.0 ** k))
            cache.scales[s_at] = s
            if new[0] > j0 and stored != s:
                ratio = np.float32(old / s)
                for j in range(j0, new[0]):
                    r = j % cache.page_size
                    codes = cache.rows[page, r]
                    cache.rows[page, r] = to_e4m3(e4m3(codes).astype(np.float32) * ratio)
            with np.errstate(invalid="ignore"):
                for j, v in zip(new, x):
                    cache.rows[page, j % cache.page_size] = to_e4m3(v / s)


class Pages:
    """Page tables and counts, kept one entry at a time."""

    def __init__(self, rows, max_pages, page_size, num_pages):
        self.tables = np.full((rows, max_pages), -1, dtype=np.int32)
        self.refs = np.zeros(num_pages, dtype=np.int32)
        self.page_size = page_size

    def columns(self, n):
        cap = self.tables.shape[1] * self.page_size
        return -(-min(max(int(n), 0), cap) // self.page_size)

    def resize(self, lens, new):
        cap = self.tables.shape[1] * self.page_size
        lens, new = np.clip(lens, 0, cap), np.clip(new, 0, cap)
        for b in range(len(lens)):
            for c in range(self.columns(new[b]), self.columns(lens[b])):
                self.refs[self.tables[b, c]] -= 1
                self.tables[b, c] = -1
        shared = self.refs.copy()
        free = [int(p) for p in np.flatnonzero(self.refs == 0)]
        moves, short = [], False
        for b in range(len(lens)):
            if new[b] <= lens[b]:
                continue
            at = int(lens[b]) // self.page_size
            if lens[b] % self.page_size and shared[self.tables[b, at]] > 1:
                if free:
                    page, old = free.pop(0), int(self.tables[b, at])
                    self.refs[page], self.refs[old] = 1, self.refs[old] - 1
                    self.tables[b, at] = page
                    moves.append((old, page))
                else:
                    short = True
            for c in range(self.columns(lens[b]), self.columns(new[b])):
                if free:
                    self.tables[b, c] = free.pop(0)
                    self.refs[self.tables[b, c]] = 1
                else:
                    self.tables[b, c], short = -1, True
        return moves, short

    def fork(self, lens, parents):
        out = lens.copy()
        for b, p in enumerate(parents):
            if p >= 0:
                for c in range(self.columns(lens[p])):
                    self.tables[b, c] = self.tables[p, c]
                    self.refs[self.tables[b, c]] += 1
                out[b] = lens[p]
        return out

    def compact(self, lens):
        n = int((self.refs > 0).sum())
        src = [p for p in range(len(self.refs)) if p >= n and self.refs[p] > 0]
        dst = [p for p in range(n) if self.refs[p] == 0]
        moves = list(zip(src, dst))
        name = dict(moves)
        for b in range(len(lens)):
            for c in range(self.columns(lens[b])):
                self.tables[b, c] = name.get(int(self.tables[b, c]), int(self.tables[b, c]))
        for a, z in moves:
            self.refs[z], self.refs[a] = self.refs[a], 0
        return moves
