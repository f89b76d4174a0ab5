"""Window attention where a few rows carry most of the weight and little of the
value: a visible first token of small values (an attention sink), one row far
above thousands of equal ones, long tails.  What the heavy row does not cover is
all that the output holds in most dims, so no weight may be rounded by more than
the output itself."""
import math

import numpy as np
import pytest
import torch

import cache_reference as R
from sparse_mla_decode_token_gb300 import cache as C
from test_cache_gpu import DEV, bf16, built, i32  # noqa: F401  (built: the library, once a module)

pytestmark = pytest.mark.gpu
OWN = 128            # dims that only the heavy row has
BMM1 = 1 / math.sqrt(512)
SHARES = (0.5, 0.9, 0.95, 0.99, 0.999, 0.9999, 0.99999, 0.02)


def visible(n, window, first):
    j = np.arange(n)
    return np.flatnonzero((j > n - 1 - window) | (j < first))


def exact(q, kv):
    """O [H, 512], natural-log LSE [H] of one token in 64 bits."""
    l = torch.from_numpy(q) @ torch.from_numpy(kv).T * BMM1
    p = torch.exp(l - l.max(dim=1, keepdim=True).values)
    return (p @ torch.from_numpy(kv) / p.sum(dim=1, keepdim=True)).numpy(), torch.logsumexp(l, dim=1).numpy()


def make(seed, n, *, window, first, amplitude, spread, mean, heavy_at=0, block=16, page=64, heads=64, size=60.0):
    """One request of n rows.  Row heavy_at has codes of `amplitude` in the first OWN dims and nothing else, every
    other row nothing there; head h gives it SHARES[h % 8] of the weight of what the last token sees.  The others'
    logits spread by `spread`, their values, codes of about `size`, share a mean of `mean` times their deviation.
    (The heavy row's small codes take query elements of some 1500 / amplitude times the others'; those are held to
    2^-22 of the largest, so the amplitude stays above size / 1000.)"""
    rng = np.random.default_rng(seed)
    pages = -(-n // page)
    codes = (rng.normal(size=(pages * page, 512)) + mean * rng.normal(size=512)) * size
    codes[:, :OWN] = 0
    sign = rng.choice([-1.0, 1.0], size=OWN)
    codes[heavy_at], codes[heavy_at, :OWN] = 0, amplitude * sign
    rows = R.to_e4m3(codes)
    order = rng.permutation(pages)
    scale = 2.0 ** -6
    kv = R.e4m3(rows)[:n] * scale
    at = visible(n, window, first)
    others = at[at != heavy_at]
    q = np.zeros((1, heads, 512))
    if spread:
        q[0, :, OWN:] = rng.normal(size=(heads, 512 - OWN))
        l = (bf16(q)[1][0] @ kv[others].T * BMM1)
        q[0] *= spread / l.std()
    l = bf16(q)[1][0] @ kv[others].T * BMM1
    total = torch.logsumexp(torch.from_numpy(l), dim=1).numpy()
    share = np.array([SHARES[h % len(SHARES)] for h in range(heads)])
    unit = np.abs(kv[heavy_at, :OWN]).sum() * BMM1         # the heavy row's logit for a query of its signs
    q[0, :, :OWN] = ((total + np.log(share / (1 - share))) / unit)[:, None] * sign[None, :]
    placed, scales = np.empty((pages, page, 512), np.uint8), np.full((pages, page // block), scale, np.float32)
    placed[order] = rows.reshape(pages, page, 512)
    g = dict(rows=torch.from_numpy(placed).to(DEV), scales=torch.from_numpy(scales).to(DEV),
             block_tables=i32(order[None]), seq_lens=i32([n]))
    return g, q, kv[at]


def call(g, q, window, first, splits):
    qt = bf16(q)[0]
    size = C.window_workspace_size(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], window=window,
                                   first_tokens=first, num_splits=splits)
    ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], ws, window=window,
                                  first_tokens=first, num_splits=splits, bmm1_scale=BMM1, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out.double().cpu().numpy()[0], lse.double().cpu().numpy()[0]


def check(got, q, kv):
    """Each head on its own: weights rounded to 2^-8 (uniformly: 2^-8.8 rms), the output to 2^-9 (2^-9.8 rms), and
    half a unit of 2^-8 for the rows that lie beside a heavy one: 2^-8 of the head's output in all."""
    want, lse = exact(bf16(q)[1][0], kv)
    err = np.sqrt(((got[0] - want) ** 2).mean(axis=1)) / np.sqrt((want ** 2).mean(axis=1))
    assert err.max() <= 2.0 ** -8, dict(enumerate(np.round(err, 5).tolist()))
    rest = np.sqrt(((got[0] - want)[:, OWN:] ** 2).mean(axis=1)) / np.sqrt((want[:, OWN:] ** 2).mean(axis=1))
    heavy = np.abs(want[:, :OWN]).max(axis=1) > 8 * np.abs(want[:, OWN:]).max(axis=1)   # (their own dims hide the rest)
    assert rest[~heavy].max(initial=0) <= 2.0 ** -7, dict(enumerate(np.round(rest, 5).tolist()))
    assert np.abs(got[1] - lse / math.log(2)).max() <= 2e-3


@pytest.mark.parametrize("n,window,first", [(100, 128, 0), (700, 512, 4), (2300, 2048, 4), (33000, 32768, 4)])
@pytest.mark.parametrize("amplitude", [0.25, 4.0, 40.0])
@pytest.mark.parametrize("spread,mean", [(0.0, 1.0), (1.0, 1.0), (1.0, 0.0)])
@pytest.mark.parametrize("splits", [1, 0])
def test_window_heavy_first_token_of_small_values(n, window, first, amplitude, spread, mean, splits):
    g, q, kv = make(n, n, window=window, first=first, amplitude=amplitude, spread=spread, mean=mean)
    check(call(g, q, window, first, splits), q, kv)


@pytest.mark.parametrize("heavy_at", [3, 130, 640, 1023])
@pytest.mark.parametrize("amplitude,size", [(0.0625, 60.0), (1.0, 60.0), (200.0, 60.0), (2.0 ** -9, 0.25), (2.0 ** -7, 8.0)])
@pytest.mark.parametrize("block", [1, 16])
def test_window_heavy_row_anywhere(heavy_at, amplitude, size, block):
    """In the first tile, between others, in the last one; codes down to E4M3's smallest, also beside rows all small."""
    g, q, kv = make(heavy_at, 1024, window=1100, first=0, amplitude=amplitude, spread=1.0, mean=1.0, heavy_at=heavy_at,
                    block=block, size=size)
    for splits in (1, 3):
        check(call(g, q, 1100, 0, splits), q, kv)


@pytest.mark.parametrize("nats", [6.0, 9.0, 10.0, 10.45, 12.0, 14.0, 20.0])
@pytest.mark.parametrize("n", [2052, 8192])
def test_window_one_row_above_equal_others(nats, n):
    """One row `nats` above thousands of equal weights; in units of one CTA and split."""
    g, q, kv = make(5, n, window=n, first=0, amplitude=16.0, spread=0.0, mean=1.0, heavy_at=n // 2 + 5)
    unit = np.abs(kv[n // 2 + 5, :OWN]).sum() * BMM1
    q[0, :, :OWN] = np.sign(kv[n // 2 + 5, :OWN])[None] * nats / unit
    for splits in (1, 0):
        check(call(g, q, n, 0, splits), q, kv)


@pytest.mark.parametrize("fall", [-40.0, -12.0, 12.0, 40.0])
def test_window_weights_that_fall_or_rise_along_the_sequence(fall):
    """Logits that move by `fall` nats from the first row to the last, over rows that share a mean: the reference
    follows them both ways, and what has become light does not count more than it is."""
    g, q, kv = make(9, 4096, window=4096, first=0, amplitude=1.0, spread=0.0, mean=1.0)
    codes = R.e4m3(g["rows"].cpu().numpy())
    order = g["block_tables"].cpu().numpy()[0]
    flat = codes[order].reshape(4096, 512)
    flat[:, 0] = np.linspace(0, 240, 4096)                 # the position, which the queries read
    flat[:, 1:OWN] = 0
    flat = R.to_e4m3(flat)
    placed = np.empty_like(g["rows"].cpu().numpy())
    placed[order] = flat.reshape(-1, 64, 512)
    g["rows"] = torch.from_numpy(placed).to(DEV)
    kv = R.e4m3(flat) * 2.0 ** -6
    q[:] = 0
    q[0, :, 0] = -fall / (240 * 2.0 ** -6 * BMM1) * np.linspace(0.5, 1.0, 64)
    for splits in (1, 0):
        check(call(g, q, 4096, 0, splits), q, kv)


def test_window_zero_rows_keep_their_weight():
    """Rows of zeros carry weight and no value, however much of it: the others' share of the output stays exact."""
    for zeros in (1, 130):
        g, q, kv = make(11, 600, window=600, first=0, amplitude=1.0, spread=1.0, mean=1.0)
        order, rows = g["block_tables"].cpu().numpy()[0], g["rows"].cpu().numpy()
        flat = rows[order].reshape(-1, 512)
        flat[:zeros] = 0
        rows[order] = flat.reshape(rows.shape)
        g["rows"] = torch.from_numpy(rows).to(DEV)
        kv = R.e4m3(flat[:600]) * 2.0 ** -6
        q[0, :, :OWN] = 0
        q[0, :, OWN:] -= 0.5 * np.linspace(0, 1, 64)[:, None] * kv[zeros:, OWN:].mean(axis=0)   # the others fall below 0
        for splits in (1, 0):
            check(call(g, q, 600, 0, splits), q, kv)


@pytest.mark.parametrize("heads", [64, 128])
def test_window_heavy_first_token_in_a_prompt(heads):
    """Hundreds of tokens: every CTA takes several units one behind another, each with its own heavy rows."""
    n, tokens, window, first = 900, 400, 300, 4
    g, q, kv_last = make(21, n, window=window, first=first, amplitude=1.0, spread=1.0, mean=1.0, heads=heads)
    order = g["block_tables"].cpu().numpy()[0]
    kv = R.e4m3(g["rows"].cpu().numpy()[order].reshape(-1, 512)[:n]) * 2.0 ** -6
    rng = np.random.default_rng(22)
    q = np.repeat(q, tokens, axis=0)
    q[:, :, :OWN] *= rng.uniform(0.6, 1.1, size=(tokens, heads, 1))     # (each token its own share)
    qt = bf16(q)[0]
    for splits in (1, 0):
        size = C.window_workspace_size(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], window=window,
                                       first_tokens=first, num_splits=splits)
        ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device=DEV)
        out, lse = C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], ws, window=window,
                                      first_tokens=first, num_splits=splits, bmm1_scale=BMM1)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for t in range(0, tokens, 7):
            pos = n - tokens + t
            check((out[t], lse[t]), q[t:t + 1], kv[:pos + 1][visible(pos + 1, window, first)])


@pytest.mark.parametrize("zeros,size", [(3000, 3400), (600000, 600100)])
def test_window_rows_of_zeros_at_the_smallest_scale(zeros, size):
    """Zero latents as the append holds them, codes of 0 with a scale of 2^-64, in front of rows whose logits lie up to
    75 below theirs: the sums of weights over scales stay finite and in step with the reference, so the LSE is right,
    and so is the output of what lies above 2^-44 of a row of zeros (which counts as a part of 2^-40)."""
    page, heads = 64, 64
    pages = -(-size // page)
    rng = np.random.default_rng(31)
    rows = torch.zeros(pages, page, 512, dtype=torch.uint8, device=DEV)
    scales = torch.full((pages, 4), 2.0 ** -64, device=DEV)
    codes = R.to_e4m3((rng.normal(size=(size - zeros, 512)) * 0.3 + np.abs(rng.normal(size=512))) * 60)
    flat = rows.view(-1, 512)
    at = zeros // 16 * 16                                  # whole blocks from here on (their first rows stay zeros)
    flat[zeros:size] = torch.from_numpy(codes).to(DEV)
    scales.view(-1)[at // 16:] = 2.0 ** -6
    g = dict(rows=rows, scales=scales, block_tables=i32(np.arange(pages)[None]), seq_lens=i32([size]))
    kv = R.e4m3(codes) * 2.0 ** -6
    mean = kv.mean(axis=0)
    fall = np.linspace(1.0, 75.0, heads)                   # nats by which the others lie below the zeros, per head
    q = (-fall[:, None] * mean[None] / (mean @ mean * BMM1))[None]
    qv = bf16(q)[1][0]
    l = torch.from_numpy(qv @ kv.T * BMM1)
    total = torch.logsumexp(torch.cat([l, torch.full((heads, 1), math.log(zeros), dtype=torch.float64)], dim=1), dim=1)
    want = (torch.exp(l - total[:, None]) @ torch.from_numpy(kv)).numpy()
    for splits in (1, 0):
        out, lse = call(g, q, size, 0, splits)
        assert np.abs(lse - total.numpy() / math.log(2)).max() <= 2e-3
        err = np.sqrt(((out - want) ** 2).mean(axis=1)) / np.sqrt((want ** 2).mean(axis=1))
        seen = fall < 44 * math.log(2)
        assert err[seen].max() <= 2.0 ** -8, err.round(5).tolist()


@pytest.mark.parametrize("code,scale", [(0x00, 2.0 ** -64), (0x38, 2.0 ** -64), (0x00, 1.0), (0x38, 1.0)])
def test_window_reference_and_sums_stay_in_step(code, scale):
    """Thousands of tiles that each move the reference by a rounding or nothing: the LSE of n equal rows is log2 n, off
    by fp32 additions of a few thousand terms (2^-14) at most."""
    n, page = 300000, 64
    pages = -(-n // page)
    rows = torch.full((pages, page, 512), code, dtype=torch.uint8, device=DEV)
    g = dict(rows=rows, scales=torch.full((pages, 4), scale, device=DEV), block_tables=i32(np.arange(pages)[None]),
             seq_lens=i32([n]))
    for splits in (1, 2, 0):
        _, lse = call(g, np.zeros((1, 64, 512)), n, 0, splits)
        assert np.abs(lse - math.log2(n)).max() <= 2.0 ** -14


def test_window_rows_of_zeros_among_rows_of_small_codes():
    """Rows of zeros, of E4M3's smallest numbers and of codes under 8 in one tile: whatever is multiplied up stays exact."""
    rng = np.random.default_rng(33)
    n, page = 500, 64
    codes = rng.normal(size=(512, 512)) * 1.5 + rng.normal(size=512)
    codes[::7] = 0
    codes[1::7] *= 2.0 ** -9
    codes[2::7] *= 2.0 ** -5
    rows = R.to_e4m3(codes)
    g = dict(rows=torch.from_numpy(rows.reshape(8, page, 512)).to(DEV), scales=torch.ones(8, 4, device=DEV),
             block_tables=i32(np.arange(8)[None]), seq_lens=i32([n]))
    kv = R.e4m3(rows)[:n]
    q = rng.normal(size=(1, 64, 512)) * np.linspace(0, 6, 64)[None, :, None]
    q[0, 32:] -= 3 * kv[3::7].mean(axis=0)                 # (half of the heads put the zeros first)
    for splits in (1, 3, 0):
        check(call(g, q, n, 0, splits), q, kv)
