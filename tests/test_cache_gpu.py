"""The paged latent cache on the GPU against its 64-bit reference: the window
attention over every kind of page, window, split and masked neighbour; the
append's codes and scales exactly; the page calls' tables, counts and moves
exactly; and a serving loop of all of them together."""
import math

import numpy as np
import pytest
import torch

import cache_reference as R
from sparse_mla_decode_token_gb300 import binding as B
from sparse_mla_decode_token_gb300 import cache as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_decode_token_gb300 import build
    build.build()
    B.lib()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def bf16(a):
    """BF16 tensor of an array, and the values it holds in float64."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.to(torch.float64).numpy()


def make(seed, lens, q_lens, *, heads=64, page_size=64, block=16, spare=3, amplitude=1.0, scale_exp=(-8, -5), junk=True):
    """A cache of random rows whose requests own random pages.  With `junk`, all
    that no request owns holds NaN codes, NaN scales and impossible pages."""
    rng = np.random.default_rng(seed)
    lens, q_lens = np.asarray(lens), np.asarray(q_lens)
    need = [-(-max(int(n), 0) // page_size) for n in lens]
    width = max(need) + 1
    pages = sum(need) + spare
    order = rng.permutation(pages)
    tables = np.full((len(lens), width), -77 if junk else -1, dtype=np.int32)
    rows = np.full((pages, page_size, 512), 0x7F, dtype=np.uint8)
    scales = np.full((pages, page_size // block), np.nan, dtype=np.float32)
    if not junk:
        rows[:], scales[:] = 0x38, 1.0
    used = 0
    for b, n in enumerate(need):
        tables[b, :n] = order[used:used + n]
        used += n
        for j0 in range(0, int(lens[b]), block):
            page, r = tables[b, j0 // page_size], j0 % page_size
            scales[page, r // block] = 2.0 ** rng.integers(*scale_exp)
            k = min(block, int(lens[b]) - j0)
            rows[page, r:r + k] = R.to_e4m3(rng.normal(size=(k, 512)) * 100.0 * amplitude)
    cum = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    cache = R.Cache(rows, scales, tables, lens, cum=cum)
    q = rng.normal(size=(int(cum[-1]), heads, 512))
    return cache, q, rng


def on_gpu(cache):
    return dict(rows=torch.from_numpy(cache.rows).to(DEV), scales=torch.from_numpy(cache.scales).to(DEV),
                block_tables=i32(cache.tables), seq_lens=i32(cache.lens))


def workspace(q, g, **kw):
    n = C.window_workspace_size(q, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], **kw)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)


def run(cache, q, *, window, first=0, sinks=None, bmm1=1 / math.sqrt(512), bmm2=1.0, splits=0, g=None, uniform=False,
        q_gpu=None, expect_flag=0):
    g = on_gpu(cache) if g is None else g
    qt = bf16(q)[0] if q_gpu is None else q_gpu
    cum = None if uniform else i32(cache.cum)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = workspace(qt, g, window=window, first_tokens=first, cum_seq_lens_q=cum, num_splits=splits)
    ws.fill_(0xFF)                                         # partials and scratch that are not written are NaN
    out = torch.full(qt.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(qt.shape[:2], float("nan"), device=DEV)
    C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], ws, window=window,
                       first_tokens=first, cum_seq_lens_q=cum, num_splits=splits, bmm1_scale=bmm1, bmm2_scale=bmm2,
                       sinks=None if sinks is None else torch.from_numpy(sinks.astype(np.float32)).to(DEV),
                       out=out, out_lse=lse, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == expect_flag
    return out.to(torch.float64).cpu().numpy(), lse.to(torch.float64).cpu().numpy()


def check(cache, q, got, **kw):
    out, lse, tol_o, tol_l = R.window(cache, bf16(q)[1], bmm1=kw.pop("bmm1", 1 / math.sqrt(512)), **kw)
    empty, nan = np.isneginf(lse), np.isnan(lse)           # (a token that sees a NaN row)
    assert np.array_equal(np.isneginf(got[1]), empty) and np.array_equal(np.isnan(got[1]), nan)
    assert np.all(got[0][empty] == 0) and np.all(np.isnan(got[0][nan]) == np.isnan(out[nan]))
    fin = ~empty & ~nan
    bad = (np.abs(got[0] - out) > tol_o) & fin[..., None]
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got[0] - out)[bad][:5], tol_o[bad][:5])
    assert np.all(np.abs(got[1][fin] - lse[fin]) <= tol_l[fin])
    # far inside the worst case: rounding errors of either sign, as the square root of their number
    if fin.any():
        scale = np.sqrt((out[fin] ** 2).mean())
        assert np.sqrt(((got[0] - out)[fin] ** 2).mean()) <= 2.0 ** -8 * scale + 1e-30


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("heads", [1, 16, 63, 64, 65, 128])
@pytest.mark.parametrize("window,first", [(1, 0), (7, 3), (128, 4), (300, 130)])
def test_window_heads_and_windows(heads, window, first):
    cache, q, rng = make(heads * 1000 + window, [1, 5, 128, 129, 470], [1, 2, 1, 3, 2], heads=heads)
    sinks = rng.normal(size=heads)
    check(cache, q, run(cache, q, window=window, first=first, sinks=sinks), window=window, first=first, sinks=sinks)


@pytest.mark.parametrize("page_size,block", [(8, 8), (8, 1), (16, 4), (24, 3), (24, 24), (32, 32), (40, 8), (64, 64),
                                             (128, 16), (144, 9), (256, 128)])
@pytest.mark.parametrize("splits", [1, 0])
def test_window_page_and_block_sizes(page_size, block, splits):
    cache, q, _ = make(page_size + block, [333, 97, 700], [2, 1, 1], page_size=page_size, block=block)
    check(cache, q, run(cache, q, window=200, first=5, splits=splits), window=200, first=5)


@pytest.mark.parametrize("splits", [1, 2, 3, 8, 64])
def test_window_splits(splits):
    """Also more splits than a token has tiles: the last ones are empty."""
    cache, q, rng = make(7, [1, 600, 1000, 0], [1, 2, 1, 1], heads=128)
    sinks = rng.normal(size=128)
    check(cache, q, run(cache, q, window=700, first=4, sinks=sinks, splits=splits), window=700, first=4, sinks=sinks)


def test_window_positions_before_and_behind():
    """More new tokens than the sequence is long (positions below 0 see nothing),
    requests without tokens, and lengths past what the table holds."""
    cache, q, _ = make(8, [3, 64, 1, 200, 80], [5, 0, 1, 0, 70])
    check(cache, q, run(cache, q, window=40, first=2), window=40, first=2)
    cache.lens = np.array([3, 64, 1, 200, 1000])           # the last request's table ends at 4 * 64 tokens ...
    cache.tables[4, 2:] = cache.tables[3, 0]               # ... all of them backed
    cache.rows[cache.tables[3, 0]] = 0x38
    cache.scales[cache.tables[3, 0]] = 1.0
    got = run(cache, q, window=900, first=2, expect_flag=B.DEVERR_INDEX_OUT_OF_RANGE)
    check(cache, q, got, window=900, first=2)


@pytest.mark.parametrize("splits", [1, 3])
def test_window_bad_pages_are_masked_and_flagged(splits):
    cache, q, _ = make(9, [500, 300], [2, 1])
    cache.tables[0, 2], cache.tables[0, 5], cache.tables[1, 4] = -1, cache.rows.shape[0], 2 ** 31 - 1
    got = run(cache, q, window=400, first=3, splits=splits, expect_flag=B.DEVERR_INDEX_OUT_OF_RANGE)
    check(cache, q, got, window=400, first=3)
    cache.tables[1, :] = -5                                # nothing is left of the second request
    got = run(cache, q, window=400, first=3, splits=splits, expect_flag=B.DEVERR_INDEX_OUT_OF_RANGE)
    check(cache, q, got, window=400, first=3)


def test_window_uniform_batch_many_units():
    """More units than SMs, without offsets: every CTA takes several, some of them empty."""
    lens = [(37 * k) % 260 for k in range(96)]
    cache, q, _ = make(10, lens, [2] * 96, heads=128, page_size=32)
    check(cache, q, run(cache, q, window=150, first=4, uniform=True), window=150, first=4)


def test_window_prefill_many_units():
    cache, q, _ = make(11, [330, 5, 129], [300, 5, 60], heads=64, page_size=16)
    check(cache, q, run(cache, q, window=100, first=1), window=100, first=1)


@pytest.mark.parametrize("splits", [1, 0])
def test_window_many_units_of_many_tiles(splits):
    """CTAs take two units of up to eight tiles: buffers and barriers go through many turns between them.  On its
    own the call splits the last few units and does the others whole."""
    lens = [600 + 5 * k for k in range(80)]
    cache, q, _ = make(22, lens, [1] * 80, heads=128)
    check(cache, q, run(cache, q, window=900, first=4, splits=splits), window=900, first=4)


def test_window_longer_than_the_sequence_is_causal():
    cache, q, _ = make(12, [140, 300], [140, 3])
    a = run(cache, q, window=2 ** 31 - 1)
    check(cache, q, a, window=10 ** 6)
    b = run(cache, q, window=1, first=2 ** 31 - 1)
    check(cache, q, b, window=10 ** 6)


def test_window_strided_tensors():
    """Rows 528 bytes apart, pages with a gap, scales and tables cut from wider
    arrays, query tokens from a wider buffer."""
    cache, q, _ = make(13, [200, 90], [1, 2], page_size=16, block=8)
    n = cache.rows.shape[0]
    rows = torch.full((n, 16 * 528 + 64), 0x7F, dtype=torch.uint8, device=DEV)
    view = rows[:, :16 * 528].view(n, 16, 528)[:, :, :512]
    view.copy_(torch.from_numpy(cache.rows))
    scales = torch.full((n, 5), float("nan"), device=DEV)
    scales[:, :2] = torch.from_numpy(cache.scales).to(DEV)
    tables = torch.full((2, cache.tables.shape[1] + 3), -9, dtype=torch.int32, device=DEV)
    tables[:, :-3] = i32(cache.tables)
    wide = torch.zeros(3, 70, 512, dtype=torch.bfloat16, device=DEV)
    wide[:, :64] = bf16(q)[0]
    g = dict(rows=view, scales=scales[:, :2], block_tables=tables[:, :-3], seq_lens=i32(cache.lens))
    check(cache, q, run(cache, q, window=120, first=4, g=g, q_gpu=wide[:, :64]), window=120, first=4)


@pytest.mark.parametrize("bmm1,bmm2", [(0.2, -0.5), (1e-4, 3.0), (-0.05, 1.0)])
def test_window_scales_as_device_tensors(bmm1, bmm2):
    cache, q, _ = make(14, [260], [2])
    got = run(cache, q, window=200, bmm1=torch.tensor([bmm1], device=DEV), bmm2=torch.tensor([bmm2], device=DEV))
    b1, b2 = float(np.float32(bmm1)), float(np.float32(bmm2))
    check(cache, q, got, window=200, bmm1=b1, bmm2=b2)
    check(cache, q, run(cache, q, window=200, bmm1=bmm1, bmm2=bmm2, splits=1), window=200, bmm1=b1, bmm2=b2)


def test_window_block_scales_far_apart():
    """Blocks of 2^-30 beside blocks of 2^0 and blocks of scale 0 (rows of zeros)."""
    cache, q, rng = make(15, [400], [2], scale_exp=(-30, 1), amplitude=0.01)
    page = cache.tables[0, 1]
    cache.scales[page, 0] = 0.0
    check(cache, q, run(cache, q, window=350, first=8), window=350, first=8)
    cache.scales[:, :] = 0.0                               # every logit is 0, every value too
    out, lse = run(cache, q, window=350)
    assert np.all(np.abs(out) < 1e-15) and np.allclose(lse, math.log2(350), atol=1e-5)


def test_window_large_logits_and_growing_maximum():
    """Logits of some hundreds, largest last: the reference moves at every tile."""
    cache, q, _ = make(16, [640], [1], scale_exp=(-4, -3))
    for j in range(640):
        page, r = cache.page(0, j), j % 64
        cache.rows[page, r] = R.to_e4m3(R.e4m3(cache.rows[page, r]) * (j + 1) / 640)
    for order in (1, -1):
        if order < 0:
            cache.tables[0, :10] = cache.tables[0, :10][::-1].copy()
        check(cache, q, run(cache, q, window=640, bmm1=0.5), window=640, bmm1=0.5)


def test_window_query_magnitudes():
    """Heads of 2^-40 and 2^20, a head of zeros, outlier dims of 2^12 times the others."""
    cache, q, _ = make(17, [300], [1], scale_exp=(-7, -6))
    q[0, 0] *= 2.0 ** -40
    q[0, 1] *= 2.0 ** 20
    q[0, 2] = 0.0
    q[0, 3, ::64] *= 2.0 ** 12
    q[0, 4] = 2.0 ** -130                                  # subnormal BF16
    bmm1 = 2.0 ** -18
    check(cache, q, run(cache, q, window=256, bmm1=bmm1), window=256, bmm1=bmm1)


def test_window_nan_and_infinity():
    """A query head with NaN or infinity is NaN alone; a visible NaN row makes its
    token's heads NaN and no other token's."""
    cache, q, _ = make(18, [200, 200], [1, 1])
    qb = bf16(q)[0]
    qb[0, 3, 17], qb[0, 5, 100] = float("nan"), float("inf")
    keep = [h for h in range(64) if h not in (3, 5)]
    out, lse, tol_o, tol_l = R.window(cache, bf16(q)[1], window=150, bmm1=1 / math.sqrt(512))
    for splits in (1, 2, 0):
        got = run(cache, q, window=150, q_gpu=qb, splits=splits)
        assert np.isnan(got[0][0, [3, 5]]).all() and np.isnan(got[1][0, [3, 5]]).all()
        assert np.all(np.abs(got[0][0, keep] - out[0, keep]) <= tol_o[0, keep])
        assert np.all(np.abs(got[0][1] - out[1]) <= tol_o[1])
    cache.rows[cache.page(0, 190), 190 % 64, 5] = 0x7F
    for splits in (1, 2, 0):
        got = run(cache, q, window=150, splits=splits)
        assert np.isnan(got[1][0]).all() and np.isnan(got[0][0, :, 5]).all()
        assert np.all(np.abs(got[0][1] - out[1]) <= tol_o[1])


def test_window_is_deterministic_and_replays_from_a_graph():
    """Captured on a side stream; the lengths and queries of a replay are those of that moment."""
    cache, q, _ = make(19, [400, 380, 64], [2, 1, 1], heads=128)
    g = on_gpu(cache)
    qt, cum = bf16(q)[0], i32(cache.cum)
    for splits in (1, 0):
        ws = workspace(qt, g, window=300, first_tokens=4, cum_seq_lens_q=cum, num_splits=splits)
        out, lse = torch.empty_like(qt), torch.empty(qt.shape[:2], device=DEV)

        def call():
            C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], ws, window=300,
                               first_tokens=4, cum_seq_lens_q=cum, num_splits=splits, out=out, out_lse=lse,
                               bmm1_scale=1 / math.sqrt(512))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                call()
        torch.cuda.synchronize()
        first = None
        for lens in ([400, 380, 64], [399, 210, 3], [400, 380, 64]):
            g["seq_lens"].copy_(i32(lens))
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            cache.lens = np.array(lens)
            check(cache, q, (out.to(torch.float64).cpu().numpy(), lse.to(torch.float64).cpu().numpy()), window=300, first=4)
            if lens[0] == 400:
                assert first is None or torch.equal(first, out)
                first = out.clone()


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("heads", [64, 80])
def test_window_padded_batch(splits, heads):
    """Tokens before the first offset and behind the last one are no request's: their outputs stay as they were."""
    cache, q, rng = make(26, [700, 40, 300], [2, 0, 3], heads=heads)
    lead, behind = 2, 4
    pad = rng.normal(size=(lead + behind, heads, 512))
    q_all = np.concatenate([pad[:lead], q, pad[lead:]])
    g = on_gpu(cache)
    cum = i32(np.concatenate([cache.cum + lead, [5 + lead]]))      # (and a request without tokens at the end)
    g["block_tables"] = torch.cat([g["block_tables"], torch.full_like(g["block_tables"][:1], -77)])
    g["seq_lens"] = torch.cat([g["seq_lens"], i32([900])])
    qt = bf16(q_all)[0]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = workspace(qt, g, window=500, first_tokens=5, cum_seq_lens_q=cum, num_splits=splits)
    ws.fill_(0xFF)
    out, lse = torch.full_like(qt, 7.0), torch.full(qt.shape[:2], 7.0, device=DEV)
    C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], ws, window=500, first_tokens=5,
                       cum_seq_lens_q=cum, num_splits=splits, bmm1_scale=1 / math.sqrt(512), out=out, out_lse=lse,
                       error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for part in (slice(0, lead), slice(lead + 5, None)):
        assert bool((out[part] == 7).all()) and bool((lse[part] == 7).all())
    own = slice(lead, lead + 5)
    check(cache, q, (out[own].double().cpu().numpy(), lse[own].double().cpu().numpy()), window=500, first=5)


def test_offsets_that_fall_stay_inside_the_arrays():
    """Offsets that are none give no result that counts, but write nothing outside the call's own tensors."""
    rng = np.random.default_rng(27)
    batch = 70
    cache, _, _ = make(27, [64] * batch, [1] * batch, junk=False)
    g = on_gpu(cache)
    qt, x = bf16(rng.normal(size=(batch, 64, 512)))[0], bf16(rng.normal(size=(batch, 512)))[0]
    for cum in (np.arange(batch, -1, -1), rng.integers(-5, 90, size=batch + 1), rng.permutation(batch + 1)):
        # the arrays lie inside larger ones: what is read behind them would be impossible pages
        wide = torch.full((3 * batch + 1,), 1 << 30, dtype=torch.int32, device=DEV)
        wide[batch:2 * batch + 1] = i32(cum)
        lens = torch.full((3 * batch,), 1 << 30, dtype=torch.int32, device=DEV)
        lens[batch:2 * batch] = 64
        before = wide.clone()
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        for splits in (1, 2):
            ws = workspace(qt, g, window=64, cum_seq_lens_q=wide[batch:2 * batch + 1], num_splits=splits)
            C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], lens[batch:2 * batch], ws, window=64,
                               cum_seq_lens_q=wide[batch:2 * batch + 1], num_splits=splits, error_word=err)
        C.append(x, g["rows"], g["scales"], g["block_tables"], lens[batch:2 * batch],
                 cum_seq_lens_q=wide[batch:2 * batch + 1], error_word=err)
        torch.cuda.synchronize()
        assert torch.equal(before, wide) and not int(err.item()) & B.DEVERR_TIMEOUT


def test_window_workspace_too_small_is_refused():
    cache, q, _ = make(20, [1000], [1])
    g, qt = on_gpu(cache), bf16(q)[0]
    with pytest.raises(B.SmlaError) as e:
        C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], None, window=900, num_splits=4)
    assert e.value.status == B.SMLA_ERR_WORKSPACE_TOO_SMALL
    assert C.window_workspace_size(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], window=900, num_splits=1) == 0


def test_empty_calls():
    cache, q, _ = make(21, [10], [1])
    g = on_gpu(cache)
    out, lse = C.window_attention(torch.empty(0, 64, 512, dtype=torch.bfloat16, device=DEV), g["rows"], g["scales"],
                                  g["block_tables"], g["seq_lens"], None, window=4)
    assert out.shape == (0, 64, 512) and lse.shape == (0, 64)
    before = g["rows"].clone()
    C.append(torch.empty(0, 512, dtype=torch.bfloat16, device=DEV), g["rows"], g["scales"], g["block_tables"], g["seq_lens"])
    assert torch.equal(before, g["rows"])


# ------------------------------------------------------------------ append

def append_both(cache, latent, g=None, uniform=False, expect_flag=0, latent_gpu=None):
    g = on_gpu(cache) if g is None else g
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    xt = bf16(latent)[0] if latent_gpu is None else latent_gpu
    C.append(xt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"],
             cum_seq_lens_q=None if uniform else i32(cache.cum), error_word=err)
    R.append(cache, xt.float().cpu().numpy())
    torch.cuda.synchronize()
    assert int(err.item()) == expect_flag
    rows, scales = g["rows"].cpu().numpy(), g["scales"].cpu().numpy()
    # NaN codes have no sign or payload that counts
    nan = np.isin(rows, (0x7F, 0xFF)) & np.isin(cache.rows, (0x7F, 0xFF))
    assert np.array_equal(np.where(nan, 0, rows), np.where(nan, 0, cache.rows))
    assert np.array_equal(scales, cache.scales, equal_nan=True)


@pytest.mark.parametrize("page_size,block", [(8, 1), (8, 8), (16, 2), (24, 3), (64, 16), (64, 64), (120, 40), (256, 128)])
def test_append_codes_and_scales(page_size, block):
    """New blocks, blocks that hold older tokens (whose scale grows or not), requests without tokens; rows and
    blocks behind the sequences stay as they were."""
    cache, _, rng = make(30 + page_size, [1, 9, 130, 77, 300, 64], [1, 9, 3, 0, 250, 1], page_size=page_size, block=block)
    x = rng.normal(size=(int(cache.cum[-1]), 512)) * 2.0 ** rng.integers(-20, 20, size=(int(cache.cum[-1]), 1))
    append_both(cache, x)


@pytest.mark.parametrize("magnitude", [1e-30, 1e-19, 0.01, 1.0, 448.0, 449.0, 1e19, 1e25, 3e38])
def test_append_magnitudes(magnitude):
    """Exponents from below 2^-64 to above 2^64 (there values saturate)."""
    cache, _, rng = make(40, [70, 40], [9, 40])
    x = rng.uniform(-1, 1, size=(49, 512)) * magnitude
    x[:, 7] = magnitude
    append_both(cache, x)


def test_append_special_values():
    """Zeros alone take the smallest scale; NaN stays NaN, infinities saturate, neither counts toward the scale."""
    cache, _, rng = make(41, [64, 16, 32, 20], [64, 16, 32, 4])
    x = rng.normal(size=(116, 512))
    x[:64] = 0.0
    x[64 + 3, 5], x[64 + 3, 6], x[64 + 4, 7] = np.nan, np.inf, -np.inf
    x[80:96] = np.nan
    append_both(cache, x)


def test_append_older_rows_and_foreign_scales():
    """Older rows in a block whose scale the caller made: any positive number, and 0 or infinity, which count as none."""
    for old in (0.3, 1e-3, 0.0, np.inf):
        cache, _, rng = make(42, [21, 37], [3, 2])
        cache.scales[cache.page(0, 16), 1] = old
        cache.scales[cache.page(1, 32), 2] = old
        append_both(cache, rng.normal(size=(5, 512)) * 30)


def test_append_token_by_token_is_append_at_once():
    """For magnitudes of one binade the scale never moves after a block's first row: one call or many, the same."""
    rng = np.random.default_rng(43)
    x = rng.uniform(1.0, 1.9, size=(50, 512)) * rng.choice([-1, 1], size=(50, 512))
    one, _, _ = make(44, [50], [50])
    g1 = on_gpu(one)
    append_both(one, x, g=g1)
    many, _, _ = make(44, [50], [50])
    g2 = on_gpu(many)
    for n in range(1, 51):
        many.lens, many.cum = np.array([n]), np.array([0, 1])
        g2["seq_lens"] = i32([n])
        append_both(many, x[n - 1:n], g=g2, uniform=True)
    assert torch.equal(g1["rows"], g2["rows"]) and torch.equal(g1["scales"].nan_to_num(), g2["scales"].nan_to_num())


def test_append_skips_and_flags_what_has_no_place():
    cache, _, rng = make(45, [3, 100, 64], [5, 40, 1])     # positions below 0
    x = rng.normal(size=(46, 512))
    append_both(cache, x, expect_flag=B.DEVERR_INDEX_OUT_OF_RANGE)
    cache, _, _ = make(45, [300, 100, 64], [5, 40, 1])
    cache.tables[1, 1], cache.tables[2, 0] = cache.rows.shape[0], -1
    append_both(cache, x, expect_flag=B.DEVERR_INDEX_OUT_OF_RANGE)
    cache, _, _ = make(45, [300, 100, 64], [5, 40, 1], junk=False)
    cache.tables = cache.tables[:, :2].copy()              # the first request is longer than its table
    append_both(cache, x, expect_flag=B.DEVERR_INDEX_OUT_OF_RANGE)


def test_append_padded_batch():
    cache, _, rng = make(49, [200, 33], [30, 2])
    x = rng.normal(size=(40, 512))
    x[32:] = np.nan                                        # behind the last offset: not looked at
    append_both(cache, x)


def test_append_strided_tensors():
    cache, _, rng = make(46, [200, 90], [30, 2], page_size=16, block=8)
    n = cache.rows.shape[0]
    store = torch.full((n, 16 * 544 + 32), 0x55, dtype=torch.uint8, device=DEV)
    view = store[:, :16 * 544].view(n, 16, 544)[:, :, :512]
    view.copy_(torch.from_numpy(cache.rows))
    scales = torch.full((n, 3), 7.0, device=DEV)
    scales[:, :2] = torch.from_numpy(cache.scales).to(DEV)
    x = torch.full((32, 528), float("nan"), dtype=torch.bfloat16, device=DEV)
    x[:, :512] = bf16(rng.normal(size=(32, 512)))[0]
    g = dict(rows=view, scales=scales[:, :2], block_tables=i32(cache.tables), seq_lens=i32(cache.lens))
    append_both(cache, None, g=g, latent_gpu=x[:, :512])
    gap = store[:, :16 * 544].view(n, 16, 544)[:, :, 512:]
    assert bool((gap == 0x55).all()) and bool((store[:, 16 * 544:] == 0x55).all()) and bool((scales[:, 2] == 7).all())


# ------------------------------------------------------------------- pages

class Both:
    """The reference and the GPU's state, stepped together and compared."""

    def __init__(self, rows, max_pages, page_size, num_pages, lens=None):
        self.ref = R.Pages(rows, max_pages, page_size, num_pages)
        self.lens = np.zeros(rows, dtype=np.int32)
        self.tables, self.refs = i32(self.ref.tables), i32(self.ref.refs)
        self.moves = C.new_moves(max(rows, num_pages // 2), DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.full((C.pages_workspace_size(self.tables, self.refs, page_size),), 0x7F, dtype=torch.uint8,
                             device=DEV)
        if lens is not None:
            self.resize(lens)

    def compare(self, moves=None, flags=0):
        torch.cuda.synchronize()
        assert np.array_equal(self.tables.cpu().numpy(), self.ref.tables)
        assert np.array_equal(self.refs.cpu().numpy(), self.ref.refs)
        if moves is not None:
            n = int(self.moves.count.item())
            got = list(zip(self.moves.src[:n].tolist(), self.moves.dst[:n].tolist()))
            assert got == [(int(a), int(b)) for a, b in moves]
        assert int(self.err.item()) == flags
        self.err.zero_()

    def resize(self, new, flags=0):
        new = np.asarray(new, dtype=np.int32)
        moves, short = self.ref.resize(self.lens, new)
        C.pages_resize(self.tables, self.refs, i32(self.lens), i32(new), self.ws, page_size=self.ref.page_size,
                       moves=self.moves, error_word=self.err)
        self.compare(moves, flags | (B.DEVERR_OUT_OF_PAGES if short else 0))
        self.lens = new
        return moves

    def fork(self, parents, flags=0):
        out = torch.full((len(parents),), -3, dtype=torch.int32, device=DEV)
        C.pages_fork(self.tables, self.refs, i32(self.lens), i32(parents), out, page_size=self.ref.page_size,
                     error_word=self.err)
        self.lens = self.ref.fork(self.lens, parents).astype(np.int32)
        self.compare(None, flags)
        assert np.array_equal(out.cpu().numpy(), self.lens)

    def compact(self):
        moves = self.ref.compact(self.lens)
        C.pages_compact(self.tables, self.refs, i32(self.lens), self.ws, page_size=self.ref.page_size,
                        moves=self.moves, error_word=self.err)
        self.compare(moves)
        return moves


# small: one cluster; large (tables + pool past 131,072 entries): launches over the whole GPU
SIZES = [(1, 1, 1, 1), (1, 5, 3, 7), (7, 9, 16, 80), (40, 33, 8, 1500), (130, 140, 4, 3000), (300, 500, 1, 160000),
         (3, 200, 64, 140001)]


@pytest.mark.parametrize("rows,max_pages,page_size,num_pages", SIZES)
def test_pages_random_walk(rows, max_pages, page_size, num_pages):
    """Growing, shrinking, ending, forking and compacting at random; now and then the pool runs out."""
    rng = np.random.default_rng(rows * 7 + num_pages)
    b = Both(rows, max_pages, page_size, num_pages)
    cap = max_pages * page_size
    for step in range(8):
        new = rng.integers(0, cap + 1, size=rows)
        new = np.where(rng.random(rows) < 0.3, 0, np.where(rng.random(rows) < 0.3, b.lens, new))
        # (a request that found no page holds -1: end it before it is used further)
        held = np.array([all(b.ref.tables[r, c] >= 0 for c in range(b.ref.columns(b.lens[r]))) for r in range(rows)])
        if not held.all():
            keep = np.array([next((c for c in range(b.ref.columns(b.lens[r])) if b.ref.tables[r, c] < 0),
                                  b.ref.columns(b.lens[r])) * page_size if not held[r] else b.lens[r] for r in range(rows)])
            b.lens = np.minimum(b.lens, keep).astype(np.int32)
            b.resize(np.minimum(b.lens, new))
        b.resize(new)
        if all(b.ref.tables[r, c] >= 0 for r in range(rows) for c in range(b.ref.columns(b.lens[r]))):
            empty, full = np.flatnonzero(b.lens == 0), np.flatnonzero(b.lens > 0)
            if len(empty) and len(full):
                parents = np.full(rows, -1)
                take = empty[rng.random(len(empty)) < 0.7]
                parents[take] = rng.choice(full, size=len(take))
                b.fork(parents)
            b.compact()


def test_pages_copy_on_write_and_rollback():
    b = Both(6, 8, 16, 40, lens=[33, 16, 0, 0, 0, 0])
    b.fork(np.array([-1, -1, 0, 0, 1, -1]))                # 0 shared by three, its last page partly filled; 1's is full
    assert b.resize(b.lens + (b.lens > 0)) != []           # a copy for each sharer of the partial page, none for 1 and 4
    b.resize([20, 5, 34, 0, 17, 100])                      # cut back into shared pages
    moves = b.resize([21, 5, 34, 0, 18, 100])              # ... and grown there: copied first
    assert len(moves) == 1
    b.compact()


def test_pages_out_of_pages_in_order():
    """The last entries go without, a copy among them keeps the shared page."""
    b = Both(4, 4, 4, 6, lens=[6, 0, 0, 0])
    b.fork(np.array([-1, 0, 0, 0]))
    b.resize([16, 7, 7, 7])                                # 2 + 1 copies and pages: 4 free
    assert (b.ref.tables[3, 1] == b.ref.tables[2, 1]) or (b.ref.tables[:, 2:] >= 0).any()


def test_pages_of_a_pool_ranked_in_several_batches():
    """Pages past two million: ranks go on over the batches in which chunks are ranked."""
    pages, used, size = 2 * (1 << 21) + 9000, 2 * (1 << 21) + 300, 8
    refs, tables = torch.zeros(pages, dtype=torch.int32, device=DEV), torch.full((3, 20), -1, dtype=torch.int32, device=DEV)
    refs[:used] = 1
    ws = torch.empty(C.pages_workspace_size(tables, refs, size), dtype=torch.uint8, device=DEV)
    moves, err = C.new_moves(pages // 2, DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = i32([80, 40, 56])
    C.pages_resize(tables, refs, i32([0, 0, 0]), lens, ws, page_size=size, moves=moves, error_word=err)
    want = np.full((3, 20), -1)
    want[0, :10], want[1, :5], want[2, :7] = used + np.arange(10), used + 10 + np.arange(5), used + 15 + np.arange(7)
    assert tables.cpu().numpy().tolist() == want.tolist() and int(refs.sum()) == used + 22
    holes = [5, 1 << 20, (1 << 21) + 7]                    # in both batches; the last three pages in use fill them
    refs[i32(holes).long()] = 0
    C.pages_compact(tables, refs, lens, ws, page_size=size, moves=moves, error_word=err)
    assert int(moves.count.item()) == 3 and moves.dst[:3].tolist() == holes
    assert moves.src[:3].tolist() == [used + 19, used + 20, used + 21]
    want[2, 4:7] = holes
    assert tables.cpu().numpy().tolist() == want.tolist() and int(err.item()) == 0
    assert int(refs[:used + 19].min()) == 1 and int(refs[used + 19:].max()) == 0


def test_pages_state_errors_are_flagged():
    b = Both(4, 3, 8, 10, lens=[9, 8, 0, 0])
    out = torch.empty(4, dtype=torch.int32, device=DEV)
    C.pages_fork(b.tables, b.refs, i32(b.lens), i32([-1, 0, 9, 1]), out, page_size=8, error_word=b.err)
    assert out.tolist() == [9, 8, 0, 8]                    # a child that holds pages, a parent that is none
    b.ref.fork(b.lens, np.array([-1, -1, -1, 1]))
    b.compare(None, B.DEVERR_PAGE_STATE)
    b.lens = np.array([9, 8, 0, 8], dtype=np.int32)
    # a length past the table counts as its whole
    C.pages_resize(b.tables, b.refs, i32(b.lens), i32([9, 8, 1000, 8]), b.ws, page_size=8, moves=b.moves, error_word=b.err)
    b.ref.resize(b.lens, np.array([9, 8, 24, 8]))
    b.compare([], B.DEVERR_PAGE_STATE)
    # a page counted 0 is not counted below, an entry outside the pool dropped without one
    refs, tables = b.refs.clone(), b.tables.clone()
    refs[int(tables[0, 0])] = 0
    tables[1, 0] = 77
    C.pages_resize(tables, refs, i32([9, 8, 24, 8]), i32([0, 0, 24, 8]), b.ws, page_size=8, moves=b.moves, error_word=b.err)
    torch.cuda.synchronize()
    assert int(b.err.item()) == B.DEVERR_PAGE_STATE and int(refs.min()) >= 0
    assert tables[0].tolist() == [-1] * 3 and tables[1].tolist() == [-1] * 3


def test_pages_without_requests_leave_no_moves():
    """A copy behind a call of no requests finds no moves, whatever the call before left."""
    moves = C.PageMoves(i32([0] * 8), i32([1] * 8), i32([5]))
    none = torch.empty(0, 4, dtype=torch.int32, device=DEV)
    refs, ws = i32([1] * 16), torch.empty(4096, dtype=torch.uint8, device=DEV)
    C.pages_resize(none, refs, i32([]), i32([]), ws, page_size=8, moves=moves)
    assert int(moves.count.item()) == 0
    moves.count.fill_(5)
    C.pages_compact(none, refs, i32([]), ws, page_size=8, moves=moves)
    assert int(moves.count.item()) == 0 and refs.tolist() == [1] * 16


def test_pages_of_lengths_near_the_end_of_32_bits():
    size = (1 << 30) + 1                                   # one page more than half of what a length can count
    tables, refs = i32([[-1], [-1]]), i32([0, 0, 0])
    ws = torch.empty(C.pages_workspace_size(tables, refs, size), dtype=torch.uint8, device=DEV)
    moves, err = C.new_moves(2, DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    C.pages_resize(tables, refs, i32([0, 0]), i32([size, size - 1]), ws, page_size=size, moves=moves, error_word=err)
    assert tables.tolist() == [[0], [1]] and refs.tolist() == [1, 1, 0] and int(err.item()) == 0
    C.pages_resize(tables, refs, i32([size, size - 1]), i32([0, size]), ws, page_size=size, moves=moves, error_word=err)
    assert tables.tolist() == [[-1], [1]] and refs.tolist() == [0, 1, 0] and int(err.item()) == 0


def test_pages_replay_from_a_graph_and_share_a_workspace():
    """Two captured calls on one workspace, replayed in turn, on the lengths of that moment."""
    b = Both(20, 30, 8, 400)
    old, new = i32(np.zeros(20)), i32(np.zeros(20))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.stream(side):
        with torch.cuda.graph(graphs[0], stream=side):
            C.pages_resize(b.tables, b.refs, old, new, b.ws, page_size=8, moves=b.moves, error_word=b.err)
        with torch.cuda.graph(graphs[1], stream=side):
            C.pages_compact(b.tables, b.refs, new, b.ws, page_size=8, moves=b.moves, error_word=b.err)
    torch.cuda.synchronize()
    rng = np.random.default_rng(3)
    for _ in range(6):
        lens = np.where(rng.random(20) < 0.4, 0, rng.integers(0, 150, size=20)).astype(np.int32)
        old.copy_(i32(b.lens))
        new.copy_(i32(lens))
        moves, _ = b.ref.resize(b.lens, lens)
        graphs[0].replay()
        b.compare(moves)
        b.lens = lens
        moves = b.ref.compact(lens)
        graphs[1].replay()
        b.compare(moves)


@pytest.mark.parametrize("shape,dtype", [((33,), torch.uint8), ((3,), torch.float32), ((5,), torch.int16), ((16, 64), torch.uint8),
                                         ((7, 513), torch.bfloat16), ((70000,), torch.uint8)])
@pytest.mark.parametrize("count", [0, 1, 37])
def test_pages_copy(shape, dtype, count):
    """Pages of 1 byte to 70 KB, aligned to 16, 4, 2 and 1 byte, more pools than one launch takes, padded pools."""
    rng = np.random.default_rng(count)
    n = 100
    one = torch.from_numpy(rng.integers(0, 100, size=(n, *shape)).astype(np.int64)).to(dtype).to(DEV)
    wide = torch.zeros((n, 2, *shape), dtype=dtype, device=DEV)
    wide[:, 0] = one
    pools = [one.clone() for _ in range(70)] + [wide[:, 0]]
    src, dst = rng.permutation(50)[:count] + 50, rng.permutation(50)[:count]
    moves = C.new_moves(40, DEV)
    moves.src[:count], moves.dst[:count], moves.count[0] = i32(src), i32(dst), count
    want = one.clone()
    want[torch.from_numpy(dst).to(DEV)] = one[torch.from_numpy(src).to(DEV)]
    C.pages_copy(pools, moves)
    torch.cuda.synchronize()
    assert all(torch.equal(p, want) for p in pools) and bool((wide[:, 1] == 0).all())


def test_pages_copy_flags_what_is_no_page():
    pool = torch.arange(80, dtype=torch.float32, device=DEV).view(10, 8)
    moves = C.new_moves(4, DEV)
    moves.src.copy_(i32([1, 10, -1, 3]))
    moves.dst.copy_(i32([0, 2, 4, 99]))
    moves.count[0] = 77                                    # more than there is room for: the room counts
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = pool.clone()
    want[0] = pool[1]
    C.pages_copy([pool], moves, error_word=err)
    torch.cuda.synchronize()
    assert torch.equal(pool, want) and int(err.item()) == B.DEVERR_PAGE_STATE


# ---------------------------------------------------------------- together

def test_serving_loop():
    """Prompts, decode steps, a fork, ends and a compaction over two layers: after
    each step the attention is that of the codes that the calls themselves left,
    and those are within a rounding of the rows that were appended."""
    rng = np.random.default_rng(50)
    rows, max_pages, page_size, block, pages, layers = 6, 6, 32, 8, 30, 2
    b = Both(rows, max_pages, page_size, pages)
    pool = [torch.full((pages, page_size, 512), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(layers)]
    scales = [torch.full((pages, page_size // block), float("nan"), device=DEV) for _ in range(layers)]
    history = [[np.zeros((0, 512)) for _ in range(rows)] for _ in range(layers)]

    def step(new):
        """New tokens for the requests that grow: pages, copies, rows, then attention of the new tokens."""
        old, new = b.lens.copy(), np.asarray(new, dtype=np.int32)
        b.resize(new)
        C.pages_copy(pool + scales, b.moves)
        q_lens = np.maximum(new - old, 0)
        cum = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        for l in range(layers):
            x, xv = bf16(rng.normal(size=(int(cum[-1]), 512)) * 2.0 ** rng.integers(-2, 3, size=(int(cum[-1]), 1)))
            err = torch.zeros(1, dtype=torch.int32, device=DEV)
            C.append(x, pool[l], scales[l], b.tables, i32(new), cum_seq_lens_q=i32(cum), error_word=err)
            for r in range(rows):
                history[l][r] = np.concatenate([history[l][r][:new[r]], xv[cum[r]:cum[r + 1]]])
            q = rng.normal(size=(int(cum[-1]), 64, 512))
            cache = R.Cache(pool[l].cpu().numpy(), scales[l].cpu().numpy(), b.tables.cpu().numpy(), new, cum=cum)
            assert int(err.item()) == 0
            g = dict(rows=pool[l], scales=scales[l], block_tables=b.tables, seq_lens=i32(new))
            check(cache, q, run(cache, q, window=50, first=3, g=g), window=50, first=3)
            for r in range(rows):
                for j in range(int(new[r])):
                    # one rounding of half E4M3's step, and one for each of the two scales that may follow: 3 * 2^-4,
                    # or half its subnormal step of the block's scale
                    s = cache.scales[cache.page(r, j), j % page_size // block]
                    assert np.all(np.abs(cache.row(r, j) - history[l][r][j]) <= 3 * 2.0 ** -4 * np.abs(history[l][r][j])
                                  + 3 * 2.0 ** -10 * s)

    step([40, 7, 0, 64, 0, 0])
    for _ in range(3):
        step(b.lens + (b.lens > 0))
    b.fork(np.array([-1, -1, 0, -1, 0, 3]))
    for l in range(layers):
        for child, parent in ((2, 0), (4, 0), (5, 3)):
            history[l][child] = history[l][parent].copy()
    for _ in range(2):
        step(b.lens + (b.lens > 0))
    step(np.where(np.arange(rows) % 2 == 0, b.lens + 5, 0))  # three end, three speculate
    step(b.lens - 3 * (b.lens > 0))                          # ... and roll back
    b.compact()
    C.pages_copy(pool + scales, b.moves)
    step(b.lens + (b.lens > 0))


def test_calls_on_another_stream_and_device_index():
    """A call takes the stream it is given, and its tensors' device whichever is current."""
    cache, q, _ = make(60, [300], [1])
    g, qt = on_gpu(cache), bf16(q)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(qt), torch.empty(qt.shape[:2], device=DEV)
    ws = workspace(qt, g, window=256)
    torch.cuda.synchronize()
    C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], ws, window=256, out=out, out_lse=lse,
                       bmm1_scale=1 / math.sqrt(512), stream=side.cuda_stream)
    side.synchronize()
    check(cache, q, (out.to(torch.float64).cpu().numpy(), lse.to(torch.float64).cpu().numpy()), window=256)


class NoExtension:
    """Answers every call with None: the Python functions do all of it."""
    def __getattr__(self, name):
        return lambda *args: None


def all_calls():
    """Results of every call once, on one state."""
    cache, q, rng = make(50, [700, 40, 300], [2, 1, 3], heads=80)
    g, cum = on_gpu(cache), i32([0, 2, 3, 6])
    qt, x = bf16(q)[0], bf16(rng.normal(size=(6, 512)))[0]
    ws = workspace(qt, g, window=500, cum_seq_lens_q=cum)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sinks, two = torch.linspace(-2, 2, 80, device=DEV), torch.tensor([2.0], device=DEV)
    C.append(x, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], cum_seq_lens_q=cum, error_word=err)
    o, l = C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], ws, window=500, first_tokens=3,
                              cum_seq_lens_q=cum, sinks=sinks, bmm1_scale=0.05, bmm2_scale=two, error_word=err)
    o2, l2 = torch.empty_like(o), torch.empty_like(l)
    assert C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], ws, window=500, first_tokens=3,
                              cum_seq_lens_q=cum, sinks=sinks, bmm1_scale=0.05, bmm2_scale=two, out=o2, out_lse=l2,
                              num_splits=2, stream=torch.cuda.current_stream().cuda_stream) == (o2, l2)
    tables, refs = torch.full((4, 6), -1, dtype=torch.int32, device=DEV), torch.zeros(20, dtype=torch.int32, device=DEV)
    pws, moves = torch.empty(C.pages_workspace_size(tables, refs, 16), dtype=torch.uint8, device=DEV), C.new_moves(10, DEV)
    C.pages_resize(tables, refs, i32([0] * 4), i32([40, 20, 0, 0]), pws, page_size=16, moves=moves, error_word=err)
    lens = torch.empty(4, dtype=torch.int32, device=DEV)
    C.pages_fork(tables, refs, i32([40, 20, 0, 0]), i32([-1, -1, 0, 0]), lens, page_size=16, error_word=err)
    C.pages_resize(tables, refs, lens.clone(), i32([0, 21, 41, 41]), pws, page_size=16, moves=moves, error_word=err)
    pool = torch.arange(20 * 6, device=DEV).view(20, 2, 3).clone()
    C.pages_copy([pool], moves, error_word=err)
    kept = [m.clone() for m in moves]
    C.pages_compact(tables, refs, i32([0, 21, 41, 41]), pws, page_size=16, moves=moves, error_word=err)
    C.pages_copy((pool, pool.new_zeros(20, 1)), moves, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return [g["rows"], g["scales"], o, l, o2, l2, tables, refs, lens, pool, moves.count] + kept


def test_both_ways_into_the_library(monkeypatch):
    """Plain tensors take the extension all the way; without it the Python functions give the same."""
    C.extension()
    with monkeypatch.context() as m:
        for name in ("_window_args", "_cache", "_pages_args", "_call"):
            m.setattr(C, name, lambda *a, **k: pytest.fail("not through the extension"))
        m.setattr(C, "window_workspace_size", lambda *a, **k: 1 << 24)
        m.setattr(C, "pages_workspace_size", lambda *a, **k: 1 << 16)
        fast = all_calls()
    monkeypatch.setattr(C, "_extension", NoExtension())
    for a, b in zip(fast, all_calls()):
        a, b = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (a, b))
        assert torch.equal(a.nan_to_num() if a.is_floating_point() else a, b.nan_to_num() if b.is_floating_point() else b)


def test_refusals_through_the_extension():
    cache, q, _ = make(51, [100], [1])
    g, qt = on_gpu(cache), bf16(q)[0]
    call = lambda **k: C.window_attention(**{**dict(q=qt, workspace_buffer=None, window=4, **g), **k})
    for over, exc, match in ((dict(window=0), B.SmlaError, "window"), (dict(window=1 << 40), ValueError, "32-bit"),
                             (dict(num_splits=2), B.SmlaError, "workspace"), (dict(q=qt.float()), TypeError, "bfloat16"),
                             (dict(seq_lens=g["seq_lens"].long()), TypeError, "int32"),
                             (dict(seq_lens=g["seq_lens"].cpu()), ValueError, "CUDA device"),
                             (dict(out=torch.empty(1, 64, 511, dtype=torch.bfloat16, device=DEV)), ValueError, "out must"),
                             (dict(bmm1_scale=torch.ones(1, dtype=torch.float64, device=DEV)), TypeError, "float32")):
        with pytest.raises(exc, match=match):
            call(**over)
    out, _ = call(bmm1_scale=1, bmm2_scale=True)            # numbers of other kinds
    assert torch.isfinite(out.float()).all()


def chain(sync, steps=40, layers=2):
    """A run of every call, one behind another without a host wait between (or with one): all it leaves."""
    rng = np.random.default_rng(60)
    rows, pages, size = 24, 200, 16
    tables = torch.full((rows, 40), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    pool = [torch.zeros(pages, size, 512, dtype=torch.uint8, device=DEV) for _ in range(layers)]
    scales = [torch.zeros(pages, size // 8, device=DEV) for _ in range(layers)]
    ws = torch.empty(C.pages_workspace_size(tables, refs, size), dtype=torch.uint8, device=DEV)
    wws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    moves, err = C.new_moves(pages, DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    latent = bf16(rng.normal(size=(steps, rows, 512)) * 2.0 ** rng.integers(-3, 4, size=(steps, rows, 1)))[0]
    q = bf16(rng.normal(size=(steps, rows, 64, 512)))[0]
    plan, lens = [], np.zeros(rows, dtype=np.int32)
    for s in range(steps):                                 # ends, forks and growth by one token, all known beforehand
        keep = np.where(rng.random(rows) < 0.1, 0, lens)
        parents = np.full(rows, -1, dtype=np.int32)
        alive = np.flatnonzero(keep > 0)
        for b in np.flatnonzero(keep == 0):
            if len(alive) and rng.random() < 0.5:
                parents[b] = rng.choice(alive)
        forked = np.where(parents >= 0, keep[np.maximum(parents, 0)], keep)
        plan.append([i32(a) for a in (lens, keep, parents, forked + 1)])
        lens = (forked + 1).astype(np.int32)
    after, outs = torch.empty(rows, dtype=torch.int32, device=DEV), []
    pause = torch.cuda.synchronize if sync else (lambda: None)
    torch.cuda.synchronize()
    for s, (old, keep, parents, new) in enumerate(plan):
        C.pages_resize(tables, refs, old, keep, ws, page_size=size, moves=moves, error_word=err), pause()
        C.pages_fork(tables, refs, keep, parents, after, page_size=size, error_word=err), pause()
        C.pages_resize(tables, refs, after, new, ws, page_size=size, moves=moves, error_word=err), pause()
        C.pages_copy(pool + scales, moves, error_word=err), pause()
        for k in range(layers):
            C.append(latent[s], pool[k], scales[k], tables, new, error_word=err), pause()
            outs.append(C.window_attention(q[s], pool[k], scales[k], tables, new, wws, window=24, first_tokens=3,
                                           num_splits=s % 3, bmm1_scale=0.04, error_word=err)), pause()
        if s % 7 == 6:
            C.pages_compact(tables, refs, new, ws, page_size=size, moves=moves, error_word=err), pause()
            C.pages_copy(pool + scales, moves, error_word=err), pause()
    torch.cuda.synchronize()
    return [tables, refs, *pool, *scales, err] + [t for pair in outs for t in pair]


def test_calls_behind_one_another_are_calls_one_by_one():
    """Kernels start while the ones before them end; none may see less than all of what those wrote."""
    one_by_one = chain(True)
    assert int(one_by_one[6].item()) == 0
    for _ in range(3):
        for a, b in zip(one_by_one, chain(False)):
            assert torch.equal(a, b)


def test_captured_behind_two_streams():
    """Calls captured behind work of two streams, and before work of both."""
    cache, _, rng = make(61, [90, 200, 33], [1, 1, 1])
    g, start = on_gpu(cache), torch.cuda.Stream()
    x, q = bf16(rng.normal(size=(3, 512)))[0], bf16(rng.normal(size=(3, 64, 512)))[0]
    latent, query, out, lse = torch.zeros_like(x), torch.zeros_like(q), torch.empty_like(q), torch.empty(3, 64, device=DEV)
    lens, ws = torch.zeros_like(g["seq_lens"]), torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    sums = torch.zeros(2, device=DEV)
    other = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=start):
        other.wait_stream(start)
        with torch.cuda.stream(other):
            query.copy_(q * 1.0)
            torch.add(g["seq_lens"], 0, out=lens)
        torch.mul(x, 1.0, out=latent)
        start.wait_stream(other)
        C.append(latent, g["rows"], g["scales"], g["block_tables"], lens)
        C.window_attention(query, g["rows"], g["scales"], g["block_tables"], lens, ws, window=64, num_splits=2, out=out, out_lse=lse)
        other.wait_stream(start)
        with torch.cuda.stream(other):
            sums[0] = out.float().sum()
        sums[1] = lse.sum()
        start.wait_stream(other)
    plain = on_gpu(cache)
    for turn in range(4):
        x.copy_(bf16(rng.normal(size=(3, 512)) * 2.0 ** turn)[0])
        q.copy_(bf16(rng.normal(size=(3, 64, 512)))[0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        C.append(x, plain["rows"], plain["scales"], plain["block_tables"], plain["seq_lens"])
        o, l = C.window_attention(q, plain["rows"], plain["scales"], plain["block_tables"], plain["seq_lens"], ws, window=64,
                                  num_splits=2)
        torch.cuda.synchronize()
        assert torch.equal(plain["rows"], g["rows"]) and torch.equal(o, out) and torch.equal(l, lse)
        assert torch.allclose(sums, torch.stack([o.float().sum(), l.sum()]), rtol=1e-3, atol=1e-2)


def test_pages_past_four_gigabytes():
    """Pages behind 2^32 bytes give what the same pages give in a small pool."""
    cache, q, rng = make(62, [300, 120], [3, 70], junk=False)
    small, cum = on_gpu(cache), i32(cache.cum)
    n, used = 140_000, cache.rows.shape[0]                 # 4.6 GB of rows
    shift = n - used
    big = dict(small, rows=torch.empty(n, 64, 512, dtype=torch.uint8, device=DEV), scales=torch.zeros(n, 4, device=DEV),
               block_tables=torch.where(small["block_tables"] >= 0, small["block_tables"] + shift, -1).to(torch.int32))
    big["rows"][shift:], big["scales"][shift:] = small["rows"], small["scales"]
    qt, x = bf16(q)[0], bf16(rng.normal(size=(73, 512)))[0]
    got = []
    for g in (small, big):
        C.append(x, g["rows"], g["scales"], g["block_tables"], g["seq_lens"], cum_seq_lens_q=cum)
        for splits in (1, 2):
            got.append(C.window_attention(qt, g["rows"], g["scales"], g["block_tables"], g["seq_lens"],
                                          workspace(qt, g, window=200, num_splits=splits, cum_seq_lens_q=cum), window=200,
                                          cum_seq_lens_q=cum, num_splits=splits, bmm1_scale=0.04))
    assert torch.equal(small["rows"], big["rows"][shift:]) and torch.equal(small["scales"], big["scales"][shift:])
    for (a, b), (c, d) in zip(got[:2], got[2:]):
        assert torch.equal(a, c) and torch.equal(b, d)
    moves = C.PageMoves(i32([n - 1, 1]), i32([0, n - 2]), i32([2]))
    big["rows"][1] = 7
    C.pages_copy([big["rows"], big["scales"]], moves)
    assert torch.equal(big["rows"][0], big["rows"][n - 1]) and bool((big["rows"][n - 2] == 7).all())


@pytest.mark.parametrize("T,window,first,splits", [(1, 1 << 30, 0, 0), (3, 1 << 30, 0, 0), (3, 1 << 30, 0, 1),
                                                   (3, 131072, 70000, 0), (3, 1, 250000, 64)])
def test_window_over_a_long_sequence(T, window, first, splits):
    """A quarter of a million rows, against 64 bits on the GPU."""
    n, H, size = 262_144 + 5, 64, 256
    gen = torch.Generator(DEV).manual_seed(63)
    pages = -(-n // size)
    rows = torch.randn(pages, size, 512, device=DEV, generator=gen).to(torch.float8_e4m3fn)
    scales = torch.exp2(torch.randint(-3, 1, (pages, size // 32), device=DEV, generator=gen).float())
    tables = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32).view(1, -1)
    q = torch.randn(T, H, 512, device=DEV, generator=gen).to(torch.bfloat16)
    g = dict(rows=rows, scales=scales, block_tables=tables, seq_lens=i32([n]))
    bmm1 = 0.05
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = C.window_attention(q, *g.values(), workspace(q, g, window=window, first_tokens=first, num_splits=splits),
                                  window=window, first_tokens=first, num_splits=splits, bmm1_scale=bmm1, error_word=err)
    order = tables[0].long()
    kv = (rows[order].double() * scales[order].double().repeat_interleave(32, 1)[..., None]).view(-1, 512)[:n]
    j = torch.arange(n, device=DEV)
    assert int(err.item()) == 0
    for t in range(T):
        pos = n - T + t
        seen = kv[(j <= pos) & ((j > pos - window) | (j < first))]
        x = q[t].double()
        l = x @ seen.T * bmm1
        # the logits' bound of the reference: fp32 sums, and the query's split
        off = (2.0 ** -18 * (x.abs() @ seen.abs().T) + 2.0 ** -17 * x.abs().amax(1, keepdim=True) * seen.abs().sum(1)) * bmm1
        p = torch.softmax(l, 1)
        want, want_lse = p @ seen, torch.logsumexp(l, 1) / math.log(2.0)
        # (sums of a thread's rows: 2049 tiles at most, 2^-24 each; a merge of 152)
        tol = 1.4427 * ((p * 2 * off).sum(1) + 2.0 ** -18 + 2201 * 2.0 ** -24) + 2.0 ** -21 * want_lse.abs()
        assert bool(((lse[t].double() - want_lse).abs() <= tol).all())
        # rounding errors of either sign: P's 2^-8 over the weights, the result's 2^-9
        spread = ((p ** 2) @ (seen ** 2)).sqrt()
        assert ((out[t].double() - want) ** 2).mean().sqrt() <= 2.0 ** -8 * (spread.square().mean() + want.square().mean()).sqrt()
