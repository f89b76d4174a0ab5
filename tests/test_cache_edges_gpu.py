"""The paged latent cache on the GPU where its calls are easiest to get wrong:
batches padded in front, and the memory around a call's own tensors."""
import numpy as np
import pytest
import torch

import cache_reference as R
from sparse_mla_decode_token_gb300 import cache as C
from test_cache_gpu import DEV, bf16, built, i32, make, on_gpu  # noqa: F401  (built: the library, once a module)

pytestmark = pytest.mark.gpu


def guarded(a, value):
    """A tensor like the array `a` inside a larger one filled with `value`: (view, whole)."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    whole = torch.full((3 * t.numel(),), value, dtype=t.dtype, device=DEV)
    view = whole[t.numel():2 * t.numel()].view(t.shape)
    view.copy_(t)
    return view, whole


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("lead", [1, 15, 16, 17, 200])
@pytest.mark.parametrize("page_size,block", [(64, 16), (16, 1), (64, 64)])
@pytest.mark.parametrize("lens,q_lens", [([1], [1]), ([40, 70], [3, 2]), ([130], [2]), ([5, 20, 64], [5, 0, 64])])
def test_append_batch_padded_in_front(lead, page_size, block, lens, q_lens):
    """Rows before the first offset are no request's: nothing is written for them, whatever the scales (also 0 and
    NaN) of the blocks that the first request holds, and nothing before or behind the cache's own memory."""
    cache, _, rng = make(60, lens, q_lens, page_size=page_size, block=block)
    if int(lens[0]) < page_size:                           # the first request's first page is page 0, where it can be
        own, other = int(cache.tables[0, 0]), 0
        for a in (cache.rows, cache.scales):
            a[[own, other]] = a[[other, own]]
        swap = {own: other, other: own}
        cache.tables = np.vectorize(lambda p: swap.get(int(p), int(p)))(cache.tables).astype(np.int32)
    start = int(lens[0]) - q_lens[0]
    for k, j in enumerate(range(0, start // block * block, block)):    # older blocks, none of which is written
        cache.scales[cache.page(0, j), j % page_size // block] = (0.0, np.nan, np.inf)[k % 3]
    x = rng.normal(size=(lead + sum(q_lens), 512))
    x[:lead] = 1e4                                         # (would raise any scale that it reached)
    rows, rows_all = guarded(cache.rows, 0x55)
    scales, scales_all = guarded(cache.scales, 0.0)
    tables, _ = guarded(cache.tables, 0)                   # (pages in front of the tables exist)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    C.append(bf16(x)[0], rows, scales, tables, i32(lens), cum_seq_lens_q=i32(cache.cum + lead), error_word=err)
    torch.cuda.synchronize()
    R.append(cache, bf16(x)[0][lead:].float().cpu().numpy())
    assert int(err.item()) == 0
    assert np.array_equal(rows.cpu().numpy(), cache.rows)
    assert np.array_equal(scales.cpu().numpy(), cache.scales, equal_nan=True)
    for whole, value, n in ((rows_all, 0x55, rows.numel()), (scales_all, 0.0, scales.numel())):
        assert bool((whole[:n] == value).all()) and bool((whole[2 * n:] == value).all())


# ---------------------------------------------------------------- refusals

def test_broadcast_tensors_never_reach_the_library():
    """Both ways into the library, the extension's and Python's, refuse tokens that share memory."""
    cache, q, rng = make(61, [40, 30], [2, 2])
    g = on_gpu(cache)
    q1, x1 = bf16(q[:1])[0], bf16(rng.normal(size=(1, 512)))[0]
    with pytest.raises(ValueError, match="share memory"):
        C.window_attention(q1.expand(4, -1, -1), g["rows"], g["scales"], g["block_tables"], g["seq_lens"], None, window=16)
    with pytest.raises(ValueError, match="share memory"):
        C.append(x1.expand(4, -1), g["rows"], g["scales"], g["block_tables"], g["seq_lens"])


# --------------------------------------------------------------- attention

def test_window_query_elements_beside_large_ones():
    """Heads with a few dims of 2^0 to 2^12 times the others, where the rows hold nothing: the logits are the other
    dims' alone.  An element is off by at most 2^-22 of its head's largest one; as evenly spread errors of 448 dims
    that is 0.0013 of a logit's deviation here (0.0022 in natural units) at 2^12, under the result's own 2^-8."""
    rng = np.random.default_rng(62)
    n, heads, scale, bmm1 = 500, 64, 2.0 ** -6, 512 ** -0.5
    codes = rng.normal(size=(8 * 64, 512)) * 85
    codes[:, ::8] = 0
    rows = R.to_e4m3(codes)
    q = rng.normal(size=(1, heads, 512))
    power = np.arange(heads) % 13
    q[0, :, ::8] *= 2.0 ** power[:, None]
    g = dict(rows=torch.from_numpy(rows.reshape(8, 64, 512)).to(DEV), scales=torch.full((8, 4), scale, device=DEV),
             block_tables=i32(np.arange(8)[None]), seq_lens=i32([n]))
    qt, qv = bf16(q)
    kv = R.e4m3(rows)[:n] * scale
    logits = qv[0] @ kv.T * bmm1
    top = logits.max(axis=1, keepdims=True)
    p = np.exp(logits - top)
    want, lse = p @ kv / p.sum(axis=1, keepdims=True), (top[:, 0] + np.log(p.sum(axis=1))) / np.log(2)
    for splits in (1, 2):
        ws = torch.empty(C.window_workspace_size(qt, *g.values(), window=n, num_splits=splits) + 256, dtype=torch.uint8,
                         device=DEV)
        out, got = C.window_attention(qt, *g.values(), ws, window=n, num_splits=splits, bmm1_scale=bmm1)
        err = np.sqrt(((out[0].double().cpu().numpy() - want) ** 2).mean(axis=1) / (want ** 2).mean(axis=1))
        assert err.max() <= 2.0 ** -8, err.round(5).tolist()
        # every logit off by its worst case, and 2^-18 of the products' sum for the fp32 additions
        off = bmm1 * (2.0 ** -22 * np.abs(qv[0]).max(axis=1) * np.abs(kv).sum(axis=1).max()
                      + 2.0 ** -18 * (np.abs(qv[0]) @ np.abs(kv).T).max(axis=1))
        assert np.all(np.abs(got[0].double().cpu().numpy() - lse) <= 1.4427 * off + 2.0 ** -16)


@pytest.mark.parametrize("splits", [1, 0, 2])
@pytest.mark.parametrize("empty", [1, 200, 500])
def test_window_units_without_rows_in_front(empty, splits):
    """A CTA's first units see nothing (positions below 0, tokens before the first offset), later ones do: the first
    products' queries stay in step with their units."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tail = 40
    cache, q, rng = make(63, [empty, 300 + tail], [2 * empty, tail])      # the first request's first half lies below 0
    lead = sms - 1                                                       # and tokens of no request before it
    q_all = np.concatenate([rng.normal(size=(lead, 64, 512)), q])
    cum = i32(cache.cum + lead)
    g, qt = on_gpu(cache), bf16(q_all)[0]
    size = C.window_workspace_size(qt, *g.values(), window=200, first_tokens=2, cum_seq_lens_q=cum, num_splits=splits)
    for _ in range(3):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device=DEV)
        out, lse = torch.full_like(qt, 7.0), torch.full(qt.shape[:2], 7.0, device=DEV)
        C.window_attention(qt, *g.values(), ws, window=200, first_tokens=2, cum_seq_lens_q=cum, num_splits=splits,
                           bmm1_scale=512 ** -0.5, out=out, out_lse=lse, error_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert bool((out[:lead] == 7).all()) and bool((lse[:lead] == 7).all())
        own = out[lead:].double().cpu().numpy(), lse[lead:].double().cpu().numpy()
        assert np.all(own[0][:empty] == 0) and np.all(np.isneginf(own[1][:empty]))
        # the last request's tokens, and those of the first that see something: a sample of both
        for t in [empty, 2 * empty - 1] + list(range(2 * empty, 2 * empty + tail, 9)):
            b, i = (0, t - 2 * empty) if t < 2 * empty else (1, t - 2 * empty - tail)
            part = R.Cache(cache.rows, cache.scales, cache.tables[b:b + 1], cache.lens[b:b + 1] + i + 1, tokens=1)
            want, wlse, tol_o, tol_l = R.window(part, bf16(q[t:t + 1])[1], window=200, first=2, bmm1=512 ** -0.5)
            assert np.all(np.abs(own[0][t] - want[0]) <= tol_o[0]) and np.all(np.abs(own[1][t] - wlse[0]) <= tol_l[0])


# ----------------------------------------------------------------- streams

def test_outputs_belong_to_the_stream_of_the_call():
    """Outputs that a call allocates are written on the stream that it was given: memory of the current stream, free
    there but not behind that stream's work, must not serve."""
    cache, q, _ = make(64, [300, 200], [2, 1], heads=64)
    g, qt, cum = on_gpu(cache), bf16(q)[0], i32(cache.cum)
    ws = torch.empty(C.window_workspace_size(qt, *g.values(), window=200, cum_seq_lens_q=cum) + 256, dtype=torch.uint8,
                     device=DEV)
    args = dict(window=200, cum_seq_lens_q=cum, bmm1_scale=512 ** -0.5)
    want, want_lse = C.window_attention(qt, *g.values(), ws, **args)
    side = torch.cuda.Stream()

    def freed(shape, dtype):
        """Addresses of two blocks that the current stream has just given back."""
        a, b = torch.empty(shape, dtype=dtype, device=DEV), torch.empty(shape, dtype=dtype, device=DEV)
        return {a.data_ptr(), b.data_ptr()}
    for k in range(3):
        out_only = torch.empty_like(want) if k == 1 else None
        lse_only = torch.empty_like(want_lse) if k == 2 else None
        torch.cuda.synchronize()
        mine = freed(want.shape, torch.bfloat16) | freed(want_lse.shape, torch.float32)
        out, lse = C.window_attention(qt, *g.values(), ws, stream=side.cuda_stream, out=out_only, out_lse=lse_only, **args)
        torch.cuda.synchronize()
        assert (k == 1 or out.data_ptr() not in mine) and (k == 2 or lse.data_ptr() not in mine)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    # on the current stream, named or not, the current stream's memory does
    here = torch.cuda.current_stream().cuda_stream
    for stream in (None, here):
        mine = freed(want.shape, torch.bfloat16)
        assert C.window_attention(qt, *g.values(), ws, stream=stream, **args)[0].data_ptr() in mine


def test_decode_outputs_belong_to_the_stream_of_the_call():
    from sparse_mla_decode_token_gb300 import binding as B
    T, H = 3, 128
    gen = torch.Generator(device=DEV).manual_seed(1)
    q, kv = (torch.randn(n, 512, generator=gen, device=DEV).to(torch.bfloat16) for n in (T * H, 512))
    idx = torch.randint(0, 512, (T, 256), generator=gen, device=DEV, dtype=torch.int32)
    lens, seq = torch.full((T,), 256, dtype=torch.int32, device=DEV), torch.full((T,), 5000, dtype=torch.int32, device=DEV)
    q = q.view(T, H, 512)
    ws = torch.empty(B.workspace_size(q, idx, seq) + 256, dtype=torch.uint8, device=DEV)
    want, want_lse = B.sparse_mla_decode(q, kv, ws, idx, kv, lens, seq, bmm1_scale=512 ** -0.5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = torch.empty_like(want), torch.empty_like(want_lse)
    mine = {a.data_ptr(), b.data_ptr()}
    del a, b
    out, lse = B.sparse_mla_decode(q, kv, ws, idx, kv, lens, seq, bmm1_scale=512 ** -0.5, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert out.data_ptr() not in mine and lse.data_ptr() not in mine
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
