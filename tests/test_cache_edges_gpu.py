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
