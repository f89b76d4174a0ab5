"""Calls of the paged latent cache that are refused without a GPU: tensors whose
layout would be taken for another one."""
import pytest
import torch

from sparse_mla_decode_token_gb300 import cache as C
from test_cache_host import host_tensors, lib  # noqa: F401  (lib: the library, built once a module)


def test_broadcast_queries_are_refused(lib):
    """A token stride of 0 means the packed one to the library, which would read past the one token's end."""
    one = torch.zeros(1, 64, 512, dtype=torch.bfloat16)
    for call in (C.window_attention, C.window_workspace_size):
        kw = host_tensors(q=one.expand(4, 64, 512))
        if call is C.window_workspace_size:
            kw.pop("workspace_buffer")
        with pytest.raises(ValueError, match="share memory"):
            call(**kw)
    with pytest.raises(ValueError, match="CUDA device"):   # one token has no stride that counts
        C.window_attention(**host_tensors(q=one.as_strided((1, 64, 512), (0, 512, 1)), seq_lens=torch.zeros(1, dtype=torch.int32),
                                          block_tables=torch.zeros(1, 4, dtype=torch.int32)))


def test_broadcast_latents_are_refused(lib):
    t = host_tensors()
    with pytest.raises(ValueError, match="share memory"):
        C.append(torch.zeros(1, 512, dtype=torch.bfloat16).expand(4, 512), t["rows"], t["scales"], t["block_tables"],
                 t["seq_lens"])
