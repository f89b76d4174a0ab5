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


def test_window_workspace_is_sized_for_the_device_of_the_queries(lib, monkeypatch):
    """The call plans for q's device, which need not be device 0."""
    asked = []

    class Library:
        def smla_window_workspace_size(self, args, device, bytes_out):
            asked.append(device)
            return 0

    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 3

    monkeypatch.setattr(C._b, "lib", lambda: Library())
    kw = host_tensors()
    kw.pop("workspace_buffer")
    C.window_workspace_size(**kw)
    kw["q"] = kw["q"].as_subclass(Elsewhere)
    C.window_workspace_size(**kw)
    C.window_workspace_size(**kw, device=1)
    assert asked == [0, 3, 1]
