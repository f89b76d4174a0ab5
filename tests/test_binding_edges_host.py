"""Layouts that the decode's binding refuses because the library would take them
for others (no GPU needed)."""
import pytest
import torch

from sparse_mla_decode_token_gb300 import binding as B

i32 = torch.int32


def decode_tensors(**over):
    t = dict(q=torch.zeros(4, 128, 512, dtype=torch.bfloat16), swa_kv=torch.zeros(64, 512, dtype=torch.bfloat16),
             compressed_kv=torch.zeros(64, 512, dtype=torch.bfloat16), sparse_indices=torch.zeros(4, 256, dtype=i32),
             seq_lens=torch.zeros(4, dtype=i32), out=torch.zeros(4, 128, 512, dtype=torch.bfloat16))
    t.update(over)
    return t


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(1, 128, 512, dtype=torch.bfloat16).expand(4, 128, 512)),
    dict(sparse_indices=torch.zeros(1, 256, dtype=i32).expand(4, 256)),
    dict(sparse_indices=torch.zeros(1, 1, 256, dtype=i32).expand(4, 1, 256)),
    dict(swa_kv=torch.zeros(1, 512, dtype=torch.bfloat16).expand(64, 512)),
    dict(compressed_kv=torch.zeros(1, 512, dtype=torch.bfloat16).expand(64, 512)),
    dict(sparse_indices=torch.zeros(4, 128, dtype=i32), comp_block_tables=torch.zeros(1, 8, dtype=i32).expand(4, 8),
         comp_page_size=16, hca_seq_lens=torch.zeros(4, dtype=i32)),
])
def test_rows_that_share_memory_are_refused(over):
    """A row stride of 0 means the packed one to the library, which would read past the one row's end."""
    with pytest.raises(ValueError, match="share memory"):
        B.make_args(**decode_tensors(**over))
    with pytest.raises(ValueError, match="CUDA device"):   # (the same shapes, each row its own)
        B.make_args(**decode_tensors(**{k: v.contiguous() if isinstance(v, torch.Tensor) else v for k, v in over.items()}))
