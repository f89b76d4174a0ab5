"""Workspace sizes without a GPU: one workspace serves all calls of at most its call's tokens, requests and table widths
(a server sizes it for its largest step).  The entry points' host sides are compiled with a device of 152 SMs."""
import os
import random
import subprocess

import pytest

from sparse_mla_decode_token_gb300 import build as smla_build

PROGRAM = r"""
#include <cuda_runtime.h>
static cudaError_t attribute(int* value, cudaDeviceAttr, int) { *value = %d; return cudaSuccess; }
#define cudaDeviceGetAttribute attribute
#include "cache_api.cu"
#include "step_api.cu"

// Each line: a call; printed: the size that is asked for, the bytes that this very call needs.
int main() {
  char kind[16];
  while (scanf("%%15s", kind) == 1) {
    size_t size = 0, need = 0;
    int sms = 0;
    device_sms(0, &sms);
    smla_status s = SMLA_OK;
    if (kind[0] == 'b') {
      smla_beam_args a = {};
      scanf("%%d %%d %%d %%d", &a.batch, &a.beams, &a.vocab, &a.dtype);
      a.num_out = 4;
      s = smla_beam_workspace_size(&a, 0, &size);
      need = beam_layout(&a, beam_plan(&a, sms)).bytes;
    } else {
      smla_window_args w = {};
      smla_prefix_args p = {};
      int tokens, heads, pages, page_size, groups, window, splits;
      scanf("%%d %%d %%d %%d %%d %%d %%d", &tokens, &heads, &pages, &page_size, &groups, &window, &splits);
      smla_cache c = {};
      c.num_pages = 1000, c.page_size = page_size, c.block_rows = page_size, c.max_pages = pages, c.batch = 1;
      w.cache = p.cache = c;
      w.sum_q = p.sum_q = tokens;
      w.num_heads = p.num_heads = heads;
      w.window = window, w.num_splits = splits, p.num_groups = groups;
      if (kind[0] == 'w') {
        s = smla_window_workspace_size(&w, 0, &size);
        need = window_plan(&w, sms).bytes;
      } else {
        s = smla_prefix_workspace_size(&p, 0, &size);
        need = shares_prefixes(&p, sms) ? prefix_layout(&p, sms).bytes : grouped_plan(&p, sms).bytes;
      }
    }
    if (s != SMLA_OK) return 1;
    printf("%%zu %%zu\n", size, need);
  }
  return 0;
}
"""


@pytest.fixture(scope="module", params=[152, 148, 7])
def sizes(request, tmp_path_factory):
    """calls -> [(size asked for, bytes needed)] on a device of so many SMs."""
    smla_build.build()
    at = tmp_path_factory.mktemp("sizes")
    (at / "sizes.cu").write_text(PROGRAM % request.param)
    subprocess.run([smla_build.nvcc(), *smla_build.GENCODE, "-std=c++17", "-I", smla_build.CSRC, "-I", smla_build.INCLUDE,
                    str(at / "sizes.cu"), "-o", str(at / "sizes"), "-L", smla_build.BUILD, "-lsmla",
                    "-Xlinker", "-rpath=" + os.path.abspath(smla_build.BUILD)], check=True)

    def ask(calls):
        r = subprocess.run([str(at / "sizes")], input="\n".join(" ".join(map(str, c)) for c in calls), capture_output=True,
                           text=True, check=True)
        return [tuple(map(int, l.split())) for l in r.stdout.splitlines()]
    return ask


def covers(sizes, grow, start, steps):
    """Along `steps` of one field the size never falls, and it is at least what every call so far needs."""
    calls = [grow(start, v) for v in steps]
    most = 0
    last = 0
    for call, (size, need) in zip(calls, sizes(calls)):
        most = max(most, need)
        assert size >= most and size >= last, (call, size, need, most, last)
        last = size


def at(i):
    return lambda call, v: call[:i] + (v,) + call[i + 1:]


TOKENS = sorted({1, 2, 3, *range(4, 400, 7), *range(1500, 3200, 61)})


@pytest.mark.parametrize("kind", ["window", "prefix"])
@pytest.mark.parametrize("heads,pages,window,groups", [
    (64, 256, 1 << 20, 1), (128, 256, 1 << 20, 1), (16, 128, 128, 4), (8, 1024, 4096, 0), (100, 3, 100, 9), (1, 16384, 2048, 2),
])
def test_attention_workspaces_cover_smaller_calls(sizes, kind, heads, pages, window, groups):
    call = (kind, 64, heads, pages, 64, groups, window, 0)
    covers(sizes, at(1), call, TOKENS)
    covers(sizes, at(3), call, range(1, 600, 3))
    for tokens in (1, 4, 77, 153, 1600):
        covers(sizes, at(3), at(1)(call, tokens), [1, 2, 3, 5, 9, 17, 64, 100, 300, 1000, 4096])
        if kind == "window":
            covers(sizes, at(6), at(1)(call, tokens), [1, 64, 128, 129, 500, 1000, 2048, 5000, 40000])
        else:
            covers(sizes, at(5), at(1)(call, tokens), [0, 1, 2, 7, 64, 1000])


def test_forced_splits_cover_fewer_tokens(sizes):
    for splits in (1, 2, 7, 64):
        covers(sizes, at(1), ("window", 1, 128, 64, 64, 0, 2048, splits), TOKENS)


def test_attention_workspaces_cover_calls_that_are_smaller_in_all(sizes):
    rng = random.Random(3)
    for kind in ("window", "prefix"):
        for _ in range(40):
            heads, page_size = rng.choice([1, 8, 16, 33, 64, 96, 128]), rng.choice([8, 16, 64, 256])
            big = (rng.randint(1, 3000), rng.randint(1, 2000), rng.randint(0, 64), rng.randint(1, 20000))
            calls = [big] + [tuple(rng.randint(min(1, v), v) for v in big) for _ in range(40)]
            got = sizes([(kind, t, heads, pages, page_size, groups, window, 0) for t, pages, groups, window in calls])
            assert got[0][0] >= max(need for _, need in got), (kind, heads, page_size, big)


@pytest.mark.parametrize("dtype", [0, 2])
def test_beam_workspaces_cover_smaller_calls(sizes, dtype):
    for beams, vocab in ((8, 128000), (1, 32000), (64, 151001), (4, 500)):
        covers(sizes, at(1), ("beam", 1, beams, vocab, dtype), range(1, 130))
    for batch, vocab in ((1, 128000), (20, 50000), (64, 128000)):
        covers(sizes, at(2), ("beam", batch, 1, vocab, dtype), range(1, 65))
    for batch, beams in ((1, 1), (19, 8), (64, 8)):
        covers(sizes, at(3), ("beam", batch, beams, 1, dtype), [*range(1, 5000, 97), *range(5000, 200000, 2311)])
