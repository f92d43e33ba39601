"""The shapes that the GPU tests list reach every instance of the attention kernels that is built: tile rule and built kernels
against the lists, host only."""

import json
import os
import re
import subprocess

import pytest

import test_gpu_rows as G
import test_gpu_rows_tiles as T
from layout_permuting_copy_amd import build as B

PROBE = r"""
#include <cstdio>
#include "paged.hpp"
int main() {
  long paged, codes, batch, tokens, heads, group, dim, len;
  while (scanf("%ld %ld %ld %ld %ld %ld %ld %ld", &paged, &codes, &batch, &tokens, &heads, &group, &dim, &len) == 8)
    printf("%ld\n", long(tc::rows_shape(paged, codes, batch, tokens, heads, group, dim, len).tile_rows));
}
"""


def _built():
    """(source of rows: 0 packed, 1 16-bit cache, 2 8-bit cache; padded head_dim; tile) of the kernels in the library."""
    if not os.path.exists(B.RESOURCES):
        pytest.skip("not built here")
    with open(B.RESOURCES) as f:
        names = " ".join(json.load(f))
    found = set()
    for bf16 in "01":
        one = {(int(s), int(d), 32 * int(w)) for s, d, w in re.findall(rf"rows_attention_kernelILb{bf16}ELi(\d)ELi(\d+)ELi(\d)ELi\dELi\dELb0E", names)}
        assert one and (not found or one == found)
        found = one
    return found


def _padded(source, dim):
    return next(d for d in ((64, 96, 128, 192, 256) if source == 0 else (64, 128, 256)) if dim <= d)


def test_listed_shapes_reach_every_instance(tmp_path):
    (tmp_path / "probe.cpp").write_text(PROBE)
    exe = str(tmp_path / "probe")
    subprocess.run(["g++", "-std=c++17", "-I", B.CSRC, "-I", os.path.join(B.ROOT, "include"), str(tmp_path / "probe.cpp"),
                    os.path.join(B.CSRC, "rows_shape.cpp"), "-o", exe], check=True)
    calls = [(0, len(n), sum(n) + 5, heads, group, dim, (sum(n) + 5) // len(n)) for heads, group, dim, n in G.SHAPES]
    calls += [(0, len(n), sum(n) + 3, heads, group, dim, (sum(m or n) + 3) // len(n)) for heads, group, dim, n, m in T.MANY_TILES]
    calls += [(0, 2, 4100, 32, 1, dim, 2050) for dim in (80, 128, 144, 256)]  # test_prompts_in_the_largest_tiles
    for source in (1, 2):
        calls += [(source, len(n), sum(n), heads, group, dim, max(lens)) for heads, group, dim, _, _, lens, n in G.TREES + G.LARGE + T.SMALL]
    lines = "\n".join(f"{int(source > 0)} {int(source == 2)} " + " ".join(map(str, rest)) for source, *rest in calls)
    tiles = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout.split()
    assert len(tiles) == len(calls)
    reached = {(source, _padded(source, dim), int(tile)) for (source, _, _, _, _, dim, _), tile in zip(calls, tiles)}
    assert reached == _built()
    first = len(G.SHAPES)
    assert set(tiles[first:first + len(T.MANY_TILES)]) == {"128"}
    for (source, _, _, _, _, dim, _), tile in list(zip(calls, tiles))[-len(T.SMALL):]:
        assert tile == "64"
