"""The page list entries that an attention call reads (csrc/pkv_token_plan.h, compiled for
the host): those of the positions that its rows see, and live ones only."""

import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from oracle.tokens import TokenStreamsOracle, visible

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_kv_cache_build_gb300", "csrc")

SHIM = """
#include "pkv_token_plan.h"
using namespace pkv;
extern "C" int entry(int f, int rows, int p0, int p1, int window, int sinks, int page_size) {
  return tok_block_entry(f, rows, p0, p1, window, sinks, page_size);
}
extern "C" int tiles(int p0, int p1, int window, int sinks, int* out) {
  const TokTiles r = tok_tiles(p0, p1, window, sinks);
  for (int j = 0; j < r.n; ++j) out[j] = tok_tile(r, j);
  return r.n;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("blocks")
    src, so = str(d / "shim.cpp"), str(d / "shim.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", so],
                   check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("page,window,sinks", [(16, 1, 0), (16, 20, 3), (16, 5, 70), (32, 40, 33), (64, 64, 1),
                                               (64, 200, 64), (192, 100, 5), (256, 47, 300), (16, 0, 0)])
def test_blocks_come_from_live_pages(plan, page, window, sinks):
    rng = random.Random(page + window)
    ora = TokenStreamsOracle(600, page)
    ora.open(0, 5000, window, sinks)
    out = (ctypes.c_int * 200)()
    for _ in range(40):
        n = rng.choice([1, 2, page, rng.randrange(1, 200)])
        ora.append([0], [n])
        st = ora.streams[0]
        # CTAs of some rows of the call
        for _ in range(5):
            p0 = rng.randrange(st["len"] - n, st["len"])
            p1 = rng.randrange(p0, st["len"])
            # no wider a window than the stream's, and no more sinks
            w = window and rng.randrange(1, window + 1)
            s = rng.choice([0, sinks])
            seen = set()
            for p in (p0, p1):
                seen.update(np.flatnonzero(visible(p, p1 + 1, w, s)).tolist())
            read = set()
            rows = min(page, 64)
            for i in range(plan.tiles(p0, p1, w, s, out)):
                for f in range(out[i] * 64, out[i] * 64 + 64, rows):
                    e = plan.entry(f, rows, p0, p1, w, s, page)
                    assert e in st["pages"], "an evicted page, or one that the stream does not have"
                    if e == f // page:
                        read.update(range(f, f + rows))
            assert seen <= read
        if rng.random() < 0.7:
            ora.evict(0)
