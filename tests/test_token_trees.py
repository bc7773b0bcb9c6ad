"""Trees of drafted tokens on the CPU: what the kernels look up of a tree (csrc/pkv_token_plan.h, compiled
for the host) against the oracle's visible sets; the oracle against hand-derived values; the
refusals of the library's own host code, linked with a CUDA runtime that keeps books."""

import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from oracle.tokens import (TokenError, TokenStreamsOracle, causal_attend_fp64, rotate_fp64, tree_attend_fp64,
                           tree_visible, visible)

from .test_token_host import HostStream, cache, handle, lib, rows   # noqa: F401 (fixtures)

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_kv_cache_build_gb300", "csrc")

SHIM = """
#include "pkv_token_plan.h"
using namespace pkv;
extern "C" {
int words() { return kTreeWords; }
int parent(int i, int p) { return tree_parent(i, p); }
int walk(const int16_t* parent, int i, int pos0, int window, int sinks, uint64_t* w) {
  return tree_walk(parent, i, pos0, window, sinks, w);
}
unsigned long long mask(int b, int pos0, int depth, const uint64_t* w, int window, int sinks) {
  return tree_mask(b, pos0, depth, w, window, sinks);
}
int full(int b, int pos0, int n, int window, int sinks) { return tree_tile_full(b, pos0, n, window, sinks); }
int needs(int t, int pos0, int n, int window, int sinks) { return tree_span(pos0, n, window, sinks).needs(t); }
int whole(int t, int pos0, int n, int window, int sinks) { return tree_span(pos0, n, window, sinks).whole(t); }
int tiles(int pos0, int n, int window, int sinks, int* out) {
  const TokTiles r = tok_tiles(pos0, pos0 + n - 1, window, sinks);
  for (int j = 0; j < r.n; ++j) out[j] = tok_tile(r, j);
  return r.n;
}
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("trees")
    src, so = str(d / "shim.cpp"), str(d / "shim.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", so],
                   check=True)
    L = ctypes.CDLL(so)
    L.mask.restype = ctypes.c_ulonglong
    return L


def tree(rng, n):
    return [rng.randrange(-1, i) if rng.random() < 0.6 else i - 1 for i in range(n)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (2, 4), (5, 300), (63, 1), (64, 64), (100, 65), (2 ** 31 - 1, 7),
                                          (3, 2 ** 31 - 1)])
def test_masks_are_the_visible_sets(plan, window, sinks):
    rng = random.Random(window + sinks)
    for before, n in ((0, 1), (0, 256), (1, 200), (63, 256), (64, 5), (127, 130), (200, 63), (500, 256), (129, 7)):
        parents = tree(rng, n)
        seen = tree_visible(parents, before, window, sinks)
        c_parents = (ctypes.c_int16 * n)(*parents)
        out = (ctypes.c_int * 40)()
        tiles = list(out[:plan.tiles(before, n, window, sinks, out)])
        assert len(set(tiles)) == len(tiles)
        for t in range(-(-(before + n) // 64)):
            some = seen[:, t * 64:t * 64 + 64]
            if some.any():
                assert t in tiles and plan.needs(t, before, n, window, sinks)
            whole = some.shape[1] == 64 and some.all()
            for said in (plan.full(t * 64, before, n, window, sinks), plan.whole(t, before, n, window, sinks)):
                assert not said or whole
        for i in range(n):
            w = (ctypes.c_uint64 * plan.words())()
            depth = plan.walk(c_parents, i, before, window, sinks, w)
            for t in tiles:
                m = plan.mask(t * 64, before, depth, w, window, sinks)
                bits = [bool(m >> b & 1) for b in range(64)]
                want = list(seen[i, t * 64:t * 64 + 64])
                assert bits == want + [False] * (64 - len(want))
    assert not plan.whole(10, 640, 3, 0, 0) and plan.whole(9, 640, 3, 0, 0)


def test_parents_come_before_their_nodes(plan):
    for i in (0, 1, 7, 255):
        for p in (-1, 0, i - 1):
            if p < i:
                assert plan.parent(i, p) == p
        for p in (i, i + 1, -2, 2 ** 31 - 1, -2 ** 31):
            assert plan.parent(i, p) == -2


def test_the_oracles_trees():
    """By hand: 0 and 3 are roots, 1 and 2 children of 0, 4 of 3, 5 of 4."""
    parents = [-1, 0, 0, -1, 3, 4]
    seen = tree_visible(parents, 2, 0, 0)
    want = [[0, 1, 2], [0, 1, 2, 3], [0, 1, 2, 4], [0, 1, 5], [0, 1, 5, 6], [0, 1, 5, 6, 7]]
    assert [list(np.flatnonzero(r)) for r in seen] == want
    # positions 2, 3, 3, 2, 3, 4: a window of 2 and a sink
    seen = tree_visible(parents, 2, 2, 1)
    want = [[0, 1, 2], [0, 2, 3], [0, 2, 4], [0, 1, 5], [0, 5, 6], [0, 6, 7]]
    assert [list(np.flatnonzero(r)) for r in seen] == want
    # a chain is causal
    for w, s in ((0, 0), (3, 0), (5, 2)):
        chain = tree_visible(list(range(-1, 8)), 20, w, s)
        assert (chain == np.stack([visible(20 + i, 29, w, s) for i in range(9)])).all()
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(5, 4, 64)), rng.normal(size=(30, 2, 64)), rng.normal(size=(30, 2, 64))
    np.testing.assert_allclose(tree_attend_fp64(q, k, v, [-1, 0, 1, 2, 3], 7, 1, 0.125),
                               causal_attend_fp64(q, k, v, 25, 7, 1, 0.125), rtol=1e-12)


@pytest.mark.parametrize("distance", [1, 2, 4, 8, 16, 32])
def test_the_oracles_rotation(distance):
    """Lengths of pairs stay, angles add up, whole turns change nothing, q . k goes by distance."""
    rng = np.random.default_rng(distance)
    freq, axis = 1000.0 ** (-np.arange(32) / 32), np.arange(32) % 3
    x, y = rng.normal(size=(4, 2, 64)), rng.normal(size=(4, 2, 64))
    a, b = rng.integers(-99, 99, (4, 3)), rng.integers(-99, 99, (4, 3))
    turn = lambda r, p: rotate_fp64(r, p, freq, axis, distance)
    np.testing.assert_allclose(turn(turn(x, a), b), turn(x, a + b), atol=1e-12)
    np.testing.assert_allclose((turn(x, a) * turn(y, b)).sum(-1), (x * turn(y, b - a)).sum(-1), atol=1e-11)
    first = np.array([i // distance * 2 * distance + i % distance for i in range(32)])
    assert sorted(np.concatenate([first, first + distance])) == list(range(64))
    one = np.zeros((1, 1, 64))
    one[0, 0, first[5]] = 1.0
    got = rotate_fp64(one, np.array([[0, 0, 7]]), freq, axis, distance)[0, 0]
    assert np.isclose(got[first[5]], np.cos(7 * freq[5])) and np.isclose(got[first[5] + distance], np.sin(7 * freq[5]))
    assert np.count_nonzero(got) == 2


@pytest.mark.parametrize("flags", [[], ["-ffp-contract=fast", "-mfma"]], ids=["plain", "contracted"])
def test_frequencies_to_turns(tmp_path, flags):
    """freq / 2 pi to 1.1 x 2^-64 of a turn, against fractions, also where the compiler fuses
    products and sums (as it does on Arm)."""
    import platform
    from fractions import Fraction
    from oracle.tokens import TWO_PI
    if platform.machine() != "x86_64":
        flags = [f for f in flags if f != "-mfma"]
    src, so = str(tmp_path / "turn.cpp"), str(tmp_path / "turn.so")
    with open(src, "w") as f:
        f.write('#include "pkv_token_plan.h"\nextern "C" uint64_t turn(double f) { return pkv::rotary_turn(f); }\n')
    subprocess.run(["g++", "-std=c++17", "-O3", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC] + flags + [src, "-o", so],
                   check=True)
    turn = ctypes.CDLL(so).turn
    turn.restype, turn.argtypes = ctypes.c_uint64, [ctypes.c_double]
    rng = random.Random(0)
    freqs = [0.0, 1.0, -1.0, np.pi, 2 * np.pi, -np.pi, 4 * np.pi, 1e-30, -1e-30, 2.0 ** 20, -2.0 ** 20, 2.0 ** -64, 1e-5]
    freqs += [10000.0 ** (-i / 32) for i in range(32)] + [rng.uniform(-1, 1) * 2.0 ** rng.uniform(-40, 20) for _ in range(500)]
    for f in freqs:
        exact = Fraction(float(f)) / Fraction(TWO_PI) * 2 ** 64
        off = (Fraction(turn(f)) - exact + 2 ** 63) % 2 ** 64 - 2 ** 63
        assert abs(off) <= Fraction(11, 10), f     # two roundings to whole numbers, and the digits' end


# --------------------------------------------------------- the library's host code
def numbers(n, fill=0):
    import torch
    return torch.full((n,), fill, dtype=torch.int32)


def test_refusals(lib, cache):
    """Arguments outside their limits are refused before anything is launched or changed."""
    import torch
    from paged_kv_cache_build_gb300 import PkvError, Rotary
    s = HostStream()
    a, b = cache.open_token_stream(500), cache.open_token_stream(100, window=10, sinks=2)
    B = cache.token_batch
    cache.append_tokens(B([a, b], [200, 60]), rows(260, 2), rows(260, 2), stream=s)
    lib.pkv_evict_window(cache.h, b, None)
    rot = Rotary.sections([16, 16])
    flat = torch.zeros(2 * 4 * 64 + 64, dtype=torch.bfloat16)
    flat = flat[(-flat.data_ptr() % 16) // 2:]
    two = torch.zeros((2, 2), dtype=torch.int32)

    def turn(batch, n, r=rot, positions=None, q=None, q_out=None, layer=0):
        positions = torch.zeros((n, r.axes), dtype=torch.int32) if positions is None else positions
        return lambda: cache.append_tokens_rotary(batch, rows(n, 2), rows(n, 2), positions, r, q=q, q_out=q_out,
                                                  layer=layer, stream=s)

    def look(batch, n, heads=4, parents=None, **kw):
        kw.setdefault("out", rows(n, heads))
        return lambda: cache.attend_tree(batch, rows(n, heads), numbers(n, -1) if parents is None else parents,
                                         stream=s, **kw)

    def keep(batch, kept, accepted):
        return lambda: cache.keep_tokens(batch, kept, accepted, stream=s)

    def state():
        free = ctypes.c_int()
        lib.pkv_free_pages(cache.h, ctypes.byref(free))
        return cache.token_info(a), cache.token_info(b), free.value, lib.fake_launches(), lib.fake_alloc_calls()

    one = rows(1, 4)
    refused = {
        "INVALID": [
            turn(B([a], [301]), 301), turn(B([a, a], [1, 1]), 2), turn(B([7], [1]), 1), turn(B([a], [1]), 1, layer=2),
            turn(B([a], [1]), 1, r=Rotary([1.0] * 32, pair_distance=3)), turn(B([a], [1]), 1, r=Rotary([1.0] * 32, pair_distance=64)),
            turn(B([a], [1]), 1, r=Rotary([1.0] * 32, pair_distance=0)), turn(B([a], [1]), 1, r=Rotary([1.0] * 32, axes=5)),
            turn(B([a], [1]), 1, r=Rotary([1.0] * 32, [-1] * 32, axes=1)), turn(B([a], [1]), 1, r=Rotary([1.0] * 32, [1] * 32, axes=1)),
            turn(B([a], [1]), 1, r=Rotary([float("nan")] * 32)), turn(B([a], [1]), 1, r=Rotary([float("inf")] * 32)),
            turn(B([a], [1]), 1, r=Rotary([2.0 ** 20 + 1] * 32)),
            turn(B([a], [1]), 1, q=flat[1:257].view(1, 4, 64), q_out=one), turn(B([a], [1]), 1, q=one, q_out=flat[1:257].view(1, 4, 64)),
            turn(B([a], [2]), 2, q=flat.as_strided((2, 4, 64), (260, 64, 1)), q_out=rows(2, 4)),
            look(B([a, a], [1, 1]), 2),
            look(B([a], [1]), 1, layer=2), look(B([a], [1]), 1, heads=3), look(B([a], [1]), 1, window=-1),
            look(B([a], [1]), 1, sinks=1), look(B([a], [1]), 1, sm_scale=float("nan")),
            keep(B([a], [201]), numbers(1), B([a], [1])), keep(B([a], [2]), numbers(3), B([a], [3])),
            keep(B([a, a], [2, 2]), numbers(2), B([a, a], [1, 1])),
        ],
        "STATE": [
            look(B([b], [1]), 1), look(B([b], [1]), 1, window=40), look(B([b], [1]), 1, window=10, sinks=17),
            look(B([a], [201]), 201), look(B([b], [30]), 30, window=10, sinks=2),
            keep(B([b], [60]), numbers(1), B([b], [1])), keep(B([b], [40]), numbers(30), B([b], [30])),
            keep(B([b], [9]), numbers(0), B([b], [0])),
        ],
        "OOM": [turn(B([a, b], [200, 10]), 210)],
        "ValueError": [
            turn(B([a], [1]), 1, positions=two), turn(B([a], [2]), 2, positions=two.long()),
            turn(B([a], [2]), 2, positions=torch.zeros((2, 4), dtype=torch.int32)[:, ::2]), turn(B([a], [1]), 1, q_out=one),
            turn(B([a], [1]), 1, q=one, q_out=rows(2, 4)), turn(B([a], [1]), 1, q=rows(2, 4)),
            lambda: Rotary([1.0] * 31), lambda: Rotary([1.0] * 32, [0] * 31), lambda: Rotary([1.0] * 32, axes=2 ** 32 + 1),
            lambda: Rotary([1.0] * 32, pair_distance=2 ** 32 + 1), lambda: Rotary([1.0] * 32, [2 ** 32] * 32, axes=1),
            lambda: Rotary.sections([16, 15]), lambda: Rotary.sections([33, -1]),
            look(B([a], [2]), 2, parents=numbers(1)), look(B([a], [2]), 2, parents=numbers(2).long()),
            look(B([a], [2]), 2, parents=numbers(4)[::2]), look(B([a], [1]), 1, out=rows(2, 4)),
            look(B([a], [1]), 1, layer=2 ** 32), look(B([a], [1]), 1, window=2 ** 32), look(B([a], [1]), 1, sm_scale=1e-45),
            keep(B([a], [3]), numbers(2), B([b], [2])), keep(B([a], [3]), numbers(2), B([a, b], [2, 0])),
            keep(B([a], [3]), numbers(3), B([a], [2])), keep(B([a], [3]), numbers(2).long(), B([a], [2])),
        ],
    }
    for code, calls in refused.items():
        for i, call in enumerate(calls):
            before = state()
            with pytest.raises((PkvError, ValueError)) as e:
                call()
            assert getattr(e.value, "code", "ValueError") == code, (i, code, e.value)
            assert state() == before
    # rows of frames and chunk streams, and null pointers
    from paged_kv_cache_build_gb300 import frame_stream_cfg
    f = cache.open_stream(frame_stream_cfg(2, 4, 16, 6))
    for call in (turn(B([f], [1]), 1), look(B([f], [1]), 1), keep(B([f], [1]), numbers(1), B([f], [1]))):
        with pytest.raises(PkvError) as e:
            call()
        assert e.value.code == "STATE"
    x = rows(1, 4).data_ptr()
    i1, off = (ctypes.c_int * 1)(a), (ctypes.c_int * 2)(0, 1)
    L, h = lib, cache.h
    for bad in (lambda: L.pkv_append_tokens_rotary(h, 1, i1, off, 0, x, x, 0, 0, x, 4, 0, x, None, rot.cfg, None),
                lambda: L.pkv_append_tokens_rotary(h, 1, i1, off, 0, x, x, 0, 0, x, 4, 0, x, x + 2, rot.cfg, None),
                lambda: L.pkv_append_tokens_rotary(h, 1, i1, off, 0, x, x, 0, 0, x, 4, 0, x, x, None, None),
                lambda: L.pkv_append_tokens_rotary(h, 1, i1, off, 0, x, x, 0, 0, None, 4, 0, x, x, rot.cfg, None),
                lambda: L.pkv_append_tokens_rotary(h, 1, i1, off, 0, x, x, 0, 0, x, -1, 0, x, x, rot.cfg, None),
                lambda: L.pkv_append_tokens_rotary(h, 1, i1, off, 0, x, x, 0, 0, x, 257, 0, x, x, rot.cfg, None),
                lambda: L.pkv_append_tokens_rotary(h, 1, i1, off, 0, x, x, 0, 0, x, 4, 264, x, x, rot.cfg, None),
                lambda: L.pkv_append_tokens_rotary(h, 1, i1, None, 0, x, x, 0, 0, x, 4, 0, x, x, rot.cfg, None),
                lambda: L.pkv_append_tokens_rotary(None, 1, i1, off, 0, x, x, 0, 0, x, 4, 0, x, x, rot.cfg, None),
                lambda: L.pkv_attend_tree(h, x, 4, 0, off, i1, 1, 0, None, x, 0, 0, 0.0, None),
                lambda: L.pkv_attend_tree(h, x, 4, 0, off, i1, 1, 0, x + 2, x, 0, 0, 0.0, None),
                lambda: L.pkv_attend_tree(h, x, 4, 0, (ctypes.c_int * 2)(0, 257), i1, 1, 0, x, x, 0, 0, 0.0, None),
                lambda: L.pkv_attend_tree(None, x, 4, 0, off, i1, 1, 0, x, x, 0, 0, 0.0, None),
                lambda: L.pkv_keep_tokens(h, 1, i1, off, off, None, None),
                lambda: L.pkv_keep_tokens(h, 1, i1, off, off, x + 2, None),
                lambda: L.pkv_keep_tokens(h, 1, i1, off, (ctypes.c_int * 2)(1, 1), x, None),
                lambda: L.pkv_keep_tokens(h, 1, i1, off, (ctypes.c_int * 2)(0, -1), x, None),
                lambda: L.pkv_keep_tokens(h, 1, i1, off, None, x, None),
                lambda: L.pkv_keep_tokens(None, 1, i1, off, off, x, None)):
        before = state()
        assert bad() == 1
        assert state() == before
    # nothing to do is no error, and launches nothing
    before = state()
    turn(B([a], [0]), 0)()
    look(B([a, b], [0, 0]), 0)()
    keep(B([a], [0]), numbers(0), B([a], [0]))()
    assert state() == before
    # the limits themselves
    turn(B([a], [1]), 1, r=Rotary([2.0 ** 20] * 32, [3] * 32, pair_distance=1))()
    keep(B([a], [1]), numbers(0), B([a], [0]))()
    look(B([a], [200]), 200)()


def test_another_device_is_refused(lib, cache):
    from paged_kv_cache_build_gb300 import PkvError, Rotary
    s = HostStream()
    sid = cache.open_token_stream(100)
    b = cache.token_batch([sid], [3])
    positions = numbers(3)
    calls = (lambda: cache.append_tokens_rotary(b, rows(3, 2), rows(3, 2), positions, Rotary([1.0] * 32), stream=s),
             lambda: cache.attend_tree(b, rows(3, 4), numbers(3, -1), out=rows(3, 4), stream=s),
             lambda: cache.keep_tokens(b, numbers(1), cache.token_batch([sid], [1]), stream=s))
    for call in calls:
        before = lib.fake_launches(), cache.token_info(sid)
        lib.fake_set_device(1)
        with pytest.raises(PkvError) as e:
            call()
        assert e.value.code == "INVALID" and "device" in str(e.value)
        lib.fake_set_device(0)
        assert (lib.fake_launches(), cache.token_info(sid)) == before
        call()
        assert lib.fake_launches() > before[0]


@pytest.mark.parametrize("seed", range(4))
def test_calls_are_accepted_as_the_page_state_allows(lib, cache, seed):
    """Random appends, trees, kept numbers, drops and evictions: each is accepted or refused,
    with its code, as the oracle's pages say, and the counters follow."""
    from paged_kv_cache_build_gb300 import PkvError, Rotary
    rng = random.Random(seed)
    S, s, rot = 16, HostStream(), Rotary([1.0] * 32)
    ora = TokenStreamsOracle(20, S)
    sids = []
    for window, sinks in [(0, 0), (1, 0), (rng.randrange(1, 60), rng.choice([0, 1, 16, 17, 40])), (33, 5)]:
        sids.append(cache.open_token_stream(200, window, sinks))
        ora.open(sids[-1], 200, window, sinks)

    def outcome(f):
        try:
            f()
        except (PkvError, TokenError) as e:
            return e.code
        return "OK"

    def sees(sid, n, window, sinks):
        st = ora.streams[sid]
        if n > st["len"]:
            raise TokenError("STATE")
        for i in range(n):                       # a node at any depth up to its number
            seen = visible(st["len"] - n + i, st["len"], window, sinks)
            if not all(p // S in st["pages"] for p in np.flatnonzero(seen)):
                raise TokenError("STATE")

    for _ in range(300):
        op = rng.choice(["append", "append", "keep", "keep", "rollback", "evict", "attend", "attend", "layer"])
        some = rng.sample(sids, rng.randrange(1, 4))
        counts = [rng.choice([0, 1, 2, 15, 16, 17, rng.randrange(1, 70)]) for _ in some]
        sid, n = some[0], counts[0]
        batch = cache.token_batch(some, counts)
        if op == "append":
            x = rows(batch.rows, 2)
            got = outcome(lambda: cache.append_tokens_rotary(batch, x, x, numbers(batch.rows), rot, stream=s))
            want = outcome(lambda: ora.append(some, counts))
        elif op == "keep":
            kept = [rng.randrange(0, c + 1) for c in counts]
            got = outcome(lambda: cache.keep_tokens(batch, numbers(sum(kept)), cache.token_batch(some, kept), stream=s))
            want = outcome(lambda: ora.keep(some, counts, kept))
            if got != "OK":                      # which of a batch's faults is named is open
                assert want != "OK"
                want = got
        elif op == "rollback":
            got = outcome(lambda: cache._check(lib.pkv_rollback_last_frame(cache.h, sid, None)))
            want = outcome(lambda: ora.rollback(sid))
        elif op == "evict":
            got, want = outcome(lambda: cache._check(lib.pkv_evict_window(cache.h, sid, None))), outcome(lambda: ora.evict(sid))
        elif op == "layer":
            last = ora.streams[sid]["last"]
            n = last or 1
            x = rows(n, 2)
            got = outcome(lambda: cache.append_tokens_rotary(cache.token_batch([sid], [n]), x, x, numbers(n), rot, layer=1,
                                                             stream=s))
            want = "OK" if last else "STATE"
        else:
            window = rng.choice([0, 1, 2, 33, rng.randrange(1, 80)])
            sinks = rng.choice([0, 1, 16, 17, 45, 300]) if window else 0
            q = rows(n, 4)
            got = outcome(lambda: cache.attend_tree(cache.token_batch([sid], [n]), q, numbers(n, -1), window=window,
                                                    sinks=sinks, out=q, stream=s))
            want = outcome(lambda: sees(sid, n, window, sinks))
        assert got == want, (op, some, counts, ora.streams)
        for i in sids:
            st = ora.streams[i]
            free = ctypes.c_int()
            lib.pkv_free_pages(cache.h, ctypes.byref(free))
            assert (cache.token_info(i)[0], free.value) == (st["len"], len(ora.free))


def test_outputs_of_a_side_streams_call_are_allocated_for_it(lib, cache, monkeypatch):
    """A block from the current stream's pool may still be in use there."""
    import contextlib
    import torch
    from paged_kv_cache_build_gb300 import Rotary
    b = cache.token_batch([cache.open_token_stream(100)], [3])
    s, on, made = HostStream(), [None], []

    @contextlib.contextmanager
    def stream(x):
        on[0] = x
        yield
        on[0] = None

    def alloc(like, **kw):
        made.append(on[0])
        return rows(*like[:2])

    monkeypatch.setattr(torch.cuda, "stream", stream)
    positions, q, k, parents = numbers(3), rows(3, 4), rows(3, 2), numbers(3, -1)
    monkeypatch.setattr(torch, "empty", alloc)
    assert cache.append_tokens_rotary(b, k, k, positions, Rotary([1.0] * 32), q=q, stream=s).shape == (3, 4, 64)
    assert cache.attend_tree(b, q, parents, stream=s).shape == (3, 4, 64)
    assert made == [s, s]
