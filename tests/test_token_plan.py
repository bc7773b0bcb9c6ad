"""Token streams on the CPU: the host's counters, tile lists and masks
(csrc/pkv_token_plan.h, compiled for the host) against the oracle's page state
machine and the visible set spelled out; the oracle against hand-derived values;
the binding's and the library's refusals that need no device."""

import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from oracle.tokens import TokenError, TokenStreamsOracle, causal_attend_fp64, visible

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_kv_cache_build_gb300", "csrc")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "token_plan_shim.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.plan_open.restype = ctypes.c_void_p
    L.plan_mask.restype = ctypes.c_ulonglong
    for f in ("plan_free", "plan_append", "plan_can_drop", "plan_drop", "plan_evict", "plan_holds", "plan_live",
              "plan_zero"):
        getattr(L, f).argtypes = [ctypes.c_void_p] + [ctypes.c_int] * {"plan_append": 1, "plan_can_drop": 1,
                                                                       "plan_drop": 1, "plan_holds": 2,
                                                                       "plan_zero": 3}.get(f, 0)
    L.plan_live.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int)]
    return L


@pytest.mark.parametrize("page,window,sinks", [(16, 0, 0), (16, 1, 0), (16, 5, 3), (32, 40, 33), (64, 64, 1),
                                               (64, 200, 64), (16, 47, 100)])
def test_counters_follow_the_page_state_machine(plan, page, window, sinks):
    rng = random.Random(page * 1000 + window)
    ora = TokenStreamsOracle(400, page)
    ora.open(0, 4000, window, sinks)
    t = plan.plan_open(page, 4000, window, sinks)
    live = (ctypes.c_int * 4)()
    for _ in range(300):
        st = ora.streams[0]
        before = len(ora.free)
        op = rng.choice(["append", "append", "append", "drop", "evict"])
        if op == "append":
            n = rng.choice([1, 2, page - 1, page, page + 1, rng.randrange(1, 150)])
            if st["len"] + n > 4000:
                break
            old = len([i for i in range(-(-st["len"] // page))])
            pos0 = st["len"]
            ora.append([0], [n])
            assert plan.plan_append(t, n) == before - len(ora.free)
            # zeroed: from the new end to the end of a page that this append opened
            end = pos0 + n
            zero = -end % page if -(-end // page) > old else 0
            assert plan.plan_zero(t, pos0, n, old) == zero
        elif op == "drop":
            n = rng.randrange(0, min(st["len"], 2 * page) + 1)
            try:
                ora.drop([0], [n])
                ok = True
            except TokenError:
                ok = False
            # the plan may refuse a drop that only a sink page's own slots would serve
            mine = bool(plan.plan_can_drop(t, n))
            assert mine <= ok
            if ok and not mine:
                pytest.fail("a drop that the pages allow is refused")
            if mine:
                assert plan.plan_drop(t, n) == len(ora.free) - before
        else:
            ora.evict(0)
            assert plan.plan_evict(t) == len(ora.free) - before
        plan.plan_live(t, live)
        held = sorted(ora.streams[0]["pages"])
        mine = list(range(live[0])) + list(range(live[2], live[3]))[:live[1]]
        assert mine == held
        # what a query of any window up to the stream's own may ask for
        if window:
            length = ora.streams[0]["len"]
            for p in (length - 1, length - 2, length - page):
                if p < 0:
                    continue
                need = np.flatnonzero(visible(p, p + 1, window, sinks))
                holds = all(j // page in ora.streams[0]["pages"] for j in need)
                lo = max(0, p - window + 1)
                if plan.plan_holds(t, lo, sinks):
                    assert holds
                elif holds:
                    # refused though held: only while the window reaches into the sinks' pages
                    assert lo < -(-sinks // page) * page
    plan.plan_free(t)


def test_tiles_and_masks(plan):
    rng = random.Random(7)
    cap = (ctypes.c_int * 4096)()
    for _ in range(400):
        p0 = rng.randrange(0, rng.choice([70, 400, 3000]))
        p1 = p0 + rng.choice([0, 0, 3, 63, 64, 300])
        window = rng.choice([0, 1, 2, 63, 64, 65, 500])
        sinks = rng.choice([0, 1, 4, 64, 65, 130]) if window else 0
        seen = np.zeros(p1 + 65, dtype=bool)
        every = np.ones(p1 + 65, dtype=bool)
        for p in range(p0, p1 + 1):
            s = visible(p, p1 + 65, window, sinks)
            seen |= s
            every &= s
        n = plan.plan_tiles(p0, p1, window, sinks, cap, 4096)
        tiles = list(cap[:n])
        assert tiles == sorted(set(tiles))
        need = sorted(set(np.flatnonzero(seen) // 64))
        assert set(need) <= set(tiles)
        # nothing but the tiles that are seen, or lie between the sinks and the window
        # of the first row when sinks reach past a position not yet written
        assert len(tiles) <= len(need) + 1 + (sinks + 63) // 64
        for tile in tiles:
            b = tile * 64
            want_full = bool(every[b:b + 64].all()) and b + 64 <= len(every)
            got_full = bool(plan.plan_full(b, p0, p1, window, sinks))
            assert not got_full or want_full
            assert bool(plan.plan_whole(tile, p0, p1, window, sinks)) == got_full
            assert bool(plan.plan_needs(tile, p0, p1, window, sinks)) >= bool(seen[b:b + 64].any())
            if got_full:
                assert plan.plan_needs(tile, p0, p1, window, sinks)
        # part of the rows: no tile that they see is left out
        q0 = rng.randrange(p0, p1 + 1)
        q1 = rng.randrange(q0, p1 + 1)
        part = np.zeros(p1 + 65, dtype=bool)
        for p in range(q0, q1 + 1):
            part |= visible(p, p1 + 65, window, sinks)
        for tile in sorted(set((np.flatnonzero(part) // 64).tolist())):
            assert plan.plan_needs(tile, q0, q1, window, sinks) and tile in tiles
        for tile in tiles:
            b = tile * 64
            for p in {p0, p1, (p0 + p1) // 2}:
                bits = plan.plan_mask(b, p, window, sinks)
                want = visible(p, b + 64, window, sinks)[b:]
                assert [bool(bits >> i & 1) for i in range(64)] == list(want)


def test_oracle_attention_by_hand():
    # two keys with equal scores: the mean; one key: itself; a window of 1: the own value
    q = np.zeros((2, 2, 64))
    k = np.zeros((2, 1, 64))
    v = np.stack([np.full((1, 64), 1.0), np.full((1, 64), 3.0)])
    out = causal_attend_fp64(q, k, v, 0, 0, 0, 0.125)
    assert np.all(out[0] == 1.0) and np.all(out[1] == 2.0)
    out = causal_attend_fp64(q, k, v, 0, 1, 0, 0.125)
    assert np.all(out[0] == 1.0) and np.all(out[1] == 3.0)
    out = causal_attend_fp64(q, k, v, 0, 1, 1, 0.125)
    assert np.all(out[1] == 2.0)
    # a score difference of log 3: weights 1/4, 3/4
    k[1, 0, 0], q[1, :, 0] = 1.0, np.log(3.0) / 0.125
    out = causal_attend_fp64(q, k, v, 0, 0, 0, 0.125)
    assert np.allclose(out[1], 0.25 * 1.0 + 0.75 * 3.0, atol=1e-15)


def test_null_handle_and_batch_refusals_without_gpu():
    from paged_kv_cache_build_gb300 import build
    build.build()
    from paged_kv_cache_build_gb300._lib import load
    from paged_kv_cache_build_gb300.cache import TokenBatch
    L = load()
    b = TokenBatch([0, 1], [1, 2])
    assert (b.n, b.rows) == (2, 3)
    sid = ctypes.c_int(0)
    assert L.pkv_stream_open_tokens(None, 10, 0, 0, ctypes.byref(sid)) == 1
    assert L.pkv_append_tokens(None, 2, b.sids, b.row_off, 0, None, None, 0, 0, None) == 1
    assert L.pkv_drop_tokens(None, 2, b.sids, b.counts, None) == 1
    assert L.pkv_read_tokens(None, 2, b.sids, None, b.row_off, 0, None, None, None) == 1
    assert L.pkv_attend_tokens(None, None, 16, 0, b.row_off, b.sids, 2, 0, None, 0, 0, 0.0, None) == 1
    assert b"null handle" in L.pkv_last_error(None)
    assert L.pkv_token_info(None, 0, None, None, None) == 1
    with pytest.raises(ValueError):
        TokenBatch([0], [1, 2])
    with pytest.raises(ValueError):
        TokenBatch([0], [-1])


@pytest.mark.parametrize("window", [1, 65, 2 ** 31 - 1])
def test_sinks_of_any_size(plan, window):
    """Sinks up to the largest int, past every key: the tiles are those without a window."""
    cap, all_of_them = (ctypes.c_int * 4096)(), (ctypes.c_int * 4096)()
    for p0, p1 in [(0, 0), (63, 64), (1000, 1500), (2 ** 17, 2 ** 17 + 100)]:
        n = plan.plan_tiles(p0, p1, 0, 0, all_of_them, 4096)
        for sinks in (p1 + 1, 2 ** 31 - 64, 2 ** 31 - 63, 2 ** 31 - 1):
            assert plan.plan_tiles(p0, p1, window, sinks, cap, 4096) == n
            assert list(cap[:n]) == list(all_of_them[:n])
            for tile in (0, p1 // 64 // 2, p1 // 64):
                assert plan.plan_needs(tile, p0, p1, window, sinks)
                assert plan.plan_whole(tile, p0, p1, window, sinks) == plan.plan_whole(tile, p0, p1, 0, 0)
                assert plan.plan_mask(64 * tile, p0, window, sinks) == plan.plan_mask(64 * tile, p0, 0, 0)


def test_stream_ids_past_32_bits_are_refused():
    from paged_kv_cache_build_gb300.cache import TokenBatch
    for sid in (2 ** 31, 2 ** 32, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            TokenBatch([sid], [1])
