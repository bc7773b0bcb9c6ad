"""Token streams' entry points without a GPU: the library's own host code, linked with a
CUDA runtime that keeps books instead of driving a device (fake_cudart.cpp)."""

import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

OK, INVALID = 0, 1


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from paged_kv_cache_build_gb300 import build
    from paged_kv_cache_build_gb300._lib import SIGNATURES
    build.build()
    so = str(tmp_path_factory.mktemp("host") / "host.so")
    objs = [os.path.join(build.BUILD, os.path.basename(s)[:-3] + ".o") for s in build.sources()]
    include = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    # -Bsymbolic: not the runtime that torch has loaded
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", include,
                    os.path.join(HERE, "fake_cudart.cpp")] + objs + ["-o", so], check=True)
    L = ctypes.CDLL(so)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    return L


@pytest.fixture(params=[False, True], ids=["bf16", "e4m3"])
def handle(lib, request):
    lib.fake_set_device(0)
    h = ctypes.c_void_p()
    create = lib.pkv_create_fp8 if request.param else lib.pkv_create_ex
    assert create(20, 16, 2, 64, 2, 8, ctypes.byref(h)) == OK
    yield h
    lib.fake_set_device(0)
    assert lib.pkv_destroy(h) == OK
    assert lib.fake_allocs(0) == lib.fake_allocs(1) == 0 and lib.fake_streams() == 0


def open_tokens(lib, h, *args):
    sid = ctypes.c_int(-1)
    return lib.pkv_stream_open_tokens(h, *args, ctypes.byref(sid)), sid.value


def test_a_new_handle_is_ready(lib, handle):
    """Neither may anything that creating a handle has queued."""
    assert lib.fake_queued() == 0


@pytest.mark.parametrize("cfg", [dict(mode=0, num_scale=2, window=4, n_patch=16, n_special=6),
                                 dict(mode=1, chunk_size=4, sliding_window_num=3, tokens_per_frame=22)],
                         ids=["frames", "chunks"])
def test_an_opened_frame_stream_is_ready(lib, handle, cfg):
    from paged_kv_cache_build_gb300._lib import StreamCfg
    sid = ctypes.c_int(-1)
    lib.cudaDeviceSynchronize()
    assert lib.pkv_stream_open(handle, ctypes.byref(StreamCfg(**cfg)), ctypes.byref(sid)) == OK
    assert lib.fake_queued() == 0


def test_an_opened_stream_is_ready(lib, handle):
    """Nothing that open has queued may still be to come when it returns: the caller's
    streams are not ordered behind the one that it was queued on."""
    for _ in range(2):                           # the first one lays out the handle's workspace, too
        lib.cudaDeviceSynchronize()
        r, _ = open_tokens(lib, handle, 100, 0, 0)
        assert r == OK
        assert lib.fake_queued() == 0


def test_another_device_is_refused(lib, handle):
    """Nothing is allocated or launched for a handle of device 0 while device 1 is
    current, and the state stays; on its own device the same calls work."""
    r, sid = open_tokens(lib, handle, 100, 20, 0)
    assert r == OK
    ints = lambda *x: (ctypes.c_int * len(x))(*x)
    rows = 2 * 64 * 2                            # bytes of a token's K or V
    mem = ctypes.create_string_buffer(90 * rows + 16)
    at = (ctypes.addressof(mem) + 15) // 16 * 16
    n = ctypes.c_size_t()
    words = (ctypes.c_int32 * 200)()
    table = (ctypes.c_int32 * 50)()
    table_at = ctypes.addressof(table)
    append = lambda c: lib.pkv_append_tokens(handle, 1, ints(sid), ints(0, c), 0, at, at, 0, 0, None)
    assert append(40) == OK
    calls = {
        "open": lambda: open_tokens(lib, handle, 100, 0, 0)[0],
        "append": lambda: append(3),
        "rollback": lambda: lib.pkv_rollback_last_frame(handle, sid, None),
        "append again": lambda: append(50),
        "read": lambda: lib.pkv_read_tokens(handle, 1, ints(sid), None, ints(0, 5), 0, at, at, None),
        "attend": lambda: lib.pkv_attend_tokens(handle, at, 2, 0, ints(0, 1), ints(sid), 1, 0, at, 20, 0, 0.0, None),
        "drop": lambda: lib.pkv_drop_tokens(handle, 1, ints(sid), ints(20), None),
        "evict": lambda: lib.pkv_evict_window(handle, sid, None),
        "table": lambda: lib.pkv_build_visible_page_table(handle, sid, table_at, table_at, 50, None, None, None),
        "export": lambda: lib.pkv_export_state(handle, sid, words, 200, ctypes.byref(n)),
        "reset": lambda: lib.pkv_stream_reset(handle, sid, None),
        "close": lambda: lib.pkv_stream_close(handle, sid, None),
    }

    def state():
        v = [ctypes.c_int() for _ in range(4)]
        assert lib.pkv_token_info(handle, sid, *map(ctypes.byref, v[:3])) == OK
        assert lib.pkv_free_pages(handle, ctypes.byref(v[3])) == OK
        return [x.value for x in v] + [lib.fake_launches(), lib.fake_alloc_calls()]

    for name, call in calls.items():
        before = state()
        lib.fake_set_device(1)
        assert call() == INVALID, name
        assert b"device" in lib.pkv_last_error(handle)
        lib.fake_set_device(0)
        assert state() == before, name
        assert call() == OK, name
    assert lib.fake_allocs(1) == 0


@pytest.fixture
def cache(lib, handle):
    """The Python class over the same host code, its tensors in host memory."""
    import torch
    from paged_kv_cache_build_gb300 import PagedKVCache
    c = PagedKVCache.__new__(PagedKVCache)
    c.lib, c.h, c.device = lib, handle, torch.device("cpu")
    c.pool_pages, c.page_size, c.heads, c.head_dim, c.layers = 20, 16, 2, 64, 2
    yield c
    c.h = None                                   # the handle is its fixture's


class HostStream:
    cuda_stream = 0


def rows(n, heads):
    import torch
    mem = torch.zeros(n * heads * 64 + 8, dtype=torch.bfloat16)
    at = (-mem.data_ptr() % 16) // 2
    return mem[at:at + n * heads * 64].view(n, heads, 64)


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 1, -2 ** 31 - 1])
def test_numbers_past_32_bits_are_refused(lib, cache, big):
    """A layer or stream id that C would cut down to a valid one."""
    sid = cache.open_token_stream(100)
    b = cache.token_batch([sid], [3])
    s = HostStream()
    cache.append_tokens(b, rows(3, 2), rows(3, 2), stream=s)
    launches = lib.fake_launches()
    for call in (lambda: cache.append_tokens(b, rows(3, 2), rows(3, 2), layer=big, stream=s),
                 lambda: cache.attend_tokens(b, rows(3, 4), layer=big, out=rows(3, 4), stream=s),
                 lambda: cache.read_tokens(b, layer=big, k_out=rows(3, 2), v_out=rows(3, 2), stream=s),
                 lambda: cache.token_info(big)):
        with pytest.raises(ValueError):
            call()
    assert lib.fake_launches() == launches
    assert cache.token_info(sid)[0] == 3


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 3e38, 1e39, 2.0 ** -127, 1e-45, 1e-50])
def test_scales_that_fp32_does_not_hold_are_refused(lib, cache, scale):
    """sm_scale (times log2 e) has to be a normal fp32 number, or 0 or less: the default."""
    from paged_kv_cache_build_gb300 import PkvError
    b = cache.token_batch([cache.open_token_stream(100)], [3])
    s = HostStream()
    cache.append_tokens(b, rows(3, 2), rows(3, 2), stream=s)
    attend = lambda x: cache.attend_tokens(b, rows(3, 4), out=rows(3, 4), sm_scale=x, stream=s)
    launches = lib.fake_launches()
    with pytest.raises((PkvError, ValueError)) as e:
        attend(scale)
    assert getattr(e.value, "code", "INVALID") == "INVALID"
    assert lib.fake_launches() == launches
    for fine in (0.0, -0.0, -1.0, float("-inf"), 2.0 ** -126, 2.3e38, 0.3, 1):
        attend(fine)
    assert lib.fake_launches() > launches


def test_outputs_of_a_side_streams_call_are_allocated_for_it(lib, cache, monkeypatch):
    """A block from the current stream's pool may still be in use there."""
    import contextlib
    import torch
    sid = cache.open_token_stream(100)
    b = cache.token_batch([sid], [3])
    s = HostStream()
    cache.append_tokens(b, rows(3, 2), rows(3, 2), stream=s)
    on, made = [None], []

    @contextlib.contextmanager
    def stream(x):
        on[0] = x
        yield
        on[0] = None

    monkeypatch.setattr(torch.cuda, "stream", stream)
    for f in ("empty", "empty_like"):
        def alloc(like, **kw):
            made.append(on[0])
            return rows(*getattr(like, "shape", like)[:2])
        monkeypatch.setattr(torch, f, alloc)
    assert cache.attend_tokens(b, rows(3, 4), stream=s).shape == (3, 4, 64)
    assert made == [s]
    assert [x.shape for x in cache.read_tokens(b, stream=s)] == [(3, 2, 64)] * 2
    assert made == [s, s, s]


@pytest.mark.parametrize("sinks", [0, 1, 16, 20])
def test_reads_across_the_sinks_end(lib, cache, sinks):
    """A range that begins in the sinks' pages and ends behind them can be read as long as
    nothing between them is evicted."""
    from paged_kv_cache_build_gb300 import PkvError
    s = HostStream()
    sid = cache.open_token_stream(200, window=50, sinks=sinks)
    cache.append_tokens(cache.token_batch([sid], [100]), rows(100, 2), rows(100, 2), stream=s)
    read = lambda pos0, n: cache.read_tokens(cache.token_batch([sid], [n]), [pos0], k_out=rows(n, 2), v_out=rows(n, 2),
                                             stream=s)
    for pos0, n in ((0, 100), (15, 2), (16, 1), (31, 2), (0, 33)):
        read(pos0, n)
    lib.pkv_evict_window(cache.h, sid, None)
    _, a, b = cache.token_info(sid)
    assert (a, b) == (-(-sinks // 16) * 16, 48)  # the next token sees from position 51 on
    read(b, 100 - b)
    if a:
        read(0, a)
    for pos0, n in ((a, 1), (b - 1, 1), (b - 1, 2), (a, b - a), (0, 100)):
        with pytest.raises(PkvError) as e:
            read(pos0, n)
        assert e.value.code == "STATE"


@pytest.mark.parametrize("seed", range(6))
def test_calls_are_accepted_as_the_page_state_allows(lib, cache, seed):
    """Random calls on streams with and without windows: each is accepted or refused, with
    its code, as the oracle's pages say, and the counters follow."""
    import random
    from oracle.tokens import TokenError, TokenStreamsOracle, visible
    from paged_kv_cache_build_gb300 import PkvError
    rng = random.Random(seed)
    S, s = 16, HostStream()
    ora = TokenStreamsOracle(20, S)
    kinds = [(0, 0), (1, 0), (rng.randrange(1, 60), rng.choice([0, 1, 16, 17, 40])), (33, 5)]
    sids = []
    for window, sinks in kinds:
        sids.append(cache.open_token_stream(200, window, sinks))
        ora.open(sids[-1], 200, window, sinks)

    def outcome(f):
        try:
            f()
        except (PkvError, TokenError) as e:
            return e.code
        return "OK"

    def live(sid, positions):
        if not all(p // S in ora.streams[sid]["pages"] for p in positions):
            raise TokenError("STATE")

    def sees(sid, n, window, sinks):
        length = ora.streams[sid]["len"]
        if n > length:
            raise TokenError("STATE")
        for p in range(length - n, length):
            live(sid, [j for j, v in enumerate(visible(p, length, window, sinks)) if v])

    for _ in range(300):
        op = rng.choice(["append", "append", "drop", "rollback", "evict", "read", "attend", "attend", "reset"])
        some = rng.sample(sids, rng.randrange(1, 4))
        counts = [rng.choice([0, 1, 2, 15, 16, 17, rng.randrange(1, 70)]) for _ in some]
        sid, n = some[0], counts[0]
        length = ora.streams[sid]["len"]
        batch = cache.token_batch(some, counts)
        if op == "append":
            x = rows(batch.rows, 2)
            got = outcome(lambda: cache.append_tokens(batch, x, x, stream=s))
            want = outcome(lambda: ora.append(some, counts))
        elif op == "drop":
            got = outcome(lambda: cache.drop_tokens(batch, stream=s))
            want = outcome(lambda: ora.drop(some, counts))
        elif op == "rollback":
            got = outcome(lambda: lib.pkv_rollback_last_frame(cache.h, sid, None) and cache._check(3))
            want = outcome(lambda: ora.rollback(sid))
        elif op == "evict":
            got, want = outcome(lambda: cache._check(lib.pkv_evict_window(cache.h, sid, None))), outcome(lambda: ora.evict(sid))
        elif op == "reset":
            if rng.random() < 0.7:
                continue
            got, want = outcome(lambda: cache._check(lib.pkv_stream_reset(cache.h, sid, None))), "OK"
            ora.release(sid)
        elif op == "read":
            n = min(n, length)
            pos0 = rng.randrange(0, length - n + 1)
            out = rows(n, 2)
            got = outcome(lambda: cache.read_tokens(cache.token_batch([sid], [n]), [pos0], k_out=out, v_out=out, stream=s))
            want = outcome(lambda: live(sid, range(pos0, pos0 + n)))
        else:
            window = rng.choice([0, 1, 2, 33, rng.randrange(1, 80)])
            sinks = rng.choice([0, 1, 16, 17, 45, 300]) if window else 0
            q = rows(n, 4)
            got = outcome(lambda: cache.attend_tokens(cache.token_batch([sid], [n]), q, window=window, sinks=sinks,
                                                      out=q, stream=s))
            want = outcome(lambda: sees(sid, n, window, sinks))
        if op == "drop" and got != "OK":         # which of a batch's faults is named is open
            assert want != "OK"
        else:
            assert got == want, (op, some, counts, ora.streams)
        for i in sids:
            st = ora.streams[i]
            free = ctypes.c_int()
            lib.pkv_free_pages(cache.h, ctypes.byref(free))
            assert (cache.token_info(i)[0], free.value) == (st["len"], len(ora.free))
            pages, tokens = ctypes.c_int(), ctypes.c_int()
            lib.pkv_visible_count(cache.h, i, ctypes.byref(pages), ctypes.byref(tokens))
            assert (pages.value, tokens.value) == (len(st["pages"]), sum(ora.table(i)[1]))
