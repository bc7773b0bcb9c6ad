"""Token streams where CUDA streams, other streams' pages and unusual rows meet (needs a
GB300). Tolerances: see test_gpu_tokens."""

import numpy as np
import pytest
import torch

from oracle.tokens import causal_attend_fp64

from .test_gpu_tokens import SCALE, Pool, _built, f64, stored, tolerance   # noqa: F401 (_built: a fixture)

pytestmark = pytest.mark.gpu


def busy(seconds=0.05):
    """Finite work on the current stream."""
    torch.cuda._sleep(int(seconds * 1.5e9))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_a_stream_opened_behind_a_busy_default_stream(fp8):
    """Opened while the default stream has work to do, and used on a side stream at once:
    the pages and the joined splits are right before and after that work ends."""
    side, done, behind = torch.cuda.Stream(), torch.cuda.Event(), []
    for waits in (0.0, 0.4):                     # the first turn loads the kernels
        p = Pool(400, 16, 2, fp8)
        torch.cuda.synchronize()
        for _ in range(2):                       # a handle's first open lays out its workspace, too
            busy(waits)
            done.record()
            sid = p.open()
            with torch.cuda.stream(side):
                batch = p.cache.token_batch([sid], [2000])
                k, v, q = p.rows(2000, 2), p.rows(2000, 2), p.rows(1, 4)
                p.ora.append([sid], [2000])
                p.cache.append_tokens(batch, k, v)
                out = p.cache.attend_tokens(p.cache.token_batch([sid], [1]), q)
                early = out.cpu()
            behind.append(not done.query())      # (not where the host was held up)
            kk, vv, qq = stored(k, fp8), stored(v, fp8), f64(q)
            ref = causal_attend_fp64(qq, kk, vv, 1999, 0, 0, SCALE)
            assert (np.abs(f64(early) - ref) <= tolerance(qq, kk, vv, ref, 1999, 0, 0, SCALE)).all()
            torch.cuda.synchronize()
            p.check_state(range(sid + 1))
            assert torch.equal(p.cache.attend_tokens(p.cache.token_batch([sid], [1]), q), out)
            torch.cuda.synchronize()
        p.cache.sync()
        p.cache.close()
    assert any(behind[2:]), "the default stream was to be busy meanwhile"


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 3, 7, 300])
@pytest.mark.parametrize("ahead,size", [(0, 1e-10), (14, 1e-4), (20, 1e-3), (25, 1e-2), (30, 1.0), (-20, 1e-12)])
def test_a_key_whose_value_is_zero(ahead, size, new, fp8):
    """Rows of zeros among small values, their scores 2^ahead times the others': they
    take weight and bring nothing, and the others' values keep their bits."""
    p = Pool(200, 16, 2, fp8, seed=new)
    n = 1500 + new
    sid = p.open(n)
    g = torch.Generator(device="cuda").manual_seed(7)
    k = torch.randn((n, 2, 64), generator=g, device="cuda")
    v = torch.randn((n, 2, 64), generator=g, device="cuda") * size
    q = torch.randn((new, 8, 64), generator=g, device="cuda")
    q[..., 0] = 8.0
    k[..., 0] = 0.0
    zero = [0, 17, 700, 1499]                    # the sink's place, and others
    k[zero] = 0.0
    k[zero, :, 0] = ahead * float(np.log(2.0))   # times 8 and the scale of 1/8
    v[zero] = 0.0
    v[17] = -0.0
    k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
    p.cache.append_tokens(p.cache.token_batch([sid], [n]), k, v)
    out = p.cache.attend_tokens(p.cache.token_batch([sid], [new]), q)
    p.cache.sync()
    kk, vv, qq = stored(k, fp8), stored(v, fp8), f64(q)
    ref = causal_attend_fp64(qq, kk, vv, n - new, 0, 0, SCALE)
    assert (np.abs(f64(out) - ref) / tolerance(qq, kk, vv, ref, n - new, 0, 0, SCALE)).max() <= 1
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 5, 300])
def test_values_that_are_all_zero(new, fp8):
    """A stream of zeros, and zeros up to the last keys, which no other part of the table
    knows of."""
    p = Pool(300, 16, 2, fp8)
    n = 1500 + new
    k, q = p.rows(n, 2), p.rows(new, 4)
    for tail in (0, 1, 70):
        sid = p.open(n)
        v = torch.zeros_like(k)
        if tail:
            v[n - tail:] = p.rows(tail, 2)
        p.cache.append_tokens(p.cache.token_batch([sid], [n]), k, v)
        out = p.cache.attend_tokens(p.cache.token_batch([sid], [new]), q)
        kk, vv, qq = stored(k, fp8), stored(v, fp8), f64(q)
        ref = causal_attend_fp64(qq, kk, vv, n - new, 0, 0, SCALE)
        assert (np.abs(f64(out) - ref) <= tolerance(qq, kk, vv, ref, n - new, 0, 0, SCALE)).all()
        p.cache.sync()
        p.cache.close_stream(sid)
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("new", [1, 7, 40, 300])
def test_another_streams_values_cannot_be_seen(new, page, fp8):
    """Pages that left a window hold another stream's rows, none of them finite: the tiles at
    the edges of the window and of the sinks, which cover such pages, bring nothing of them."""
    window, sinks = 20, 3
    p = Pool(64, page, 2, fp8, layers=2)
    a, b = p.open(window=window, sinks=sinks), p.open()
    for n in (403, 77):                          # two evictions: pages at the front and the back
        p.append([a], [n])
        p.cache.evict_window(a)
        p.ora.evict(a)
    p.append([a], [new])
    free = p.cache.free_pages()
    batch = p.cache.token_batch([b], [free * page])
    bad = torch.full((free * page, 2, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    bad[::3] = float("inf")
    for layer in range(2):
        p.cache.append_tokens(batch, bad, bad, layer=layer)
    assert p.cache.free_pages() == 0
    for layer in range(2):
        p.check_attend([a], [new], 2, window, sinks, layer=layer)
        p.check_attend([a], [min(new, 5)], 4, 2, 1, layer=layer)
    p.cache.close()


@pytest.mark.parametrize("new,fp8", [(1, False), (5, False), (40, False), (300, False), (1, True), (5, True)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_a_value_that_is_no_number_shows(what, new, fp8):
    """A visible key or value that is no number shows in every row that sees it, with the
    keys split over CTAs or not, and in no other head (on E4M3 pages with few rows: the
    matrix-unit kernel's conversion has no such code)."""
    p = Pool(300, 16, 2, fp8, max_streams=64)
    n = 3000 + new
    k, v, q = p.rows(n, 2), p.rows(n, 2), p.rows(new, 4)
    (k if what == "k" else v)[100, 1] = float("nan")
    sid = p.open(n)
    p.cache.append_tokens(p.cache.token_batch([sid], [n]), k, v)
    short = [p.open(1) for _ in range(50)]       # streams that fill the card with one CTA a block
    p.cache.append_tokens(p.cache.token_batch(short, [1] * 50), k[-50:], v[-50:])
    for others in ([], short):
        batch = p.cache.token_batch([sid] + others, [new] + [1] * len(others))
        qq = torch.cat([q, p.rows(len(others), 4)])
        out = p.cache.attend_tokens(batch, qq)
        assert torch.isnan(out[:new, 2:]).all()
        assert torch.isfinite(out[:new, :2]).all() and torch.isfinite(out[new:]).all()
    # a window that begins behind it hides it
    assert torch.isfinite(p.cache.attend_tokens(p.cache.token_batch([sid], [new]), q, window=2000)).all()
    p.cache.sync()
    p.cache.close()


def test_outputs_of_a_call_on_a_side_stream():
    """What the current stream still has to do with memory that was freed there does not
    reach the outputs of a call on another stream."""
    p = Pool(40, 64, 2)
    sid = p.open()
    p.append([sid], [500])
    batch = p.cache.token_batch([sid], [300])
    q = p.rows(300, 4)
    want = p.cache.attend_tokens(batch, q), *p.cache.read_tokens(batch)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy()
    for shape in ((300, 4, 64), (300, 2, 64), (300, 2, 64)):
        used = [torch.empty(shape, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
        for x in used:
            x.fill_(7.0)                         # behind the busy work
        del used, x
    got = p.cache.attend_tokens(batch, q, stream=side), *p.cache.read_tokens(batch, stream=side)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    p.cache.sync()
    p.cache.close()


@pytest.mark.parametrize("copies", [1, 40], ids=["few rows", "many rows"])
def test_ties_go_to_the_even_code(copies):
    """Every value half way between two codes, in rows of many exponents: the read-back is
    the even code's value (and the oracle's)."""
    code = np.arange(127)
    value = np.where(code < 8, code / 8 * 2.0 ** -6, (1 + code % 8 / 8) * 2.0 ** (code // 8 - 7.0))
    middle = (value[1:] + value[:-1]) / 2
    even = value[(np.arange(126) + 1) // 2 * 2]
    rows, want = [], []
    for e in list(range(-12, 13)) + [-110, -64, 63, 110]:
        for part in (slice(0, 63), slice(63, 126)):
            for sign in (1.0, -1.0):
                rows.append(np.concatenate([[448.0], sign * middle[part]]) * 2.0 ** e)
                want.append(np.concatenate([[448.0], sign * even[part]]) * 2.0 ** e)
    n = len(rows)
    x = torch.tensor(np.stack(rows)[:, None].repeat(2, 1), dtype=torch.float32).bfloat16().cuda()
    np.testing.assert_array_equal(f64(x)[:, 0], np.stack(rows))      # bf16 holds the middles
    x = x.repeat(copies, 1, 1)
    p = Pool(-(-copies * n // 64), 64, 2, True)
    sid = p.open()
    batch = p.cache.token_batch([sid], [copies * n])
    p.cache.append_tokens(batch, x, x)
    for got in p.cache.read_tokens(batch):
        np.testing.assert_array_equal(f64(got), np.stack(want * copies)[:, None].repeat(2, 1))
        np.testing.assert_array_equal(f64(got), stored(x, True))
    p.cache.sync()
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_no_call_on_a_token_stream_allocates(fp8):
    """Every call between a stream's opening and its end, few rows and many, on both layers:
    the device's free memory stays, and so does the frame calls' scratch."""
    for attempt in ("the kernels are loaded", "what is looked at"):
        p = Pool(700, 16, 2, fp8, layers=2)
        a, b = p.cache.open_token_stream(9000, 500, 20), p.cache.open_token_stream(9000)
        B = p.cache.token_batch
        x = {n: (p.rows(n, 2), p.rows(n, 2), p.rows(n, 8)) for n in (6000, 300, 9, 2)}
        outs = {n: tuple(torch.empty_like(t) for t in v) for n, v in x.items()}
        batches = {6000: B([a, b], [5000, 1000]), 300: B([b], [300]), 9: B([a, b], [5, 4]), 2: B([a, b], [1, 1])}
        scratch = p.cache.scratch_info()
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        for n, batch in batches.items():
            k, v, q = x[n]
            for layer in range(2):
                p.cache.append_tokens(batch, k, v, layer=layer)
                p.cache.attend_tokens(batch, q, layer=layer, window=400, sinks=20, out=outs[n][2])
                p.cache.read_tokens(batch, layer=layer, k_out=outs[n][0], v_out=outs[n][1])
            if n == 9:
                p.cache.drop_tokens(batch)
            if n == 2:
                p.cache.rollback_last_frame(b)
            p.cache.evict_window(a)
        p.cache.reset_stream(b)
        torch.cuda.synchronize()
        assert p.cache.scratch_info() == scratch
        after = torch.cuda.mem_get_info()[0]
        p.cache.close()
    assert after == free


def poison(cache):
    """Every free page's rows, on every layer, become NaN and infinities; the free stack stays."""
    n = cache.free_pages() * cache.page_size
    sid = cache.open_token_stream(n)
    batch = cache.token_batch([sid], [n])
    bad = torch.full((n, cache.heads, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    bad[::3] = float("inf")
    for layer in range(cache.layers):
        cache.append_tokens(batch, bad, bad, layer=layer)
    cache.drop_tokens(batch)                     # (closing alone would turn the free stack over)
    cache.close_stream(sid)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 192])
def test_a_served_run_on_used_pages(page, fp8):
    """Steps of three streams on two layers where every free page holds values that are not
    finite, again before each step: appends over page ends, drops, rollbacks, evictions."""
    p = Pool(4000 // page, page, 2, fp8, layers=2, seed=page)
    poison(p.cache)
    W, K = 70, 21
    a, b, c = p.open(), p.open(window=W, sinks=K), p.open(window=W)
    sids = [a, b, c]
    for step, n in enumerate([(1, 130, 300), (64, 1, 1), (5, 7, 3), (1, 1, 1), (200, 90, 1), (1, 1, 1), (2, 3, 260), (1, 1, 1)]):
        poison(p.cache)
        batch = p.append(sids, n)
        for layer in range(2):
            p.check_attend(sids, n, 2, W, 0, layer=layer, batch=batch)
            p.check_attend([a, b], n[:2], 4, W, K, layer=layer)
            p.check_attend([a], n[:1], 1, layer=layer)
        if step % 3 == 2:
            p.drop(sids, [min(2, x) for x in n])
            p.check_attend([a], [1], 2, layer=1)
        if step % 3 == 1:
            p.cache.rollback_last_frame(a)
            p.ora.rollback(a)
            for layer in p.kv[a]:
                layer[:] = [x[:len(x) - n[0]] for x in layer]
        for s in (b, c):
            p.cache.evict_window(s)
            p.ora.evict(s)
        p.check_state(sids)
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_frames_on_pages_that_a_token_stream_used(fp8):
    """A frame stream and a chunked one give the same bits on pages that a token stream left
    values in that are not finite."""
    from paged_kv_cache_build_gb300 import PagedKVCache, chunked_stream_cfg, frame_stream_cfg
    g = torch.Generator(device="cuda").manual_seed(8)
    frames = [[torch.randn((22, 4, 64), generator=g, device="cuda").bfloat16() for _ in range(3)] for _ in range(9)]
    results = []
    for used in (False, True):
        cache = PagedKVCache(64, 16, 4, layers=2, fp8=fp8)
        if used:
            poison(cache)
        f, c = cache.open_stream(frame_stream_cfg(2, 4, 16, 6)), cache.open_stream(chunked_stream_cfg(3, 2, 22))
        outs = []
        for i, (q, k, v) in enumerate(frames):
            for layer in range(2):
                cache.append_frame(f, k, v, layer=layer)
                outs.append(cache.attend(q, f, layer=layer))
                cache.append_frame(c, k, v, layer=layer)
                whole = torch.cat([x[0] for x in frames[i // 3 * 3:i + 1]])
                outs.append(cache.attend_chunked(whole, c, layer=layer))
            if i % 3 == 1:
                cache.rollback_last_frame(f)
            else:
                cache.evict_window(f)
            if i % 3 == 2:
                cache.evict_window(c)
            if used:
                poison(cache)
        results.append(torch.cat(outs))
        cache.sync()
        cache.close()
    assert torch.isfinite(results[1]).all()
    assert torch.equal(results[0], results[1])


@pytest.mark.parametrize("new", [1, 5, 200])
def test_two_handles_on_two_streams(new):
    """Calls of two handles that run at the same time: each one's split results are its own."""
    pools = [Pool(400, 16, 2, bool(i), seed=i) for i in range(2)]
    work = []
    for p in pools:
        sids = [p.open(), p.open()]
        p.append(sids, [2500 + new, 900 + new])
        batch = p.cache.token_batch(sids, [new, new])
        q = p.rows(2 * new, 4)
        work.append((p, batch, q, p.cache.attend_tokens(batch, q), [torch.empty_like(q) for _ in range(30)]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pools]
    for i in range(30):
        for s, (p, batch, q, _, outs) in zip(streams, work):
            p.cache.attend_tokens(batch, q, out=outs[i], stream=s)
    torch.cuda.synchronize()
    for p, _, _, want, outs in work:
        assert all(torch.equal(x, want) for x in outs)
        p.cache.sync()
        p.cache.close()
