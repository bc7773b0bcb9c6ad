"""Token streams against the fp64 oracle (needs a GB300): append, read-back, drop,
eviction, and causal attention with and without a window, on bf16 and E4M3 pages.

Tolerance of an attention output, per element, with A = the attention of |v| (the
same weights over the values' magnitudes), from the roundings the kernel makes:
  2^-8 |out|      out is rounded to bf16 (half a step)
  2^-8 A          the probabilities are rounded to bf16 for the second product
                  (E4M3 pages: to f16, 2^-11, with what lies below 2^-24 lost
                  against a largest of 2^15: n 2^-40, less than the bf16 bound)
  2 ds A          scores: 64 fp32 products and sums, |ds| <= 68 * 2^-24 * S, S the
                  largest sm_scale * sum |q||k|, plus two roundings of |s| log2(e)
  (n 2^-24 + 2^-20) A   fp32 sums over n keys; two approximate exponentials, 2^-22 each
"""

import numpy as np
import pytest
import torch

from oracle.fp8 import roundtrip_rows
from oracle.tokens import TokenStreamsOracle, causal_attend_fp64
from synth.inputs import bf16_bits_to_f64

pytestmark = pytest.mark.gpu

SCALE = 0.125


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_build_gb300 import build
    build.build()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def f64(t):
    return bf16_bits_to_f64(bits(t))


def stored(t, fp8):
    """What the cache returns for appended rows, as float64."""
    return bf16_bits_to_f64(roundtrip_rows(bits(t))) if fp8 else f64(t)


def tolerance(q, k, v, ref, pos0, window, sinks, sm_scale):
    a = causal_attend_fp64(q, k, np.abs(v), pos0, window, sinks, sm_scale)
    group = q.shape[1] // k.shape[1]
    s = 0.0
    for g in range(q.shape[1]):
        s = max(s, (np.abs(q[:, g]) @ np.abs(k[:, g // group]).T).max() * sm_scale)
    ds = 70 * 2.0 ** -24 * s
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * ds + k.shape[0] * 2.0 ** -24 + 2.0 ** -20) * a


class Pool:
    """A cache with the oracle's page state and every stream's rows on the host."""

    def __init__(self, pages, page, heads, fp8=False, layers=1, max_streams=64, seed=0):
        from paged_kv_cache_build_gb300 import PagedKVCache
        self.cache = PagedKVCache(pages, page, heads, layers=layers, max_streams=max_streams, fp8=fp8)
        self.ora = TokenStreamsOracle(pages, page)
        self.heads, self.fp8, self.layers = heads, fp8, layers
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.kv = {}

    def rows(self, n, heads, lift=0.0):
        x = torch.randn((n, heads, 64), generator=self.gen, device="cuda")
        x[..., ::16] += lift
        return x.bfloat16()

    def open(self, max_tokens=100000, window=0, sinks=0):
        sid = self.cache.open_token_stream(max_tokens, window, sinks)
        self.ora.open(sid, max_tokens, window, sinks)
        self.kv[sid] = [[np.zeros((0, self.heads, 64)) for _ in range(2)] for _ in range(self.layers)]
        return sid

    def append(self, sids, counts):
        batch = self.cache.token_batch(sids, counts)
        self.ora.append(sids, counts)
        for layer in range(self.layers):
            k, v = self.rows(batch.rows, self.heads, 2.0), self.rows(batch.rows, self.heads)
            self.cache.append_tokens(batch, k, v, layer=layer)
            at = 0
            for sid, n in zip(sids, counts):
                for i, x in enumerate((k, v)):
                    self.kv[sid][layer][i] = np.concatenate([self.kv[sid][layer][i],
                                                             stored(x[at:at + n], self.fp8)])
                at += n
        return batch

    def drop(self, sids, counts):
        self.cache.drop_tokens(self.cache.token_batch(sids, counts))
        self.ora.drop(sids, counts)
        for sid, n in zip(sids, counts):
            for layer in self.kv[sid]:
                for i in range(2):
                    layer[i] = layer[i][:len(layer[i]) - n]

    def check_state(self, sids):
        for sid in sids:
            free, idx, lens, words = self.cache.export_state(sid)
            assert free == self.ora.free
            assert (idx, lens) == self.ora.table(sid)
            assert words[0] == self.ora.streams[sid]["len"] == self.cache.token_info(sid)[0]

    def check_attend(self, sids, counts, group, window=0, sinks=0, layer=0, sm_scale=0.0, batch=None):
        batch = batch or self.cache.token_batch(sids, counts)
        q = self.rows(batch.rows, self.heads * group)
        out = self.cache.attend_tokens(batch, q, layer=layer, window=window, sinks=sinks, sm_scale=sm_scale)
        again = self.cache.attend_tokens(batch, q, layer=layer, window=window, sinks=sinks, sm_scale=sm_scale)
        self.cache.sync()
        assert torch.equal(out, again)
        got, qq, at = f64(out), f64(q), 0
        assert np.isfinite(got).all()
        scale = sm_scale if sm_scale > 0 else SCALE
        for sid, n in zip(sids, counts):
            if n:
                k, v = self.kv[sid][layer]
                pos0 = len(k) - n
                ref = causal_attend_fp64(qq[at:at + n], k, v, pos0, window, sinks, scale)
                err = np.abs(got[at:at + n] - ref)
                tol = tolerance(qq[at:at + n], k, v, ref, pos0, window, sinks, scale)
                assert (err <= tol).all(), f"stream {sid}: worst {(err / tol).max():.2f} of the tolerance"
            at += n
        return q, out


# (heads, group, page, past, new): lengths from one token on, odd ones, page and tile edges
SHAPES = [
    (1, 1, 16, [0], [1]),
    (2, 1, 16, [0, 15, 16, 17], [1, 1, 1, 1]),
    (2, 4, 64, [63, 64, 65, 127, 128], [1, 1, 1, 1, 1]),
    (3, 5, 32, [700, 3], [1, 1]),
    (16, 1, 256, [776], [1]),
    (4, 8, 256, [2000, 10, 300], [1, 1, 1]),
    (2, 16, 64, [1500], [1]),
    (2, 32, 16, [333], [1]),
    (1, 64, 64, [200], [1]),
    (2, 128, 64, [70], [1]),
    (4, 3, 16, [100, 0, 37], [5, 3, 1]),
    (2, 4, 128, [500, 1], [4, 8]),
    (2, 7, 64, [250], [9]),
    (2, 1, 64, [0], [33]),
    (2, 2, 16, [0, 60], [64, 65]),
    (2, 3, 256, [0, 130], [300, 129]),
    (1, 4, 32, [1000, 0, 5], [200, 2, 64]),
    (4, 1, 64, [0], [513]),
    (2, 1, 64, [3000], [257]),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention_matches_the_oracle(shape, fp8):
    heads, group, page, past, new = shape
    need = sum(-(-(a + b) // page) for a, b in zip(past, new))
    p = Pool(need + 2, page, heads, fp8)
    sids = [p.open(a + b) for a, b in zip(past, new)]
    p.append(sids, past)
    p.append(sids, new)
    p.check_attend(sids, new, group)
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (63, 1), (64, 0), (65, 64), (100, 65), (128, 4),
                                          (300, 200), (5000, 7)])
def test_window_and_sinks(window, sinks, fp8):
    p = Pool(200, 16 if window % 2 else 64, 2, fp8, seed=window)
    past, new = [0, 500, 64, 1300], [1, 1, 70, 30]
    sids = [p.open(2000) for _ in past]
    p.append(sids, past)
    p.append(sids, new)
    p.check_attend(sids, new, 2, window, sinks)
    p.check_attend(sids, [1, 1, 1, 1], 3, window, sinks)
    p.check_attend(sids, [1, 300, 130, 400], 1, window, sinks)
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_read_back(page, fp8):
    p = Pool(60, page, 3, fp8)
    sids = [p.open(1000) for _ in range(3)]
    p.append(sids, [5, 0, 2 * page])
    p.append(sids, [page, 1, 1])
    p.check_state(sids)
    lens = [page + 5, 1, 2 * page + 1]
    for pos0, counts in ((None, lens), ([3, 0, page - 1], [page, 1, 2]), ([0, 0, 0], [1, 0, 2 * page])):
        k, v = p.cache.read_tokens(p.cache.token_batch(sids, counts), pos0)
        at = 0
        for i, sid in enumerate(sids):
            a = pos0[i] if pos0 else lens[i] - counts[i]
            for x, want in ((k, p.kv[sid][0][0]), (v, p.kv[sid][0][1])):
                np.testing.assert_array_equal(f64(x[at:at + counts[i]]), want[a:a + counts[i]])
            at += counts[i]
    p.cache.sync()
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page,heads", [(16, 3), (256, 1), (64, 5)])
def test_many_rows_written_and_read(page, heads, fp8):
    """Thousands of rows in a call, ragged, from strided tensors, of every size that a
    bf16 row may have, over pages that were used before."""
    from paged_kv_cache_build_gb300 import PagedKVCache
    counts = [1800, 0, 7, 1501, 333]
    n = sum(counts)
    cache = PagedKVCache(sum(-(-c // page) for c in counts) + 1, page, heads, fp8=fp8)
    g = torch.Generator(device="cuda").manual_seed(page)
    both = torch.randn((n, 2 * heads + 1, 64), generator=g, device="cuda")
    both *= torch.exp2(torch.randint(-120, 119, (n, 2 * heads + 1, 1), generator=g, device="cuda").float())
    both *= torch.exp2(torch.randint(-12, 1, (n, 2 * heads + 1, 64), generator=g, device="cuda").float())
    both = both.bfloat16()
    both[5] = 0
    k, v = both[:, :heads], both[:, heads:2 * heads]
    for turn in range(2):
        sids = [cache.open_token_stream(c + 1) for c in counts]
        batch = cache.token_batch(sids, counts)
        cache.append_tokens(batch, k, v)
        # one row further: its page's other slots, zeros or old rows, are not read
        cache.append_tokens(cache.token_batch(sids[:1], [1]), k[:1], v[:1])
        kk, vv = cache.read_tokens(batch, [0] * len(counts))
        np.testing.assert_array_equal(f64(kk), stored(k, fp8))
        np.testing.assert_array_equal(f64(vv), stored(v, fp8))
        one, _ = cache.read_tokens(cache.token_batch(sids[:1], [1]))
        np.testing.assert_array_equal(f64(one), stored(k[:1], fp8))
        cache.sync()
        for s in sids:
            cache.close_stream(s)
        k, v = v, k
    cache.close()


def test_quantised_extremes_round_trip():
    """Rows of zeros, of one value, of the largest and smallest magnitudes, at the
    borders of the exponent: the stored codes are the oracle's."""
    p = Pool(4, 16, 2, True)
    sid = p.open()
    rows = [np.zeros(64), np.full(64, 448.0), np.full(64, 449.0), np.full(64, 447.0), np.full(64, 2.0 ** -126),
            np.full(64, 2.0 ** 120), np.concatenate([[2.0 ** 100], np.full(63, 1e-30)]),
            np.arange(64) - 32.0, np.full(64, 0.875), np.full(64, 0.8828125)]
    x = torch.tensor(np.stack([np.stack([r, -r]) for r in rows]), dtype=torch.float32).bfloat16().cuda()
    batch = p.cache.token_batch([sid], [len(rows)])
    p.cache.append_tokens(batch, x, x.flip(0).contiguous())
    k, v = p.cache.read_tokens(batch)
    np.testing.assert_array_equal(f64(k), stored(x, True))
    np.testing.assert_array_equal(f64(v), stored(x.flip(0), True))
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_rows_of_very_different_size(fp8):
    """Keys, values and queries whose rows differ by many powers of two, and scores
    so large that one key takes all: sums and references must hold them."""
    from paged_kv_cache_build_gb300 import PagedKVCache
    heads, group, n = 2, 2, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn((n, heads, 64), generator=g, device="cuda")
    v = torch.randn((n, heads, 64), generator=g, device="cuda")
    v *= torch.exp2(torch.randint(-40, 40, (n, heads, 1), generator=g, device="cuda").float())
    k *= torch.exp2(torch.randint(-20, 5, (n, heads, 1), generator=g, device="cuda").float())
    q = torch.randn((4, heads * group, 64), generator=g, device="cuda")
    q *= torch.exp2(torch.randint(-20, 5, (4, heads * group, 1), generator=g, device="cuda").float())
    k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
    cache = PagedKVCache(30, 16, heads, fp8=fp8)
    sid = cache.open_token_stream(n)
    cache.append_tokens(cache.token_batch([sid], [n]), k, v)
    out = cache.attend_tokens(cache.token_batch([sid], [4]), q)
    kk, vv, qq = stored(k, fp8), stored(v, fp8), f64(q)
    ref = causal_attend_fp64(qq, kk, vv, n - 4, 0, 0, SCALE)
    err = np.abs(f64(out) - ref)
    assert (err <= tolerance(qq, kk, vv, ref, n - 4, 0, 0, SCALE)).all()
    cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 5, 40, 130, 700])
def test_scores_that_grow(new, fp8):
    """Scores that rise by about one factor of two from key to key: every step moves
    the references of all rows, and what was summed before with them."""
    p = Pool(300, 16, 2, fp8, seed=new)
    sid, n = p.open(3000), 2000 + new
    g = torch.Generator(device="cuda").manual_seed(new)
    u = torch.where(torch.rand((1, 2, 64), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    k = (u * (torch.arange(n, device="cuda") / 100.0).view(-1, 1, 1)).bfloat16()
    v = torch.randn((n, 2, 64), generator=g, device="cuda").bfloat16()
    q = (u.repeat_interleave(2, 1) * 8 + torch.randn((new, 4, 64), generator=g, device="cuda")).bfloat16()
    p.cache.append_tokens(p.cache.token_batch([sid], [n]), k, v)
    out = p.cache.attend_tokens(p.cache.token_batch([sid], [new]), q)
    p.cache.sync()
    kk, vv, qq = stored(k, fp8), stored(v, fp8), f64(q)
    ref = causal_attend_fp64(qq, kk, vv, 2000, 0, 0, SCALE)
    err = np.abs(f64(out) - ref)
    assert (err <= tolerance(qq, kk, vv, ref, 2000, 0, 0, SCALE)).all()
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_a_served_run(fp8):
    """Prompts, single tokens, drafts accepted in part, eviction, a stream closed and
    its pages used again, over two layers: the pages follow the oracle, and every
    step's attention does."""
    p = Pool(120, 16, 2, fp8, layers=2, seed=5)
    W, K = 50, 5
    a, b, c = p.open(), p.open(window=W, sinks=K), p.open(window=W, sinks=0)
    sids = [a, b, c]
    p.append(sids, [70, 130, 20])
    for step in range(6):
        for s in (b, c):
            p.cache.evict_window(s)
            p.ora.evict(s)
        p.check_state(sids)
        n = [1, 1, 1] if step % 2 else [4, 7, 3]
        batch = p.append(sids, n)
        for layer in range(2):
            p.check_attend(sids, n, 2, W, 0, layer=layer, batch=batch)
            p.check_attend([a, b], n[:2], 1, W, K, layer=layer)
            p.check_attend([a], n[:1], 2, layer=layer)
        if step % 2 == 0:
            p.drop(sids, [2, 3, 0])
        p.check_state(sids)
    # a closed stream's pages are used again
    p.cache.close_stream(c)
    p.ora.release(c)
    assert p.cache.free_pages() == len(p.ora.free)
    d = p.open()
    assert d == c
    p.append([d], [90])
    p.check_state([a, b, d])
    p.check_attend([a, d], [3, 90], 1, layer=1)
    # rollback and reset
    p.append([a], [40])
    p.cache.rollback_last_frame(a)
    p.ora.rollback(a)
    for layer in p.kv[a]:
        for i in range(2):
            layer[i] = layer[i][:-40]
    p.check_state([a, b, d])
    p.check_attend([a], [2], 2)
    p.cache.reset_stream(a)
    p.ora.release(a)
    p.check_state([a, b, d])
    p.cache.sync()
    p.cache.close()


def test_strided_rows():
    """q, k and v as parts of one projection's rows; other rows stay untouched."""
    from paged_kv_cache_build_gb300 import PagedKVCache
    heads, group, n = 4, 2, 77
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((n, (heads * group + 2 * heads) * 64), generator=g, device="cuda").bfloat16()
    q, k, v = x.split([heads * group * 64, heads * 64, heads * 64], 1)
    q, k, v = q.view(n, -1, 64), k.view(n, -1, 64), v.view(n, -1, 64)
    outs = []
    for strided in (True, False):
        cache = PagedKVCache(8, 64, heads)
        sid = cache.open_token_stream(n)
        b = cache.token_batch([sid], [n])
        f = (lambda t: t) if strided else (lambda t: t.contiguous())
        cache.append_tokens(b, f(k), f(v))
        outs.append(cache.attend_tokens(b, f(q)))
        cache.close()
    assert torch.equal(outs[0], outs[1])


def test_batch_rows_are_those_of_single_calls():
    """A stream's rows in a batch agree with a call of its own within the rounding of
    the split, and nothing behind the batch's rows is written."""
    p = Pool(100, 64, 2)
    past, new = [400, 3, 0, 900], [2, 1, 0, 40]
    sids = [p.open() for _ in past]
    p.append(sids, past)
    p.append(sids, new)
    batch = p.cache.token_batch(sids, new)
    q = p.rows(batch.rows, 4)
    room = torch.full((batch.rows + 5, 4, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    out = p.cache.attend_tokens(batch, q, out=room[:batch.rows])
    assert (room[batch.rows:] == 7.0).all()
    at = 0
    for sid, n in zip(sids, new):
        if n:
            one = p.cache.attend_tokens(p.cache.token_batch([sid], [n]), q[at:at + n].contiguous())
            # both are within 2^-8 (|out| + A) of the exact value, and A <= max |v| < 6
            assert (one.float() - out[at:at + n].float()).abs().max() <= 2 * 2.0 ** -8 * 12
        at += n
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_graph_replays(fp8):
    """append, attention, read-back and drop captured once: each replay works on the
    inputs of its time, and the cache is as before it."""
    p = Pool(100, 16, 2, fp8)
    sids = [p.open(), p.open()]
    p.append(sids, [300, 40])
    batch = p.cache.token_batch(sids, [17, 1])
    k, v, q = p.rows(18, 2), p.rows(18, 2), p.rows(18, 4)

    def step():
        p.cache.append_tokens(batch, k, v)
        out = p.cache.attend_tokens(batch, q)
        back = p.cache.read_tokens(batch)
        p.cache.drop_tokens(batch)
        return (out,) + back

    eager = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(eager, got):
        assert torch.equal(x, y)
    k.copy_(p.rows(18, 2))
    q.copy_(p.rows(18, 4))
    graph.replay()
    replayed = [t.clone() for t in got]
    for x, y in zip(step(), replayed):
        assert torch.equal(x, y)
    p.check_state(sids)
    p.cache.sync()
    p.cache.close()


def test_offsets_beyond_32_bits():
    """Pages more than 2^32 bytes into the pool."""
    from paged_kv_cache_build_gb300 import PagedKVCache
    heads, page = 16, 256
    pages = (2 ** 32 + 2 ** 28) // (2 * heads * page * 128)
    cache = PagedKVCache(pages, page, heads)
    front = cache.open_token_stream(pages * page)
    n = (pages - 3) * page
    zeros = torch.zeros((n, heads, 64), dtype=torch.bfloat16, device="cuda")
    cache.append_tokens(cache.token_batch([front], [n]), zeros, zeros)
    del zeros
    sid = cache.open_token_stream(600)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.randn((600, heads, 64), generator=g, device="cuda").bfloat16() for _ in range(3))
    b = cache.token_batch([sid], [600])
    cache.append_tokens(b, k, v)
    back = cache.read_tokens(b)
    assert torch.equal(back[0], k) and torch.equal(back[1], v)
    out = cache.attend_tokens(cache.token_batch([sid], [5]), q[-5:].contiguous())
    kk, vv, qq = f64(k), f64(v), f64(q[-5:])
    ref = causal_attend_fp64(qq, kk, vv, 595, 0, 0, SCALE)
    assert (np.abs(f64(out) - ref) <= tolerance(qq, kk, vv, ref, 595, 0, 0, SCALE)).all()
    # the long stream's queries reach the far pages, too: keys of zeros give the mean of v = 0
    out = cache.attend_tokens(cache.token_batch([front], [1]), q[:1].contiguous())
    assert (out == 0).all()
    cache.close()


def test_frames_and_tokens_share_a_pool():
    """A frame stream's results are the same bits with and without token streams in
    its pool, and token streams refuse the frame calls (and the other way round)."""
    from paged_kv_cache_build_gb300 import PagedKVCache, PkvError, frame_stream_cfg
    g = torch.Generator(device="cuda").manual_seed(8)
    frames = [[torch.randn((22, 4, 64), generator=g, device="cuda").bfloat16() for _ in range(3)] for _ in range(8)]
    results = []
    for tokens in (False, True):
        cache = PagedKVCache(64, 16, 4)
        f = cache.open_stream(frame_stream_cfg(2, 4, 16, 6))
        t = cache.open_token_stream(500) if tokens else None
        outs = []
        for q, k, v in frames:
            cache.append_frame(f, k, v)
            if tokens:
                cache.append_tokens(cache.token_batch([t], [22]), k, v)
            outs.append(cache.attend(q, f))
            if tokens:
                cache.attend_tokens(cache.token_batch([t], [22]), q)
            cache.evict_window(f)
        results.append(torch.stack(outs))
        if tokens:
            for call in (lambda: cache.append_frame(t, k, v), lambda: cache.attend(q, t),
                         lambda: cache.attend_chunked(q, t), lambda: cache.attend_batched([q], [t]),
                         lambda: cache.attend_noalloc(q, t), lambda: cache.attend_sampled(q, t),
                         lambda: cache.attend_blocksparse(q, t, keep=1),
                         lambda: cache.stream_frames(t, *(x[None] for x in (q, k, v))),
                         lambda: cache.append_tokens(cache.token_batch([f], [22]), k, v),
                         lambda: cache.attend_tokens(cache.token_batch([f], [22]), q),
                         lambda: cache.token_info(f)):
                with pytest.raises(PkvError) as e:
                    call()
                assert e.value.code == "STATE"
        cache.sync()
        cache.close()
    assert torch.equal(results[0], results[1])


def test_refusals_change_nothing():
    from paged_kv_cache_build_gb300 import PkvError
    p = Pool(10, 16, 2, layers=2, max_streams=3)
    cache = p.cache
    a, b = p.open(100), p.open(100, window=10, sinks=2)
    p.append([a, b], [20, 60])
    cache.evict_window(b)
    p.ora.evict(b)
    x1, x2 = p.rows(1, 2), p.rows(2, 2)
    x200 = p.rows(200, 2)
    q1 = p.rows(1, 4)
    B = cache.token_batch

    def refused(code, call):
        with pytest.raises(PkvError) as e:
            call()
        assert e.value.code == code, e.value
        p.check_state([a, b])

    refused("INVALID", lambda: cache.open_token_stream(0))
    refused("INVALID", lambda: cache.open_token_stream(10, window=-1))
    refused("INVALID", lambda: cache.open_token_stream(10, window=0, sinks=2))
    refused("INVALID", lambda: cache.open_token_stream(10, window=3, sinks=-1))
    refused("INVALID", lambda: cache.append_tokens(B([a, a], [1, 1]), x2, x2))
    refused("INVALID", lambda: cache.append_tokens(B([a, 7], [1, 1]), x2, x2))
    refused("INVALID", lambda: cache.append_tokens(B([2], [1]), x1, x1))
    refused("INVALID", lambda: cache.append_tokens(B([a], [1]), x1, x1, layer=2))
    refused("INVALID", lambda: cache.append_tokens(B([a], [200]), x200, x200))
    refused("OOM", lambda: cache.append_tokens(B([a, b], [78, 40]), x200[:118], x200[:118]))
    refused("INVALID", lambda: cache.append_tokens(B([a], [5]), x200[:5], x200[:5], layer=1))
    refused("STATE", lambda: cache.append_tokens(B([b], [5]), x200[:5], x200[:5], layer=1))
    refused("INVALID", lambda: cache.drop_tokens(B([a], [21])))
    refused("STATE", lambda: cache.drop_tokens(B([b], [30])))
    refused("STATE", lambda: cache.rollback_last_frame(b))
    refused("STATE", lambda: cache.read_tokens(B([b], [10]), [20]))
    refused("INVALID", lambda: cache.read_tokens(B([a], [10]), [11]))
    refused("INVALID", lambda: cache.read_tokens(B([a], [1]), [-1]))
    refused("STATE", lambda: cache.attend_tokens(B([b], [1]), q1))
    refused("STATE", lambda: cache.attend_tokens(B([b], [1]), q1, window=40))
    refused("STATE", lambda: cache.attend_tokens(B([b], [1]), q1, window=10, sinks=17))
    refused("STATE", lambda: cache.attend_tokens(B([a], [21]), p.rows(21, 4)))
    refused("INVALID", lambda: cache.attend_tokens(B([a], [1]), q1, window=-1))
    refused("INVALID", lambda: cache.attend_tokens(B([a], [1]), q1, sinks=1))
    refused("INVALID", lambda: cache.attend_tokens(B([a], [1]), p.rows(1, 3)))
    refused("INVALID", lambda: cache.attend_tokens(B([], []), q1[:0]))
    for bad in (lambda: cache.append_tokens(B([a], [1]), x2, x1), lambda: cache.append_tokens(B([a], [1]), x1, x1.float()),
                lambda: cache.append_tokens(B([a], [1]), x1.cpu(), x1),
                lambda: cache.append_tokens(B([a], [2]), x1.expand(2, 2, 64), x2),
                lambda: cache.append_tokens(B([a], [2]), x2.transpose(0, 1), x2),
                lambda: cache.attend_tokens(B([a], [1]), q1, out=p.rows(2, 4)),
                lambda: cache.read_tokens(B([a], [1]), [0, 1])):
        with pytest.raises(ValueError):
            bad()
    p.check_state([a, b])
    # an unaligned base, a stride that is not whole vectors
    flat = torch.zeros(2 * 2 * 64 + 64, dtype=torch.bfloat16, device="cuda")
    refused("INVALID", lambda: cache.append_tokens(B([a], [1]), flat[1:129].view(1, 2, 64), x1))
    refused("INVALID", lambda: cache.append_tokens(B([a], [2]), flat.as_strided((2, 2, 64), (132, 64, 1)), x2))
    # nothing to do is no error
    empty = p.rows(0, 2)
    cache.append_tokens(B([a], [0]), empty, empty)
    cache.drop_tokens(B([a], [0]))
    assert cache.attend_tokens(B([a, b], [0, 0]), p.rows(0, 4)).shape == (0, 4, 64)
    p.check_attend([a], [1], 2)
    p.check_attend([b], [1], 2, 10, 2)
    p.cache.close()


def test_many_streams_in_one_batch():
    p = Pool(600, 16, 1, max_streams=256)
    sids = [p.open(200) for _ in range(256)]
    past = [(i * 37) % 23 for i in range(256)]
    p.append(sids, past)
    p.append(sids, [1] * 256)
    p.check_attend(sids, [1] * 256, 4)
    p.drop(sids, [1] * 256)
    p.check_state(sids[:3])
    p.cache.close()


def test_another_stream():
    """Calls on a side stream follow what that stream did before them."""
    p = Pool(40, 64, 2)
    sid = p.open()
    p.append([sid], [500])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    batch = p.cache.token_batch([sid], [3])
    with torch.cuda.stream(side):
        k, v, q = p.rows(3, 2), p.rows(3, 2), p.rows(3, 4)
        p.cache.append_tokens(batch, k, v)
        out = p.cache.attend_tokens(batch, q)
    side.synchronize()
    for i, x in enumerate((k, v)):
        p.kv[sid][0][i] = np.concatenate([p.kv[sid][0][i], f64(x)])
    kk, vv = p.kv[sid][0]
    ref = causal_attend_fp64(f64(q), kk, vv, 500, 0, 0, SCALE)
    assert (np.abs(f64(out) - ref) <= tolerance(f64(q), kk, vv, ref, 500, 0, 0, SCALE)).all()
    p.cache.close()


def test_no_token_call_allocates():
    """Token calls have partial results of their own: the scratch of the frame calls,
    which grows and moves, is not theirs."""
    for attempt in ("the kernels are loaded", "what is looked at"):
        p = Pool(300, 16, 2)
        before = p.cache.scratch_info()
        sid = p.open()
        p.append([sid], [4000])
        q = [p.rows(n, 2 * g) for n, g in ((1, 1), (9, 4), (300, 2))]
        batches = [p.cache.token_batch([sid], [len(x)]) for x in q]
        outs = [torch.empty_like(x) for x in q]
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        for x, b, o in zip(q, batches, outs):
            p.cache.attend_tokens(b, x, out=o)
        p.cache.drop_tokens(batches[2])
        torch.cuda.synchronize()
        after = torch.cuda.mem_get_info()[0]
        assert p.cache.scratch_info() == before
        p.cache.close()
    assert after == free


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 40, 300])
def test_large_values_behind_growing_scores(new, fp8):
    """Values near 2^95 and scores that end 2^80 above the first ones': no sum on the
    way may leave fp32."""
    p = Pool(100, 16, 1, fp8)
    sid, n = p.open(), 640 + new
    g = torch.Generator(device="cuda").manual_seed(11)
    k = torch.zeros((n, 1, 64), device="cuda")
    k[:, :, 0] = torch.arange(n, device="cuda").view(-1, 1) * (8.0 / n)
    v = torch.randn((n, 1, 64), generator=g, device="cuda") * 2.0 ** 93
    q = torch.zeros((new, 2, 64), device="cuda")
    q[:, :, 0] = 56.0                                  # scores up to 56, 80 in powers of two
    k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
    p.cache.append_tokens(p.cache.token_batch([sid], [n]), k, v)
    out = p.cache.attend_tokens(p.cache.token_batch([sid], [new]), q)
    p.cache.sync()
    kk, vv, qq = stored(k, fp8), stored(v, fp8), f64(q)
    ref = causal_attend_fp64(qq, kk, vv, 640, 0, 0, SCALE)
    assert (np.abs(f64(out) - ref) <= tolerance(qq, kk, vv, ref, 640, 0, 0, SCALE)).all()
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 20, 200])
def test_largest_window_sinks_and_a_scale(new, fp8):
    """Windows and sinks up to the largest int see every key; sm_scale is the caller's."""
    p = Pool(60, 32, 2, fp8)
    sid = p.open()
    p.append([sid], [900 + new])
    batch = p.cache.token_batch([sid], [new])
    q, every = p.check_attend([sid], [new], 3, sm_scale=0.3)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1), (7, 900 + new)):
        assert torch.equal(p.cache.attend_tokens(batch, q, window=window, sinks=sinks, sm_scale=0.3), every)
    for window, sinks in ((2 ** 31, 0), (2 ** 32 + 5, 0), (5, 2 ** 32)):
        with pytest.raises(ValueError):
            p.cache.attend_tokens(batch, q, window=window, sinks=sinks)
    with pytest.raises(ValueError):
        p.cache.read_tokens(batch, [2 ** 32])
    with pytest.raises(ValueError):
        p.cache.open_token_stream(2 ** 32 + 5)
    p.cache.sync()
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_drafts_on_either_side_of_the_row_blocks(fp8):
    """4 .. 68 query rows per KV head, alone and together, small and large on the whole."""
    p = Pool(400, 16, 2, fp8, max_streams=8)
    counts = [1, 2, 4, 5, 8, 9, 16, 17]
    sids = [p.open() for _ in counts]
    p.append(sids, [500 + 31 * n for n in counts])
    p.check_attend(sids, counts, 4)
    p.check_attend(sids[4:], counts[4:], 4)
    for sid, n in zip(sids, counts):
        p.check_attend([sid], [n], 4, 100, 5)
    p.cache.close()


def test_a_stream_shorter_than_its_sinks():
    """Sinks beyond a stream's largest length: nothing is ever evicted."""
    p = Pool(20, 16, 2)
    sid = p.cache.open_token_stream(90, window=5, sinks=100)
    batch = p.cache.token_batch([sid], [90])
    k, v, q = p.rows(90, 2), p.rows(90, 2), p.rows(90, 4)
    p.cache.append_tokens(batch, k, v)
    p.cache.evict_window(sid)
    assert p.cache.token_info(sid) == (90, 0, 0)
    out = p.cache.attend_tokens(batch, q, window=5, sinks=100)
    assert torch.equal(out, p.cache.attend_tokens(batch, q))
    p.cache.sync()
    p.cache.close()
