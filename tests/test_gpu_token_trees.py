"""Trees of drafted tokens on token streams against the fp64 oracle (needs a GB300): rotary
appends, tree attention, and the drafts that are kept.

Tolerances. Tree attention makes the roundings of pkv_attend_tokens, and its outputs are held to
the same bound (test_gpu_tokens). A rotated value y = x_a cos - x_b sin stored in bf16 is rounded once,
half a step (2^-8 |y|), and before that off by fp32's cosine and sine (2^-22, angles cut to
2^-32 of a turn and rounded once among it) and three roundings: 2^-21 (|x_a| + |x_b|). E4M3 rows are held to
the codes of the exact values, or of values next to them that lie on the other side of a border: a
frequency is kept to 1.1 x 2^-64 of a turn (two roundings to half of that), so that an angle is off by
position x 1.1 x 2^-64 x 2 pi < position x 2^-61, and doubles add a few 2^-53:
(position x 2^-61 + 2^-48) (|x_a| + |x_b|)."""

import numpy as np
import pytest
import torch

from oracle.fp8 import e4m3_decode, e4m3_encode, row_exponent
from oracle.tokens import rotate_fp64, tree_attend_fp64

from .test_gpu_tokens import SCALE, Pool, _built, bits, f64, stored   # noqa: F401 (_built: a fixture)

pytestmark = pytest.mark.gpu

FP8 = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def stored64(y):
    """What E4M3 pages return for rows of doubles."""
    e = np.vectorize(row_exponent, otypes=[np.float64])(np.abs(y).max(axis=-1))[..., None] if y.size else y[..., :1]
    return e4m3_decode(e4m3_encode(y * np.exp2(-e))) * np.exp2(e)


def tree_tolerance(q, k, v, ref, parents, window, sinks, sm_scale):
    a = tree_attend_fp64(q, k, np.abs(v), parents, window, sinks, sm_scale)
    group = q.shape[1] // k.shape[1]
    s = 0.0
    for g in range(q.shape[1]):
        s = max(s, (np.abs(q[:, g]) @ np.abs(k[:, g // group]).T).max() * sm_scale)
    ds = 70 * 2.0 ** -24 * s
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * ds + k.shape[0] * 2.0 ** -24 + 2.0 ** -20) * a


def random_parents(rng, n):
    """Wide ones, long branches, several roots."""
    return [int(rng.integers(-1, i)) if rng.random() < 0.6 else i - 1 for i in range(n)]


def check_tree(p, sids, trees, group, window=0, sinks=0, layer=0, sm_scale=0.0):
    counts = [len(t) for t in trees]
    batch = p.cache.token_batch(sids, counts)
    q = p.rows(batch.rows, p.heads * group)
    parents = ints([x for t in trees for x in t])
    kw = dict(layer=layer, window=window, sinks=sinks, sm_scale=sm_scale)
    room = torch.full((batch.rows + 3, p.heads * group, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    out = p.cache.attend_tree(batch, q, parents, out=room[:batch.rows], **kw)
    again = p.cache.attend_tree(batch, q, parents, **kw)
    p.cache.sync()
    assert torch.equal(out, again) and (room[batch.rows:] == 7.0).all()
    got, qq, at = f64(out), f64(q), 0
    assert np.isfinite(got).all()
    scale = sm_scale if sm_scale > 0 else SCALE
    for sid, t in zip(sids, trees):
        if t:
            k, v = p.kv[sid][layer]
            x = qq[at:at + len(t)]
            ref = tree_attend_fp64(x, k, v, t, window, sinks, scale)
            err = np.abs(got[at:at + len(t)] - ref)
            tol = tree_tolerance(x, k, v, ref, t, window, sinks, scale)
            assert (err <= tol).all(), f"stream {sid}: worst {(err / tol).max():.2f} of the tolerance"
        at += len(t)
    return q, out


# (heads, group, page, past, nodes): both kernels and their row blocks, tile and page edges
TREES = [
    (1, 1, 16, [0], [1]),
    (2, 1, 16, [0, 15, 16, 17], [2, 1, 3, 0]),
    (2, 4, 64, [62, 63, 64, 65], [2, 2, 2, 2]),
    (2, 4, 64, [127, 128, 5], [4, 5, 6]),
    (3, 5, 32, [700, 3], [3, 4]),
    (16, 1, 256, [776], [16]),
    (2, 8, 16, [1000, 37], [3, 2]),
    (2, 1, 16, [333, 60], [17, 24]),
    (2, 1, 64, [3000], [33]),
    (4, 3, 16, [100, 0, 37], [21, 7, 9]),
    (2, 2, 16, [0, 60], [64, 65]),
    (1, 4, 32, [1000, 0, 5], [64, 2, 33]),
    (2, 1, 128, [63, 64, 1], [130, 128, 200]),
    (1, 8, 256, [2500], [64]),
    (2, 5, 64, [0, 191], [256, 255]),
    (1, 16, 16, [77], [256]),
    (1, 128, 64, [70], [9]),
]


@FP8
@pytest.mark.parametrize("shape", TREES, ids=str)
def test_tree_attention_matches_the_oracle(shape, fp8):
    heads, group, page, past, nodes = shape
    rng = np.random.default_rng(len(past) * 1000 + nodes[0])
    p = Pool(sum(-(-(a + b) // page) for a, b in zip(past, nodes)) + 2, page, heads, fp8)
    sids = [p.open(a + b) for a, b in zip(past, nodes)]
    p.append(sids, past)
    p.append(sids, nodes)
    check_tree(p, sids, [random_parents(rng, n) for n in nodes], group)
    # only roots, and one branch
    check_tree(p, sids, [[-1] * n for n in nodes], group, sm_scale=0.3)
    check_tree(p, sids, [list(range(-1, n - 1)) for n in nodes], group)
    p.cache.close()


@FP8
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (3, 600), (63, 1), (64, 0), (65, 64), (100, 65), (300, 200),
                                          (5000, 7), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_trees_under_a_window(window, sinks, fp8):
    """Windows and sinks go by depth: branches of a tree see back equally far."""
    rng = np.random.default_rng(window)
    p = Pool(300, 16 if window % 2 else 64, 2, fp8, seed=window % 1000)
    past = [0, 500, 64, 1300]
    for nodes, group in (([3, 5, 1, 7], 2), ([40, 1, 30, 64], 1), ([200, 130, 5, 90], 3)):
        sids = [p.open(2000) for _ in past]
        p.append(sids, past)
        p.append(sids, nodes)
        check_tree(p, sids, [random_parents(rng, n) for n in nodes], group, window, sinks)
        for s in sids:
            p.cache.close_stream(s)
            p.ora.release(s)
    p.cache.close()


@FP8
def test_one_branch_is_a_causal_draft(fp8):
    """The same rows as a chain and as a draft of attend_tokens: within twice the tolerance of
    either, 2^-8 (|out| + A), A below the largest value."""
    p = Pool(100, 64, 2, fp8)
    for n, group in ((1, 1), (5, 4), (24, 1), (90, 3)):
        sid = p.open()
        p.append([sid], [700])
        batch = p.append([sid], [n])
        q = p.rows(n, 2 * group)
        a = p.cache.attend_tokens(batch, q)
        b = p.cache.attend_tree(batch, q, ints(range(-1, n - 1)))
        assert (a.float() - b.float()).abs().max() <= 2 * 2.0 ** -8 * 12
        p.cache.close_stream(sid)
    p.cache.close()


@FP8
@pytest.mark.parametrize("n,group", [(6, 1), (6, 4), (100, 3)])
def test_parents_out_of_order(n, group, fp8):
    """A parent that is no earlier node is taken for none, and noted; other streams and rows
    are as they should be."""
    from paged_kv_cache_build_gb300 import PkvError
    p = Pool(60, 16, 2, fp8)
    sids = [p.open(), p.open()]
    p.append(sids, [90, 200])
    p.append(sids, [n, n])
    bad = [-1, 0, 1, 3, 2 ** 31 - 1, -2 ** 31] + [0] * (n - 6)
    good = [-1, 0, 1, -1, -1, -1] + [0] * (n - 6)
    batch = p.cache.token_batch(sids, [n, n])
    q = p.rows(2 * n, 2 * group)
    want = p.cache.attend_tree(batch, q, ints(good + good))
    p.cache.sync()
    got = p.cache.attend_tree(batch, q, ints(bad + good))
    with pytest.raises(PkvError) as e:
        p.cache.sync()
    assert e.value.code == "DEVICE"
    assert torch.equal(got, want)
    p.cache.close()


@FP8
def test_an_evicted_streams_tree_reads_no_freed_page(fp8):
    """Under a window, with pages given back that another stream has filled with NaN."""
    p = Pool(14, 16, 2, fp8)
    a = p.open(400, window=20, sinks=3)
    p.append([a], [150])
    p.append([a], [1])
    p.cache.evict_window(a)
    p.ora.evict(a)
    b = p.cache.open_token_stream(100)
    if not fp8:                                  # an E4M3 row of NaN has no exponent
        x = torch.full((90, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        p.cache.append_tokens(p.cache.token_batch([b], [90]), x, x)
        p.ora.free = p.ora.free[:-6]
    for n, group in ((7, 1), (9, 2), (20, 7)):
        p.append([a], [n])
        check_tree(p, [a], [random_parents(np.random.default_rng(n), n)], group, 20, 3)
        check_tree(p, [a], [random_parents(np.random.default_rng(n), n)], group, 5, 1)
        p.drop([a], [n])
    p.cache.close()


# ------------------------------------------------------------------ rotary
def rotation(distance, axes, seed=0):
    rng = np.random.default_rng(seed)
    freq = 10000.0 ** (-np.arange(32) / 32.0)
    axis = np.sort(rng.integers(0, axes, 32))
    return freq, axis


def check_rotary(p, sids, counts, positions, freq, axis, distance, group, layer=0, k=None, v=None, q=None):
    from paged_kv_cache_build_gb300 import Rotary
    batch = p.cache.token_batch(sids, counts)
    if layer == 0:
        p.ora.append(sids, counts)
    k = p.rows(batch.rows, p.heads, 2.0) if k is None else k
    v = p.rows(batch.rows, p.heads) if v is None else v
    q = p.rows(batch.rows, p.heads * group) if q is None and group else q
    rot = Rotary(freq, axis, distance, axes=positions.shape[1])
    out = p.cache.append_tokens_rotary(batch, k, v, ints(positions), rot, q=q, layer=layer)
    kk, vv = p.cache.read_tokens(batch, layer=layer)
    p.cache.sync()
    np.testing.assert_array_equal(f64(vv), stored(v, p.fp8))
    first = np.array([i // distance * 2 * distance + i % distance for i in range(32)])
    for x, y in ((q, out), (k, kk)):
        if x is None:
            assert y is None
            continue
        x64 = f64(x)
        want = rotate_fp64(x64, positions, freq, axis, distance)
        size = np.zeros_like(x64)
        size[..., first] = size[..., first + distance] = np.abs(x64[..., first]) + np.abs(x64[..., first + distance])
        if x is k and p.fp8:
            got, near = f64(y), size * (np.abs(positions).max() * 2.0 ** -61 + 2.0 ** -48)
            other = (got != stored64(want)) & (got != stored64(want - near)) & (got != stored64(want + near))
            assert not other.any(), (got[other], want[other])
            continue
        assert (np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * size).all()
    at = 0
    for sid, n in zip(sids, counts):
        for i, x in enumerate((kk, vv)):
            p.kv[sid][layer][i] = np.concatenate([p.kv[sid][layer][i], f64(x[at:at + n])])
        at += n
    return batch, k, v, q, out


@FP8
@pytest.mark.parametrize("distance", [1, 2, 4, 8, 16, 32])
@pytest.mark.parametrize("heads,group,page,counts", [(1, 1, 16, [1]), (2, 4, 64, [5, 0, 70]), (3, 0, 32, [33, 1]),
                                                     (4, 2, 256, [300, 7])], ids=str)
def test_rotary_append(heads, group, page, counts, distance, fp8):
    rng = np.random.default_rng(distance)
    axes = 1 + distance % 4
    freq, axis = rotation(distance, axes, distance)
    p = Pool(40, page, heads, fp8, layers=2)
    sids = [p.open() for _ in counts]
    p.append(sids, [9] * len(counts))
    n = sum(counts)
    positions = rng.integers(-50, 5000, (n, axes))
    for layer in range(2):
        check_rotary(p, sids, counts, positions, freq, axis, distance, group, layer)
    p.check_state(sids)
    # the next rows, and reading across both appends
    check_rotary(p, sids, [2] * len(counts), rng.integers(0, 9, (2 * len(counts), axes)), freq, axis, distance, group)
    p.check_state(sids)
    for sid, c in zip(sids, counts):
        k, v = p.cache.read_tokens(p.cache.token_batch([sid], [9 + c + 2]), [0])
        np.testing.assert_array_equal(f64(k), p.kv[sid][0][0])
        np.testing.assert_array_equal(f64(v), p.kv[sid][0][1])
    p.cache.close()


@FP8
def test_rotary_of_many_rows(fp8):
    """Thousands of rows of several streams, three axes, pages that were used before."""
    rng = np.random.default_rng(0)
    freq, axis = rotation(32, 3)
    p = Pool(90, 64, 3, fp8)
    counts = [1800, 0, 7, 1501, 333]
    for turn in range(2):
        sids = [p.open() for _ in counts]
        check_rotary(p, sids, counts, rng.integers(0, 100000, (sum(counts), 3)), freq, axis, 32, 2)
        p.check_state(sids)
        for s in sids:
            p.cache.close_stream(s)
            p.ora.release(s)
    p.cache.close()


@FP8
def test_rotary_far_positions_and_odd_frequencies(fp8):
    """The largest 32-bit positions, frequencies of whole turns, negative, tiny and large."""
    freq = np.array([1.0, -1.0, 2 * np.pi, np.pi, 0.0, 1e-30, 2.0 ** 20, -2.0 ** 20] + list(1e6 ** (-np.arange(24) / 24)))
    axis = np.arange(32) % 2
    far = [0, 1, -1, 2 ** 24 + 1, 1234567, -7654321, 2 ** 31 - 1, -2 ** 31]
    positions = np.array([[a, b] for a in far for b in far])
    p = Pool(20, 16, 2, fp8)
    sid = p.open()
    check_rotary(p, [sid], [len(positions)], positions, freq, axis, 32, 2)
    check_rotary(p, [sid], [len(positions)], positions, freq, axis, 1, 1)
    p.cache.close()


@FP8
@pytest.mark.parametrize("zero", ["position", "frequency"])
def test_rotary_by_nothing_is_an_append(zero, fp8):
    """Angles of 0: the same bits as append_tokens stores, ties between two codes among them."""
    from paged_kv_cache_build_gb300 import Rotary
    p = Pool(60, 16, 2, fp8)
    a, b = p.open(), p.open()
    g = torch.Generator(device="cuda").manual_seed(4)
    # values of few bits, so that many lie midway between two codes
    k = (torch.randint(-64, 65, (200, 2, 64), generator=g, device="cuda") / 8).bfloat16()
    v, q = p.rows(200, 2), p.rows(200, 4)
    positions = torch.zeros((200, 2), dtype=torch.int32, device="cuda")
    freq = [1.0] * 32
    if zero == "frequency":
        positions, freq = positions + 77, [0.0] * 32
    out = p.cache.append_tokens_rotary(p.cache.token_batch([a], [200]), k, v, positions,
                                       Rotary(freq, [0] * 16 + [1] * 16), q=q)
    p.cache.append_tokens(p.cache.token_batch([b], [200]), k, v)
    assert torch.equal(out, q)
    for x, y in zip(*(p.cache.read_tokens(p.cache.token_batch([s], [200])) for s in (a, b))):
        assert torch.equal(x, y)
    p.cache.close()


@FP8
def test_rotary_rows_next_to_the_border_of_two_codes(fp8):
    """Pairs turned by a quarter less or more than nothing: values that end within 2^-30 .. 2^-23 of a
    border between two codes, or two exponents, on either side."""
    freq = np.array([2.0 ** -(24 + i % 8) for i in range(32)])
    p = Pool(60, 16, 1, fp8)
    sid = p.open()
    n = 300
    rng = np.random.default_rng(3)
    # codes' borders: odd numbers of 5 bits
    x = (2 * rng.integers(8, 16, (n, 1, 64)) + 1) * 2.0 ** rng.integers(-3, 2, (n, 1, 1)) * rng.choice([-1, 1], (n, 1, 64))
    x[:, :, 5] = 448.0 * rng.choice([-1, 1], (n, 1))
    positions = rng.choice([-3, -1, 1, 2, 100], (n, 1))
    k = torch.tensor(x, dtype=torch.float32, device="cuda").bfloat16()
    check_rotary(p, [sid], [n], positions, freq, np.zeros(32, dtype=int), 32, 1, k=k)
    p.cache.close()


def test_rotary_of_strided_rows_and_in_place():
    """q, k and v as parts of one projection's rows; q turned into itself; nothing behind the
    rows is written; no q."""
    from paged_kv_cache_build_gb300 import Rotary
    heads, group, n = 4, 2, 77
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((n, (heads * group + 2 * heads) * 64), generator=g, device="cuda").bfloat16()
    q, k, v = (t.view(n, -1, 64) for t in x.split([heads * group * 64, heads * 64, heads * 64], 1))
    positions = ints(np.arange(n) * 3)
    rot = Rotary.sections([32])
    results = []
    for kind in ("strided", "contiguous", "in place", "without q"):
        from paged_kv_cache_build_gb300 import PagedKVCache
        cache = PagedKVCache(8, 64, heads)
        b = cache.token_batch([cache.open_token_stream(n)], [n])
        room = torch.full((n + 2, heads * group, 64), 7.0, device="cuda", dtype=torch.bfloat16)
        if kind == "strided":
            out = cache.append_tokens_rotary(b, k, v, positions, rot, q=q, q_out=room[:n])
            assert (room[n:] == 7.0).all()
        elif kind == "contiguous":
            out = cache.append_tokens_rotary(b, k.contiguous(), v.contiguous(), positions[:, None], rot,
                                             q=q.contiguous())
        elif kind == "in place":
            out = q.contiguous()
            assert cache.append_tokens_rotary(b, k, v, positions, rot, q=out, q_out=out) is out
        else:
            assert cache.append_tokens_rotary(b, k, v, positions, rot) is None
            out = results[0][0]
        results.append((out.clone(),) + cache.read_tokens(b))
        cache.sync()
        cache.close()
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))


# -------------------------------------------------------------------- keep
def keep(p, sids, counts, lists):
    """keep_tokens on the cache, the oracle's pages and the host's rows."""
    batch, accepted = p.cache.token_batch(sids, counts), p.cache.token_batch(sids, [len(x) for x in lists])
    p.cache.keep_tokens(batch, ints([i for x in lists for i in x]), accepted)
    p.ora.keep(sids, counts, [len(x) for x in lists])
    for sid, n, x in zip(sids, counts, lists):
        for layer in p.kv[sid]:
            for i in range(2):
                base = len(layer[i]) - n
                layer[i] = np.concatenate([layer[i][:base], layer[i][base + np.asarray(x, dtype=int)]])
    return accepted


def check_rows(p, sids):
    p.check_state(sids)
    for layer in range(p.layers):
        for sid in sids:
            n = len(p.kv[sid][layer][0])
            for got, want in zip(p.cache.read_tokens(p.cache.token_batch([sid], [n]), [0], layer=layer), p.kv[sid][layer]):
                np.testing.assert_array_equal(f64(got), want)


@FP8
@pytest.mark.parametrize("page,heads,layers", [(16, 1, 3), (64, 3, 2), (256, 2, 1)])
def test_kept_tokens(page, heads, layers, fp8):
    rng = np.random.default_rng(page)
    p = Pool(60, page, heads, fp8, layers=layers)
    sids = [p.open() for _ in range(4)]
    p.append(sids, [5, 100, 0, 63])
    for counts in ([16, 3, 1, 0], [70, 1, 33, 2], [256, 40, 300, 31], [1, 64, 65, 128]):
        p.append(sids, counts)
        lists = [sorted(rng.choice(n, rng.integers(0, n + 1), replace=False)) for n in counts]
        keep(p, sids, counts, lists)
        check_rows(p, sids)
        for s in sids:                           # nothing is pending
            assert p.ora.streams[s]["last"] is None or counts[sids.index(s)] == 0
    # all, none, the first, the last
    for lists in ([list(range(40))] * 4, [[]] * 4, [[0], [39], list(range(20, 40)), list(range(0, 40, 2))]):
        p.append(sids, [40] * 4)
        keep(p, sids, [40] * 4, lists)
        check_rows(p, sids)
    p.cache.sync()
    p.cache.close()


@FP8
def test_kept_numbers_out_of_order(fp8):
    """Numbers beyond the tree, negative, not rising: noted, and no other stream's rows move."""
    from paged_kv_cache_build_gb300 import PkvError
    for bad in ([0, 5, 8], [-1, 2, 3], [0, 0, 1], [1, 0, 2], [3, 3, 4], [2 ** 31 - 1, 4, 5], [-2 ** 31, 1, 2]):
        p = Pool(30, 16, 2, fp8, layers=2)
        sids = [p.open() for _ in range(3)]
        p.append(sids, [30, 30, 30])
        p.append(sids, [8, 8, 8])
        p.cache.sync()
        lists = [[1, 2, 7], bad, [0, 4]]
        batch, accepted = p.cache.token_batch(sids, [8] * 3), p.cache.token_batch(sids, [3, 3, 2])
        p.cache.keep_tokens(batch, ints([i for x in lists for i in x]), accepted)
        with pytest.raises(PkvError) as e:
            p.cache.sync()
        assert e.value.code == "DEVICE"
        for sid, x, length in ((sids[0], lists[0], 33), (sids[2], lists[2], 32), (sids[1], None, 33)):
            assert p.cache.token_info(sid)[0] == length
            for layer in range(2):
                rows = p.cache.read_tokens(p.cache.token_batch([sid], [length]), [0], layer=layer)
                for got, want in zip(rows, p.kv[sid][layer]):
                    np.testing.assert_array_equal(f64(got)[:30], want[:30])
                    if x is not None:
                        np.testing.assert_array_equal(f64(got)[30:], want[30 + np.asarray(x)])
        p.cache.close()


@FP8
def test_kept_tokens_under_a_window(fp8):
    """With pages evicted behind the window; refused where what stays, or what the stream's
    window sees then, is gone."""
    from paged_kv_cache_build_gb300 import PkvError
    p = Pool(60, 16, 2, fp8)
    sid = p.open(window=20, sinks=2)
    p.append([sid], [100])
    p.cache.evict_window(sid)
    p.ora.evict(sid)
    p.append([sid], [30])
    keep(p, [sid], [30], [[0, 3, 29]])
    p.check_state([sid])
    p.append([sid], [60])
    p.cache.evict_window(sid)
    p.ora.evict(sid)
    B = p.cache.token_batch
    for n, m in ((60, 1), (60, 50), (19, 0), (30, 11)):
        with pytest.raises(PkvError) as e:
            p.cache.keep_tokens(B([sid], [n]), ints(range(m)), B([sid], [m]))
        assert e.value.code == "STATE"
        p.check_state([sid])
    p.cache.close()


# ---------------------------------------------------------- used together
@FP8
def test_a_speculative_run(fp8):
    """Prompts with rotary positions, then steps of drafted trees (nodes' positions by depth), their
    attention on both layers, a path kept; a stream under a window, one closed in between. Each step's
    outputs, rows and pages follow the oracle."""
    from paged_kv_cache_build_gb300 import Rotary
    rng = np.random.default_rng(7)
    freq, axis = rotation(32, 3, 1)
    p = Pool(200, 16, 2, fp8, layers=2, seed=9)
    a, b, c = p.open(), p.open(window=50, sinks=4), p.open()
    sids = [a, b, c]
    prompt = [70, 130, 20]
    text = np.concatenate([np.arange(n) for n in prompt])[:, None].repeat(3, 1)
    for layer in range(2):
        check_rotary(p, sids, prompt, text, freq, axis, 32, 2, layer)
    for step in range(5):
        p.cache.evict_window(b)
        p.ora.evict(b)
        counts = [[16, 9, 5], [1, 30, 70], [3, 3, 3], [8, 1, 0], [60, 2, 33]][step]
        trees = [random_parents(rng, n) for n in counts]
        place = []
        for sid, t in zip(sids, trees):
            depth = []
            for x in t:
                depth.append(0 if x < 0 else depth[x] + 1)
            place += [len(p.kv[sid][0][0]) + d for d in depth]
        place = np.array(place)[:, None].repeat(3, 1)
        for layer in range(2):
            check_rotary(p, sids, counts, place, freq, axis, 32, 2, layer)
            check_tree(p, sids, trees, 2, 50, 4, layer=layer)
            check_tree(p, sids[:1], trees[:1], 3, layer=layer)
        p.check_state(sids)
        lists = []
        for t in trees:                          # a path from a root on
            path, at = [], -1
            for i, x in enumerate(t):
                if x == at and rng.random() < 0.7:
                    path.append(i)
                    at = i
            lists.append(path)
        keep(p, sids, counts, lists)
        p.check_state(sids)
        p.check_attend(sids, [min(1, n) for n in counts], 2, 50, 4, layer=1)
        if step == 2:
            p.cache.close_stream(c)
            p.ora.release(c)
            c = p.open()
            sids = [a, b, c]
            for layer in range(2):
                check_rotary(p, [c], [40], np.arange(40)[:, None].repeat(3, 1), freq, axis, 32, 2, layer)
    p.cache.sync()
    p.cache.close()


@FP8
@pytest.mark.parametrize("nodes", [[7, 1], [60, 100]])
def test_captured_steps_take_the_inputs_of_their_time(nodes, fp8):
    """Rotary append, tree attention, keep and read-back captured once: each replay takes that
    time's rows, positions, parents and kept numbers."""
    from paged_kv_cache_build_gb300 import Rotary
    rng = np.random.default_rng(1)
    p = Pool(100, 16, 2, fp8)
    sids = [p.open(), p.open()]
    p.append(sids, [300, 40])
    n, kept = sum(nodes), [3, 1]
    batch, accepted = p.cache.token_batch(sids, nodes), p.cache.token_batch(sids, kept)
    k, v, q = p.rows(n, 2), p.rows(n, 2), p.rows(n, 4)
    rot = Rotary.sections([10, 11, 11])
    positions, parents, numbers = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((n, 3), (n,), (4,)))

    def fresh():
        k.copy_(p.rows(n, 2))
        q.copy_(p.rows(n, 4))
        positions.copy_(ints(rng.integers(0, 999, (n, 3))))
        parents.copy_(ints([x for m in nodes for x in random_parents(rng, m)]))
        numbers.copy_(ints([i for m, c in zip(nodes, kept) for i in sorted(rng.choice(m, c, replace=False))]))

    def step():
        turned = p.cache.append_tokens_rotary(batch, k, v, positions, rot, q=q)
        out = p.cache.attend_tree(batch, turned, parents)
        p.cache.keep_tokens(batch, numbers, accepted)
        back = p.cache.read_tokens(accepted)
        p.cache.drop_tokens(accepted)
        return (turned, out) + back

    fresh()
    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        fresh()
        graph.replay()
        replayed = [t.clone() for t in got]
        for x, y in zip(step(), replayed):
            assert torch.equal(x, y)
        p.check_state(sids)
    p.cache.sync()
    p.cache.close()


def test_other_streams_and_many():
    """On a side stream, behind what that stream did; 256 streams in one batch."""
    from paged_kv_cache_build_gb300 import Rotary
    p = Pool(800, 16, 1, max_streams=256)
    sids = [p.open(200) for _ in range(256)]
    past = [(i * 37) % 23 for i in range(256)]
    p.append(sids, past)
    counts = [i % 5 for i in range(256)]
    p.append(sids, counts)
    rng = np.random.default_rng(0)
    check_tree(p, sids, [random_parents(rng, n) for n in counts], 4)
    keep(p, sids, counts, [sorted(rng.choice(n, (n + 1) // 2, replace=False)) for n in counts])
    check_rows(p, sids[:9])
    p.check_state(sids[::50])
    torch.cuda.synchronize()
    freq, axis = rotation(32, 1)
    side = torch.cuda.Stream()
    one = sids[7]
    batch = p.cache.token_batch([one], [6])
    n = len(p.kv[one][0][0])
    with torch.cuda.stream(side):
        k, v, q = p.rows(6, 1), p.rows(6, 1), p.rows(6, 4)
        positions, parents = ints(np.arange(6)), ints([-1, 0, 0, 1, 2, -1])
        turned = p.cache.append_tokens_rotary(batch, k, v, positions, Rotary(freq, axis), q=q)
        out = p.cache.attend_tree(batch, turned, parents)
        kk, vv = p.cache.read_tokens(batch)
    side.synchronize()
    keys = [np.concatenate([p.kv[one][0][i], f64(x)]) for i, x in enumerate((kk, vv))]
    assert len(keys[0]) == n + 6
    ref = tree_attend_fp64(f64(turned), *keys, [-1, 0, 0, 1, 2, -1], 0, 0, SCALE)
    assert (np.abs(f64(out) - ref) <= tree_tolerance(f64(turned), *keys, ref, [-1, 0, 0, 1, 2, -1], 0, 0, SCALE)).all()
    p.cache.close()


def test_offsets_beyond_32_bits():
    """Pages more than 2^32 bytes into the pool: rotary rows, a tree, and what is kept of it."""
    from paged_kv_cache_build_gb300 import PagedKVCache, Rotary
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
    k, v = (torch.randn((600, heads, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    cache.append_tokens_rotary(cache.token_batch([sid], [600]), k, v, ints(np.arange(600)), Rotary.sections([32]))
    b = cache.token_batch([sid], [600])
    kk, vv = cache.read_tokens(b)
    want = rotate_fp64(f64(k), np.arange(600)[:, None], 10000.0 ** (-np.arange(32) / 32.0), np.zeros(32, dtype=int), 32)
    assert (np.abs(f64(kk) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17).all() and torch.equal(vv, v)
    tree = cache.token_batch([sid], [9])
    q = torch.randn((9, heads, 64), generator=g, device="cuda").bfloat16()
    parents = [-1, 0, 0, 1, 1, 2, -1, 6, 7]
    out = cache.attend_tree(tree, q, ints(parents))
    ref = tree_attend_fp64(f64(q), f64(kk), f64(vv), parents, 0, 0, SCALE)
    assert (np.abs(f64(out) - ref) <= tree_tolerance(f64(q), f64(kk), f64(vv), ref, parents, 0, 0, SCALE)).all()
    kept = cache.token_batch([sid], [3])
    cache.keep_tokens(tree, ints([0, 2, 5]), kept)
    k2, v2 = cache.read_tokens(kept)
    rows = [591, 593, 596]
    assert torch.equal(k2, kk[rows]) and torch.equal(v2, vv[rows])
    cache.sync()
    cache.close()


@FP8
@pytest.mark.parametrize("heads,group,past,nodes", [
    (4, 4, [190 + 7 * i for i in range(40)], [9 + i % 3 for i in range(40)]),       # blocks of 128 rows in many CTAs
    (8, 2, [300] * 20 + [2500], [1 + i % 8 for i in range(20)] + [70]),             # few and many rows
    (8, 1, [1500] * 60 + [40], [1] * 60 + [200]),                                   # mostly single nodes
    (2, 4, [2000, 9, 640, 5000], [16, 64, 33, 3]),                                  # unequal, split
    (8, 3, [4100, 3000], [5, 15]),                                                  # 15 and 45 rows, alone on the card
    (1, 8, [9000], [200]),
], ids=["many", "mixed", "single nodes", "unequal", "alone", "large"])
def test_batches_of_every_shape(heads, group, past, nodes, fp8):
    """Batches that take each kernel, alone and together, with few and many CTAs."""
    rng = np.random.default_rng(sum(nodes))
    p = Pool(sum(-(-(a + b) // 64) for a, b in zip(past, nodes)) + 2, 64, heads, fp8, max_streams=64)
    sids = [p.open(a + b) for a, b in zip(past, nodes)]
    p.append(sids, past)
    p.append(sids, nodes)
    check_tree(p, sids, [random_parents(rng, n) for n in nodes], group)
    check_tree(p, sids, [random_parents(rng, n) for n in nodes], group, 300, 70)
    p.check_attend(sids, nodes, group)
    p.cache.close()


@FP8
def test_two_graphs_of_one_handle(fp8):
    """Two captured tree calls share the handle's partial results and counters: replayed in turn
    they give what the calls give."""
    rng = np.random.default_rng(2)
    p = Pool(300, 16, 2, fp8)
    sids = [p.open(), p.open()]
    p.append(sids, [3000, 900])
    calls = []
    p.append(sids, [40, 5])
    for sid, n, group in ((sids[0], 40, 4), (sids[1], 5, 2)):
        batch, q = p.cache.token_batch([sid], [n]), p.rows(n, 2 * group)
        calls.append((batch, q, ints(random_parents(rng, n))))
    eager = [p.cache.attend_tree(*c) for c in calls]
    graphs, outs = [], []
    for c in calls:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(p.cache.attend_tree(*c))
        graphs.append(g)
        torch.cuda.current_stream().wait_stream(s)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], eager[i])
    p.cache.sync()
    p.cache.close()
