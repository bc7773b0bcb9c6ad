"""Token streams' attention by the kernel that a call takes, against the fp64 oracle (needs a GB300).

Tolerance where weights are f16 (E4M3 pages, few rows): as in test_gpu_tokens, with 2^-11 of A, half
a step of f16, in place of bf16's 2^-8; n 2^-40 for weights below f16's range is less than the 2^-20
that stands there for the exponentials."""

import numpy as np
import pytest
import torch

from oracle.tokens import causal_attend_fp64

from .test_gpu_token_trees import check_rotary, check_tree, ints, random_parents, rotation
from .test_gpu_tokens import SCALE, Pool, _built, f64, stored, tolerance   # noqa: F401 (_built: a fixture)
from .test_token_kernels import SMALL_LANES

pytestmark = pytest.mark.gpu


def opposite_values(p, sid, n):
    """n tokens more whose values come in pairs that cancel but for the weights' difference: a weight's
    rounding shows in full where the output's own is small."""
    batch = p.cache.token_batch([sid], [n])
    p.ora.append([sid], [n])
    k = (p.rows(n, p.heads) * 0.5).bfloat16()
    v = (1 + torch.randint(0, 8, (n, p.heads, 64), generator=p.gen, device="cuda") / 8).bfloat16()
    v[1::2] = -v[0:n - 1:2]
    p.cache.append_tokens(batch, k, v)
    p.kv[sid][0] = [np.concatenate([old, stored(x, p.fp8)]) for old, x in zip(p.kv[sid][0], (k, v))]


@pytest.mark.parametrize("small,large", [([1] * 8, [200]), ([1, 8, 2, 4] * 3, [60, 300]), ([16, 1, 2, 12, 1, 3] * 12, [])],
                         ids=["single tokens beside a chunk", "drafts beside chunks", "up to 64 rows"])
def test_few_rows_on_e4m3_pages_have_f16_weights(small, large):
    heads, group = 2, 4
    p = Pool(200, 64, heads, True, max_streams=100)
    counts = small + large
    sids = [p.open() for _ in counts]
    for s, n in zip(sids, counts):
        opposite_values(p, s, n + n % 2 + (2 if n < 100 else 100))
    q, out = p.check_attend(sids, counts, group)
    qq, got, at = f64(q), f64(out), 0
    for sid, n in zip(sids, counts):
        if n in small:
            k, v = p.kv[sid][0]
            x = qq[at:at + n]
            ref = causal_attend_fp64(x, k, v, len(k) - n, 0, 0, SCALE)
            a = causal_attend_fp64(x, k, np.abs(v), len(k) - n, 0, 0, SCALE)
            tol = tolerance(x, k, v, ref, len(k) - n, 0, 0, SCALE) - (2.0 ** -8 - 2.0 ** -11) * a
            err = np.abs(got[at:at + n] - ref)
            assert (err <= tol).all(), f"stream {sid}: worst {(err / tol).max():.2f} of the tolerance"
        at += n
    p.cache.close()


@pytest.mark.parametrize("past,heads,lanes", SMALL_LANES, ids=["even", "ragged", "waves", "ragged waves"])
def test_both_numbers_of_lanes(past, heads, lanes):
    """Blocks of 128 rows on bf16 pages, in CTAs of two and of four lanes."""
    p = Pool(sum(-(-(n + 30) // 16) for n in past), 16, heads, max_streams=len(past))
    sids = [p.open(n + 30) for n in past]
    new = [30] * len(past)
    p.append(sids, past)
    p.append(sids, new)
    rng = np.random.default_rng(lanes)
    for window, sinks in ((0, 0), (50, 3)):
        p.check_attend(sids, new, 4, window, sinks)
        check_tree(p, sids, [random_parents(rng, 30) for _ in past], 4, window, sinks)
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("past,rows", [([40000], [16]), ([30000, 100], [12, 16])], ids=str)
def test_up_to_64_rows_over_long_histories(past, rows, fp8):
    p = Pool(1300, 64, 2, fp8)
    sids = [p.open() for _ in past]
    p.append(sids, past)
    p.append(sids, rows)
    p.check_attend(sids, rows, 4)
    check_tree(p, sids, [random_parents(np.random.default_rng(n), n) for n in rows], 4)
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("streams", [16, 17, 64, 256])
def test_rotary_of_batches_of_many_streams(streams, fp8):
    """A server's step: streams of 0 to 4 rows, empty ones first, between and last, so that a warp's four
    tokens are of several streams, some of them slots that a new page's end leaves to be zeroed."""
    rng = np.random.default_rng(streams)
    freq, axis = rotation(32, 3)
    p = Pool(2 * streams + 10, 16, 2, fp8, layers=2, max_streams=streams)
    sids = [p.open(100) for _ in range(streams)]
    p.append(sids, [(i * 7) % 19 for i in range(streams)])
    counts = [0] + [int(rng.integers(0, 5)) for _ in range(streams - 2)] + [0]
    positions = rng.integers(0, 3000, (sum(counts), 3))
    for layer in range(2):
        check_rotary(p, sids, counts, positions, freq, axis, 32, 4, layer)
    p.check_state(sids)
    for sid in sids[::7]:
        n = len(p.kv[sid][0][0])
        for layer in range(2):
            for x, want in zip(p.cache.read_tokens(p.cache.token_batch([sid], [n]), layer=layer), p.kv[sid][layer]):
                np.testing.assert_array_equal(f64(x), want)
    p.check_attend(sids, [min(1, n) for n in counts], 4)
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n,group", [(1, 1), (5, 4), (24, 1), (64, 1), (90, 3), (200, 2)])
def test_a_tree_without_branches_to_a_rounding(n, group, fp8):
    """A chain as a tree and as a draft of attend_tokens: each within the tolerance of every element, so
    that a tile that is left out (0.05 in most outputs, 0.003 of tolerance) shows."""
    p = Pool(100, 64, 2, fp8)
    sid = p.open()
    p.append([sid], [700])
    batch = p.append([sid], [n])
    q = p.rows(n, 2 * group)
    chain = p.cache.attend_tokens(batch, q)
    tree = p.cache.attend_tree(batch, q, ints(range(-1, n - 1)))
    p.cache.sync()
    k, v = p.kv[sid][0]
    ref = causal_attend_fp64(f64(q), k, v, 700, 0, 0, SCALE)
    tol = tolerance(f64(q), k, v, ref, 700, 0, 0, SCALE)
    assert (np.abs(f64(chain) - ref) <= tol).all() and (np.abs(f64(tree) - ref) <= tol).all()
    # (what this would miss: the last whole tile's share of the outputs)
    hole = np.ones(len(k), dtype=bool)
    hole[640:700 // 64 * 64 + 64] = False
    hole[700:] = True
    less = np.stack([causal_attend_fp64(f64(q)[i:i + 1], k[:700 + i + 1][hole[:700 + i + 1]], v[:700 + i + 1][hole[:700 + i + 1]],
                                        int(hole[:700 + i + 1].sum()) - 1, 0, 0, SCALE)[0] for i in range(n)])
    assert (np.abs(less - ref) > 2 * tol).mean() > 0.5
    p.cache.close()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("past,new", [([9000, 9000, 100, 5000], [1, 60, 300, 16]), ([7000], [30]), ([20000, 3], [16, 1])], ids=str)
def test_captured_batches_that_take_several_launches(past, new, fp8):
    """Two kernels in turn over the same partial results, and joins, replayed among eager calls on the
    capture's stream: the same bits each time."""
    p = Pool(800, 64, 2, fp8)
    sids = [p.open() for _ in past]
    p.append(sids, past)
    batch = p.append(sids, new)
    q, want = p.check_attend(sids, new, 4, batch=batch)
    stream, out = torch.cuda.Stream(), torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(3):
            p.cache.attend_tokens(batch, q, out=out)
    for _ in range(4):
        with torch.cuda.stream(stream):
            out.zero_()
            graph.replay()
            again = p.cache.attend_tokens(batch, q)
        stream.synchronize()
        assert torch.equal(out, want) and torch.equal(again, want)
    p.cache.sync()
    p.cache.close()
