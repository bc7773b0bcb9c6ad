"""Which kernel an attention call on token streams takes, without a GPU: the library's own host code,
linked with a CUDA runtime that keeps what was launched (recording_cudart.cpp)."""

import ctypes
import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

OK = 0
FEW = re.compile(r"token_few_kernelILi(\d)ELb([01])ELb([01])E")
TC = re.compile(r"token_tc_kernelILi(\d)ELb([01])ELi(\d)ELb([01])E")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from paged_kv_cache_build_gb300 import build
    from paged_kv_cache_build_gb300._lib import SIGNATURES
    build.build()
    so = str(tmp_path_factory.mktemp("host") / "recording.so")
    objs = [os.path.join(build.BUILD, os.path.basename(s)[:-3] + ".o") for s in build.sources()]
    include = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    # -Bsymbolic: not the runtime that torch has loaded
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", include, "-I", HERE,
                    os.path.join(HERE, "recording_cudart.cpp")] + objs + ["-o", so], check=True)
    L = ctypes.CDLL(so)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    L.recorded_kernel.restype = ctypes.c_char_p
    return L


def launches(lib, past, new, heads, group, fp8, tree=False, page=64):
    """What attending each stream's last new[i] of past[i] + new[i] tokens launches: ("few", 8-row
    groups a block), ("tc", row blocks of 128, lanes) or ("join",), in order."""
    ints = lambda x: (ctypes.c_int * len(x))(*x)  # noqa: E731
    h = ctypes.c_void_p()
    create = lib.pkv_create_fp8 if fp8 else lib.pkv_create_ex
    lengths = [a + b for a, b in zip(past, new)]
    pages = sum(-(-n // page) for n in lengths)
    assert create(pages, page, heads, 64, 1, len(past), ctypes.byref(h)) == OK
    mem = ctypes.create_string_buffer(64)
    at = (ctypes.addressof(mem) + 15) // 16 * 16
    sids = []
    for n in lengths:
        sid = ctypes.c_int()
        assert lib.pkv_stream_open_tokens(h, n, 0, 0, ctypes.byref(sid)) == OK
        sids.append(sid.value)
        assert lib.pkv_append_tokens(h, 1, ints([sid.value]), ints([0, n]), 0, at, at, 0, 0, None) == OK
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    lib.recorded_clear()
    if tree:
        r = lib.pkv_attend_tree(h, at, heads * group, 0, ints(off), ints(sids), len(sids), 0, at, at, 0, 0, 0.0, None)
    else:
        r = lib.pkv_attend_tokens(h, at, heads * group, 0, ints(off), ints(sids), len(sids), 0, at, 0, 0, 0.0, None)
    assert r == OK, lib.pkv_last_error(h)
    got = []
    for i in range(lib.recorded_launches()):
        name = lib.recorded_kernel(i).decode()
        few, tc = FEW.search(name), TC.search(name)
        assert few or tc or "token_combine_kernel" in name, name
        assert not (few or tc) or bool(int((few or tc).group(2))) == fp8
        assert not (few or tc) or bool(int((few or tc).groups()[-1])) == tree
        got.append(("few", int(few.group(1))) if few else ("tc", int(tc.group(1)), int(tc.group(3))) if tc else ("join",))
    assert lib.pkv_destroy(h) == OK
    return got


def kinds(got):
    return [x[0] for x in got if x[0] != "join"]


@pytest.mark.parametrize("past,new", [([4000] * 12, [1500] + [1] * 11), ([4000] * 16, list(range(4, 68, 4))),
                                      ([300, 300], [1, 200]), ([2000] * 101, [1500] + [1] * 100)], ids=str)
def test_few_rows_on_e4m3_pages_keep_f16_weights(lib, past, new):
    """Streams of few rows go through the kernel whose weights are f16, whatever else the batch holds:
    the matrix-unit kernel's are bf16, three bits less."""
    assert kinds(launches(lib, past, new, 8, 4, True)) == ["few", "tc"]


@pytest.mark.parametrize("rows", [[4, 8, 16, 24, 32, 40, 48, 64] * 2, [64, 1, 1, 1] * 10], ids=str)
def test_up_to_64_rows_on_e4m3_pages_keep_f16_weights(lib, rows):
    """So do those of up to 64 rows where such streams have 32 at most on average."""
    assert kinds(launches(lib, [2000] * len(rows), rows, 8, 1, True)) == ["few"]


# (past, KV heads, lanes): 30 new tokens of four query heads a KV head, few keys
SMALL_LANES = [([700] * 3, 2, 4), ([700, 3, 1300], 3, 4), ([90 + 3 * i for i in range(51)], 3, 2),
               ([40 * i for i in range(90)], 2, 2)]


# bf16 pages, 8 KV heads of four query heads, 30 new tokens: blocks of 128 rows
@pytest.mark.parametrize("tree", [False, True], ids=["tokens", "tree"])
@pytest.mark.parametrize("past,lanes", [([4001] * 16, 4), ([1000] * 16, 4), ([4000] * 18, 4), ([131000], 4),
                                        ([2000] * 32, 2), ([4000] * 12, 2), ([500 + 233 * i for i in range(16)], 2),
                                        ([300] * 64, 2)], ids=str)
def test_lanes_of_128_row_blocks(lib, past, lanes, tree):
    """One CTA of four lanes an SM where each SM has one CTA, two of two lanes where they come in waves or
    differ in length (16 even streams of 4031 tokens 30.7 us with four, 35.1 with two)."""
    got = launches(lib, past, [30] * len(past), 8, 4, False, tree)
    assert got[0] == ("tc", 1, lanes)
    assert kinds(got) == ["tc"]


@pytest.mark.parametrize("past,heads,lanes", SMALL_LANES, ids=["even", "ragged", "waves", "ragged waves"])
def test_lanes_of_the_gpu_tests_shapes(lib, past, heads, lanes):
    for tree in (False, True):
        assert launches(lib, past, [30] * len(past), heads, 4, False, tree, page=16)[0] == ("tc", 1, lanes)


# (streams, past, rows, fp8, few): measured, 8 KV heads of four query heads
LENGTHS = [(1, 1000, 64, False, True), (1, 4000, 64, False, True), (1, 8000, 48, False, True),
           (1, 32000, 64, False, False), (1, 131000, 40, False, False), (1, 131000, 64, False, False),
           (2, 16000, 64, False, False), (4, 500, 48, False, True), (4, 8000, 64, False, False),
           (1, 4000, 64, True, True), (1, 8000, 64, True, True), (1, 131000, 48, True, False),
           (1, 131000, 64, True, False), (2, 16000, 64, True, False), (4, 8000, 64, True, False)]


@pytest.mark.parametrize("tree", [False, True], ids=["tokens", "tree"])
@pytest.mark.parametrize("streams,past,rows,fp8,few", LENGTHS, ids=str)
def test_33_to_64_rows_by_length(lib, streams, past, rows, fp8, few, tree):
    """Blocks of 16 rows read such a stream's keys several times: the longer they are, the sooner the
    matrix-unit kernel ends (64 rows over 131000 tokens 56 us, 80 in blocks of 16; over 4000 12.9 and 11.1)."""
    got = launches(lib, [past] * streams, [rows // 4] * streams, 8, 4, fp8, tree)
    assert kinds(got) == ["few" if few else "tc"]


@pytest.mark.parametrize("past,rows,heads,few", [([2000] * 64, [64] * 4 + [1] * 60, 8, True),
                                                 ([200 + 40 * i for i in range(100)], [1 + i % 48 for i in range(100)], 1, True),
                                                 ([500] * 64, [64] * 16 + [8] * 48, 2, True),
                                                 ([4000] * 16, [48] * 16, 8, False), ([1000] * 128, [40] * 128, 1, False)],
                         ids=["a few of 64 among single tokens", "ragged", "short", "even", "many"])
def test_33_to_64_rows_in_batches(lib, past, rows, heads, few):
    """Measured, few rows / matrix units: 47 / 55, 17 / 19, 7 / 10, 51 / 31 us; the last 13 there."""
    assert kinds(launches(lib, past, rows, heads, 1, False)) == ["few" if few else "tc"]


@pytest.mark.parametrize("tree", [False, True], ids=["tokens", "tree"])
@pytest.mark.parametrize("past,new,lanes", [([4001] * 16, 30, 4), ([131000], 30, 4), ([1000] * 16, 30, 4),
                                            ([16000], 30, 4), ([131000], 16, 2), ([4000] * 16, 12, 2), ([2000] * 32, 30, 2),
                                            ([500 + 233 * i for i in range(16)], 30, 2), ([300] * 64, 30, 2)], ids=str)
def test_lanes_of_128_row_blocks_on_e4m3_pages(lib, past, new, lanes, tree):
    """Two lanes and four: 56 / 51 us for 16 even streams of 4031 tokens with 120 rows, 97 / 91 for one of
    131000, 86 / 91 where it has 64 rows."""
    got = launches(lib, past, [new] * len(past), 8, 4, True, tree)
    assert got[0] == ("tc", 1, lanes) and kinds(got) == ["tc"]


def test_ragged_trees_on_e4m3_pages_go_together(lib):
    """33 us in one launch, 41 in two."""
    past = [500 + 233 * i for i in range(16)]
    assert kinds(launches(lib, past, [1 + i * 11 // 15 for i in range(16)], 8, 4, True, True)) == ["tc"]


def test_a_few_long_trees_take_two_lanes(lib):
    """23 us, 24 with four."""
    assert launches(lib, [8000] * 4, [4, 16, 8, 32], 8, 4, False, True)[0] == ("tc", 1, 2)


# (tokens, KV heads, query heads, warps a quad of tokens on bf16 and on E4M3 pages)
SHARES = [(1, 16, 16, 48, 48), (64, 8, 32, 48, 48), (300, 8, 32, 15, 15), (1000, 8, 32, 4, 4), (1000, 2, 8, 4, 4),
          (3000, 16, 16, 4, 4), (3000, 1, 4, 1, 1), (10992, 2, 2, 1, 1), (10992, 16, 16, 4, 1), (13754, 16, 16, 4, 1),
          (40000, 8, 32, 1, 1), (300, 1, 0, 2, 2), (1000, 8, 0, 4, 4)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("tokens,heads,q_heads,bf16,e4m3", SHARES, ids=str)
def test_warps_of_a_rotary_append(lib, tokens, heads, q_heads, bf16, e4m3, fp8):
    """Shares of fewer than 12 planes, whose angles would take as long, only where an SM has few warps (1000
    tokens of 48 planes: 6.4 us in four shares, 14.1 in 48)."""
    from paged_kv_cache_build_gb300 import Rotary
    ints = lambda x: (ctypes.c_int * len(x))(*x)  # noqa: E731
    h, sid = ctypes.c_void_p(), ctypes.c_int()
    create = lib.pkv_create_fp8 if fp8 else lib.pkv_create_ex
    assert create(-(-tokens // 64), 64, heads, 64, 1, 1, ctypes.byref(h)) == OK
    assert lib.pkv_stream_open_tokens(h, tokens, 0, 0, ctypes.byref(sid)) == OK
    mem = ctypes.create_string_buffer(64)
    at = (ctypes.addressof(mem) + 15) // 16 * 16
    lib.recorded_clear()
    assert lib.pkv_append_tokens_rotary(h, 1, ints([sid.value]), ints([0, tokens]), 0, at, at, 0, 0, at, q_heads, 0, at, at,
                                        Rotary.sections([32]).cfg, None) == OK
    assert lib.recorded_launches() == 1 and b"rotary" in lib.recorded_kernel(0)
    quads = -(-(-(-tokens // 64) * 64) // 4)     # with the slots to be zeroed
    assert lib.recorded_grid(0) == -(-quads * (e4m3 if fp8 else bf16) // 4)
    assert lib.pkv_destroy(h) == OK
