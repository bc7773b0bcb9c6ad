// Arguments and launchers of the token streams' kernels.
#pragma once

#include <cstddef>
#include <cstring>

#include "pkv_internal.cuh"
#include "pkv_token_plan.h"

namespace pkv {

constexpr int kMaxTokenBatch = 256;   // streams of one token call
// Kernels that single tokens go through exist for argument blocks of a few streams, too: a
// launch's arguments are copied (10 KB for 256 streams; a call takes 0.5 us less without).
constexpr int kSmallTokenBatch = 16;

// One stream of an append or a read: rows row0 .. row0 + n - 1 of the packed
// tensors are its positions pos0 .. pos0 + n - 1.
struct TokenRows {
  int32_t* pages;                   // the stream's page list
  int unit0;                        // first of the call's row numbers (an append numbers
                                    // the slots it zeroes behind the stream's rows, too)
  int row0, n;
  int pos0;
  int old_pages;                    // append: list entries before it
  int pop0;                         // append: pages that the batch pops before this stream's
};

template <int kStreams>
struct TokenRowsArgsOf {
  PoolView pool;
  uint16_t* k;                      // read: outputs, contiguous
  uint16_t* v;
  long long k_stride, v_stride;     // elements from one token's row to the next one's
  int32_t* free_stack;
  int top;
  int is_meta;                      // append: pop pages and write the lists (layer 0)
  int n;                            // streams
  int units;                        // row numbers in all
  int* err;
  TokenRows item[kStreams];
};
using TokenRowsArgs = TokenRowsArgsOf<kMaxTokenBatch>;

// Page list entries start, start - 1, .. (count of them) go back on the free
// stack from free[top + base] on.
struct TokenDropItem {
  const int32_t* pages;
  int start, count, base;
};
template <int kStreams>
struct TokenDropArgsOf {
  int32_t* free_stack;
  int top;
  int n;
  int pool_pages;
  int* err;
  TokenDropItem item[kStreams];
};
using TokenDropArgs = TokenDropArgsOf<kMaxTokenBatch>;

// One stream of an attention call. Its query rows (token, head of the group) are
// numbered token * group + member for each KV head and cut into blocks of the
// kernel's rows; a CTA takes one (block, KV head, split).
struct TokenQuery {
  const int32_t* pages;
  int row0, n;                      // its token rows in q and out
  int pos0;                         // position of the first
  int cta0;                         // its first CTA
  int blocks, splits;
};

template <int kStreams>
struct TokenAttendArgsOf {
  const uint16_t* q;                // [rows][q_heads][64], rows q_stride elements apart
  uint16_t* out;                    // [rows][q_heads][64]
  const int32_t* parents;           // trees: [rows]
  long long q_stride;
  int heads, group;                 // KV heads, query heads per KV head
  PoolView pool;
  int window, sinks;
  float scale_log2;                 // sm_scale * log2(e)
  float* part_o;                    // [cta][rows][64], unnormalised
  float* part_ml;                   // [cta][rows][2]: max (log2 units) and sum
  unsigned* joined;                 // [cta]: splits of the row block that have ended; 0 between calls
  int* err;
  int n;
  int ctas;
  int rows;                         // query rows per CTA
  int lanes;                        // matrix-unit kernel: its lanes per CTA, 2 or 4
  TokenQuery item[kStreams];
};
using TokenAttendArgs = TokenAttendArgsOf<kMaxTokenBatch>;

// The arguments with their first streams only (the items come last).
template <template <int> class Args>
Args<kSmallTokenBatch> small_args(const Args<kMaxTokenBatch>& a) {
  static_assert(offsetof(Args<kSmallTokenBatch>, item) == offsetof(Args<kMaxTokenBatch>, item), "a common start");
  Args<kSmallTokenBatch> r;
  std::memcpy(static_cast<void*>(&r), &a, sizeof(r));
  return r;
}

// The item whose CTAs (units) the index falls into: the last one that starts at
// or before it and is not empty. First entries grow with i.
template <typename Item, int Item::*First>
__device__ __forceinline__ int find_item(const Item* item, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (item[mid].*First <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Page of the list's entry pi; an append on layer 0 takes its new ones from the free stack.
template <typename Args>
__device__ __forceinline__ int page_of(const Args& a, const TokenRows& it, int pi) {
  const int page = a.is_meta && pi >= it.old_pages
                       ? a.free_stack[a.top - 1 - it.pop0 - (pi - it.old_pages)]
                       : it.pages[pi];
  if (page < 0 || page >= a.pool.pool_pages) {
    atomicOr(a.err, kErrPageRange);
    return -1;
  }
  return page;
}

// Eight bf16 values to E4M3 codes of v * 2^-e (fp8_row_exponent's e, of the row that 8
// neighbouring lanes hold), with all arithmetic on pairs. The largest magnitude's bits
// as an integer are E * 128 + mantissa, and e = E - 135, one more where the mantissa is
// above 0.75: a carry. v * 2^-e is exact in bf16 but for values that no code reaches.
__device__ __forceinline__ uint2 quantise8(const uint4& val, int* e_out) {
  const uint32_t w[4] = {val.x, val.y, val.z, val.w};
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t mag = w[i] & 0x7FFF7FFFu;
    asm("max.bf16x2 %0, %0, %1;\n" : "+r"(big) : "r"(mag));
  }
  const unsigned group = 0xFFu << (threadIdx.x & 24);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) {
    const uint32_t other = __shfl_xor_sync(group, big, d);
    asm("max.bf16x2 %0, %0, %1;\n" : "+r"(big) : "r"(other));
  }
  const int top = max((int)(big & 0xFFFFu), (int)(big >> 16));
  const int e = top == 0 ? 0 : max(((top + 31) >> 7) - 135, -126);
  *e_out = e;
  const uint32_t s1 = (uint32_t)(127 - e) << 7, scale = s1 | (s1 << 16);   // 2^-e, -120 <= -e <= 126
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x;
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(x) : "r"(w[i]), "r"(scale));
    c[i] = fp8_pack2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One CTA's share of an attention call.
struct TokenWork {
  int item, block, head, split;
  int r0, rows;                     // its query rows in the (stream, head): first, count
  int p0, p1;                       // positions of the first and the last row
};
template <bool TREE, typename Args>
__device__ __forceinline__ TokenWork token_work(const Args& a, int cta) {
  TokenWork w;
  w.item = find_item<TokenQuery, &TokenQuery::cta0>(a.item, a.n, cta);
  const TokenQuery& t = a.item[w.item];
  int x = cta - t.cta0;
  w.split = x % t.splits;
  x /= t.splits;
  w.head = x % a.heads;
  // the last block, which sees the most keys, goes first
  w.block = t.blocks - 1 - x / a.heads;
  w.r0 = w.block * a.rows;
  w.rows = min(a.rows, t.n * a.group - w.r0);
  // (a tree's nodes may be at any depth)
  w.p0 = t.pos0 + (TREE ? 0 : w.r0 / a.group);
  w.p1 = t.pos0 + (TREE ? t.n - 1 : (w.r0 + w.rows - 1) / a.group);
  return w;
}

// A batch's trees as one stream's CTA sees them: the parents, and what each of `rows` rows
// (few rows: the CTA's; else every node) sees of the tree's slots.
template <int kRows>
struct TreeSmem {
  uint64_t words[kRows][kTreeWords];
  int depth[kRows];
  int16_t parent[kTreeNodes];
};
// The stream's parents into shared memory, by `threads` threads; bad ones are noted and
// taken for none. A barrier must follow.
template <typename Tree>
__device__ __forceinline__ void load_parents(Tree& tree, const int32_t* parents, int n, int tid, int threads,
                                             int* err) {
  for (int i = tid; i < n; i += threads) {
    const int p = tree_parent(i, parents[i]);
    if (p < -1) atomicOr(err, kErrTree);
    tree.parent[i] = (int16_t)max(p, -1);
  }
}
template <typename Tree>
__device__ __forceinline__ void walk_tree(Tree& tree, int row, int node, int pos0, int window, int sinks) {
#pragma unroll
  for (int i = 0; i < kTreeWords; ++i) tree.words[row][i] = 0;
  tree.depth[row] = tree_walk(tree.parent, node, pos0, window, sinks, tree.words[row]);
}

// A rotary append: what turns k and q (pkv_append_tokens_rotary).
constexpr int kMaxAxes = 4;
struct RotaryArgs {
  const uint16_t* q;                // [rows][q_heads][64], rows q_stride elements apart
  uint16_t* q_out;                  // [rows][q_heads][64]
  long long q_stride;
  int q_heads;                      // 0: no q
  const int32_t* positions;         // [rows][axes]
  int axes;
  int distance;                     // between a pair's elements
  unsigned long long turn[kHeadDim / 2];   // turns per unit of position, 2^64 to the turn
  uint8_t axis[kHeadDim / 2];
};

// Accepted drafts of one stream: slots pos0 + kept[i] move to pos0 + i (i < m), and the list
// entries start, start - 1, .. (count of them) go back on the free stack from top + base on.
struct TokenKeepItem {
  const int32_t* pages;
  int pos0, n, m;                   // nodes, and how many stay
  int kept0;                        // first of its entries in kept
  int start, count, base;
};
template <int kStreams>
struct TokenKeepArgsOf {
  PoolView pool;                    // layer 0's
  long long layer_bytes;
  int layers;
  const int32_t* kept;
  int32_t* free_stack;
  int top;
  int n;
  int* err;
  TokenKeepItem item[kStreams];
};
using TokenKeepArgs = TokenKeepArgsOf<kMaxTokenBatch>;

cudaError_t launch_token_append(const TokenRowsArgs& a, cudaStream_t s);
cudaError_t launch_token_append_rotary(const TokenRowsArgs& a, const RotaryArgs& r, int num_sms, cudaStream_t s);
cudaError_t launch_token_keep(const TokenKeepArgs& a, cudaStream_t s);
cudaError_t launch_token_read(const TokenRowsArgs& a, cudaStream_t s);
cudaError_t launch_token_drop(const TokenDropArgs& a, cudaStream_t s);

// Attention in blocks of 8, 16 or 24 query rows (a.rows). A stream of more rows reads its keys once a
// block, from L2 but for the first, so this kernel takes streams of at most kTokenFewRowsAll rows per KV
// head, or of kTokenFewRows where this is estimated to end first (or for f16 weights, see attend_rows).
// (16 streams of 4001 tokens, 8 KV heads, 32 / 48 / 64 rows: 28 / 51 / 49 us on bf16 pages and 39 / 72 /
// 77 us on E4M3 pages, in launch_token_tc's blocks of 128 rows 31 / 31 / 31 and 50 / 51 / 51 us; streams
// of 500 .. 4001 tokens with 4 .. 48 / 4 .. 64 rows: 25 / 32 against 24 / 24 us, on E4M3 pages 37 / 45
// against 32 / 33 us. One stream with 64 rows, here / there: 4000 tokens 11.1 / 12.9 us, 16000 16.9 /
// 16.9, 32000 26 / 24, 131000 80 / 56, with 48 rows 10.9 / 12.8, 15.2 / 16.9, 22.1 / 23.5, 65 / 56; on
// E4M3 pages, 64 rows, 14.2 / 16.5, 24.1 / 23.0, 39 / 34, 131 / 87. Four of 8000 with 48 / 64 rows 21 /
// 27 against 19 / 20 us.)
constexpr int kTokenFewRows = 64;
constexpr int kTokenFewRowsAll = 32;
cudaError_t launch_token_few(const TokenAttendArgs& a, cudaStream_t s);
// What a 64-slot tile takes a CTA of that many rows, in us, beside the SM's other one.
inline double token_few_tile_us(int rows) { return rows == 24 ? 0.8 : 0.55; }
// The same on bf16 pages where several blocks read the same keys.
constexpr double kTokenFewSharedTileUs = 0.33;
// Resident CTAs per SM of that kernel.
int token_few_ctas_per_sm();
// Attention of 128, 256 or (on E4M3 pages) 512 query rows per CTA (a.rows).
int token_tc_max_rows(bool fp8);
int token_tc_ctas_per_sm(int lanes);
// What a 64-slot tile takes a CTA of it, in us, beside the SM's others, where a stream has up to
// `most` rows.
double token_tc_tile_us(bool fp8, int rows, int lanes, int most);
// What a CTA's start and end take beyond CtaCost's tiles, in us; and what a split adds to the join.
double token_tc_start_us(bool fp8, int lanes, bool tree);
constexpr double kTokenSplitUs = 0.25;
cudaError_t launch_token_tc(const TokenAttendArgs& a, cudaStream_t s);
// Joins the splits of the items that have several (launch_token_few does so itself).
cudaError_t launch_token_combine(const TokenAttendArgs& a, cudaStream_t s);

}  // namespace pkv
