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

// One CTA's share of an attention call.
struct TokenWork {
  int item, block, head, split;
  int r0, rows;                     // its query rows in the (stream, head): first, count
  int p0, p1;                       // positions of the first and the last row
};
template <typename Args>
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
  w.p0 = t.pos0 + w.r0 / a.group;
  w.p1 = t.pos0 + (w.r0 + w.rows - 1) / a.group;
  return w;
}

cudaError_t launch_token_append(const TokenRowsArgs& a, cudaStream_t s);
cudaError_t launch_token_read(const TokenRowsArgs& a, cudaStream_t s);
cudaError_t launch_token_drop(const TokenDropArgs& a, cudaStream_t s);

// Attention in blocks of 8, 16 or 24 query rows (a.rows). A stream of more rows reads its keys
// once a block, from L2 but for the first, so this kernel takes at most kTokenFewRowsAll of
// them per KV head, or kTokenFewRows where the streams up to that size have no more than
// kTokenFewRowsAll on average. (16 streams of 4001 tokens, 8 KV heads, all of them with
// 32 / 48 / 64 rows: 29.5 / 52.4 / 49.7 us on bf16 pages and 41 / 75 / 80 us on E4M3 pages
// against 31.8 and 53 us in launch_token_tc's blocks of 128 rows. Streams of 500 .. 4001
// tokens, with 32 / 4 .. 48 / 4 .. 64 rows: 28 / 25 / 33 against 32 / 40 / 40 us, and on
// E4M3 pages 36 / 40 / 46 against 46 / 54 / 55 us.)
constexpr int kTokenFewRows = 64;
constexpr int kTokenFewRowsAll = 32;
cudaError_t launch_token_few(const TokenAttendArgs& a, cudaStream_t s);
// Resident CTAs per SM of that kernel.
int token_few_ctas_per_sm();
// Attention of 128, 256 or (on E4M3 pages) 512 query rows per CTA (a.rows).
int token_tc_max_rows(bool fp8);
int token_tc_ctas_per_sm(bool fp8, int rows);
cudaError_t launch_token_tc(const TokenAttendArgs& a, cudaStream_t s);
// Joins the splits of the items that have several (launch_token_few does so itself).
cudaError_t launch_token_combine(const TokenAttendArgs& a, cudaStream_t s);

}  // namespace pkv
