// Token streams: the host's counters and the index arithmetic that the host and
// the kernels share. Plain C++ (no CUDA), so that it can be checked on a CPU.
//
// A token stream holds the keys and values of positions 0 .. len-1, position j in
// slot j % page_size of entry j / page_size of the stream's page list. With a
// retention window, whole pages that no later query can see are freed, except the
// pages that hold the first `sinks` tokens: the freed entries are keep0 .. gap1-1,
// and the live ones 0 .. min(keep0, n_pages)-1 and gap1 .. n_pages-1.
#pragma once

#include <stdint.h>

#ifndef PKV_HD
#ifdef __CUDACC__
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif
#endif

namespace pkv {

struct TokenCounts {
  int page_size = 0;
  int max_tokens = 0;
  int window = 0;        // retention window (0: every token is kept)
  int sinks = 0;
  int len = 0;
  int n_pages = 0;       // entries of the page list, freed ones included
  int keep0 = 0;         // pages that hold the sinks
  int gap1 = 0;          // first live entry behind the freed ones; keep0: none freed
  int u_pos0 = 0;        // the last append: its first position, and the entries
  int u_old_pages = 0;   // that the list had before it
  bool pending = false;  // it may be continued on further layers or rolled back
};

PKV_HD int tok_pages(int len, int page_size) { return (len + page_size - 1) / page_size; }

// First position that a query at position p sees inside its window.
PKV_HD int tok_window_lo(int p, int window) { return window > 0 && p >= window ? p - window + 1 : 0; }

inline void tok_open(TokenCounts* t, int page_size, int max_tokens, int window, int sinks) {
  *t = TokenCounts();
  t->page_size = page_size;
  t->max_tokens = max_tokens;
  t->window = window;
  t->sinks = window > 0 ? sinks : 0;
  t->keep0 = t->gap1 = tok_pages(t->sinks, page_size);
}
inline int tok_live_front(const TokenCounts& t) { return t.n_pages < t.keep0 ? t.n_pages : t.keep0; }
inline int tok_live_back(const TokenCounts& t) { return t.n_pages > t.gap1 ? t.n_pages - t.gap1 : 0; }
// Pages that an append of n tokens pops.
inline int tok_append_need(const TokenCounts& t, int n) {
  return tok_pages(t.len + n, t.page_size) - t.n_pages;
}
inline void tok_append(TokenCounts* t, int n) {
  t->u_pos0 = t->len;
  t->u_old_pages = t->n_pages;
  t->n_pages += tok_append_need(*t, n);
  t->len += n;
  t->pending = true;
}
// Slots behind the last token of a page that the append opens: they are zeroed.
inline int tok_zero_slots(const TokenCounts& t, int pos0, int n, int old_pages) {
  const int end = pos0 + n;
  if (n == 0 || tok_pages(end, t.page_size) <= old_pages) return 0;
  return tok_pages(end, t.page_size) * t.page_size - end;
}
// Whether the last n tokens can be dropped: every position that a query at the
// new end sees must still be held.
inline bool tok_can_drop(const TokenCounts& t, int n) {
  if (n < 0 || n > t.len) return false;
  return t.gap1 == t.keep0 || tok_window_lo(t.len - n, t.window) >= t.gap1 * t.page_size;
}
// Pages that the drop frees: the list's last ones.
inline int tok_drop_pages(const TokenCounts& t, int n) { return t.n_pages - tok_pages(t.len - n, t.page_size); }
inline void tok_drop(TokenCounts* t, int n) {
  t->n_pages -= tok_drop_pages(*t, n);
  t->len -= n;
  t->pending = false;
}
// The first live entry behind the freed ones once everything that no later query
// sees is freed: entries gap1 .. the result - 1 go.
inline int tok_evict_to(const TokenCounts& t) {
  if (t.window == 0) return t.gap1;
  const int g = tok_window_lo(t.len, t.window) / t.page_size;
  return g > t.gap1 ? g : t.gap1;
}
// Whether positions lo .. len-1 and the first `sinks` ones are held.
inline bool tok_holds(const TokenCounts& t, int lo, int sinks) {
  if (t.gap1 == t.keep0) return true;
  return lo >= t.gap1 * t.page_size && sinks <= t.keep0 * t.page_size;
}

// ---------------------------------------------------------- attention tiles
constexpr int kTokTile = 64;

PKV_HD int tok_tiles_of(int n) { return n / kTokTile + (n % kTokTile > 0); }   // (n may be INT_MAX)

// The 64-slot tiles that queries at positions p0 .. p1 see: n_front of them from
// the first on (the sinks), then those from `lo` on, n in all.
struct TokTiles {
  int n_front, lo, n;
};
PKV_HD TokTiles tok_tiles(int p0, int p1, int window, int sinks) {
  TokTiles r;
  const int hi = p1 / kTokTile + 1;
  r.lo = tok_window_lo(p0, window) / kTokTile;
  r.n_front = tok_tiles_of(sinks);
  if (r.n_front >= r.lo) r.n_front = r.lo = 0;
  r.n = r.n_front + hi - r.lo;
  return r;
}
PKV_HD int tok_tile(const TokTiles& r, int j) { return j < r.n_front ? j : r.lo + (j - r.n_front); }

// Whether every slot of the tile that starts at position b is seen from every
// position p0 .. p1.
PKV_HD bool tok_tile_full(int b, int p0, int p1, int window, int sinks) {
  return b + kTokTile - 1 <= p0 && (b >= tok_window_lo(p1, window) || b + kTokTile <= sinks);
}
PKV_HD uint64_t tok_low_bits(int n) {
  return n <= 0 ? 0ull : (n >= 64 ? ~0ull : ((1ull << n) - 1ull));
}
// The tiles (by number) that queries at positions p0 .. p1 see something of, and
// those that all of them see whole.
struct TokSpan {
  int front, lo, hi;             // needed: t < front (and <= hi), or lo <= t <= hi
  int full_front, f0, f1;        // whole: t < full_front, or f0 <= t < f1
  PKV_HD bool needs(int t) const { return t <= hi && (t >= lo || t < front); }
  PKV_HD bool whole(int t) const { return t < f1 && (t >= f0 || t < full_front); }
};
PKV_HD TokSpan tok_span(int p0, int p1, int window, int sinks) {
  TokSpan s;
  s.front = tok_tiles_of(sinks);
  s.lo = tok_window_lo(p0, window) / kTokTile;
  s.hi = p1 / kTokTile;
  s.full_front = sinks / kTokTile;
  s.f0 = (tok_window_lo(p1, window) + kTokTile - 1) / kTokTile;
  s.f1 = (p0 + 1) / kTokTile;
  return s;
}
// The page list entry that slots f .. f + rows - 1 of a tile (rows of one page) are read
// from for queries at positions p0 .. p1. Where none of them sees any of the slots, the
// entry may be freed, its page another stream's by now, and what that holds may be no
// number (0 * NaN is NaN in a product): such a block takes its masked rows from the page of
// p1, which the stream holds.
PKV_HD int tok_block_entry(int f, int rows, int p0, int p1, int window, int sinks, int page_size) {
  const bool seen = f <= p1 && (f + rows > tok_window_lo(p0, window) || f < sinks);
  return (seen ? f : p1) / page_size;
}
// Bit i: whether slot b + i is seen from position p.
PKV_HD uint64_t tok_mask(int b, int p, int window, int sinks) {
  return tok_low_bits(p - b + 1) & (~tok_low_bits(tok_window_lo(p, window) - b) | tok_low_bits(sinks - b));
}

}  // namespace pkv
