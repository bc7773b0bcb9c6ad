// The token streams' host-side plan, callable from Python.
#include "pkv_token_plan.h"

#include <cstddef>

using namespace pkv;

extern "C" {
TokenCounts* plan_open(int page_size, int max_tokens, int window, int sinks) {
  auto* t = new TokenCounts;
  tok_open(t, page_size, max_tokens, window, sinks);
  return t;
}
void plan_free(TokenCounts* t) { delete t; }
int plan_append(TokenCounts* t, int n) {
  const int need = tok_append_need(*t, n);
  tok_append(t, n);
  return need;
}
int plan_can_drop(TokenCounts* t, int n) { return tok_can_drop(*t, n); }
int plan_drop(TokenCounts* t, int n) {
  const int p = tok_drop_pages(*t, n);
  tok_drop(t, n);
  return p;
}
int plan_evict(TokenCounts* t) {
  const int g = tok_evict_to(*t), n = g - t->gap1;
  t->gap1 = g;
  return n;
}
int plan_holds(TokenCounts* t, int lo, int sinks) { return tok_holds(*t, lo, sinks); }
void plan_live(TokenCounts* t, int* out) {
  out[0] = tok_live_front(*t);
  out[1] = tok_live_back(*t);
  out[2] = t->gap1;
  out[3] = t->n_pages;
}
int plan_zero(TokenCounts* t, int pos0, int n, int old_pages) { return tok_zero_slots(*t, pos0, n, old_pages); }
int plan_tiles(int p0, int p1, int window, int sinks, int* out, int cap) {
  const TokTiles r = tok_tiles(p0, p1, window, sinks);
  for (int j = 0; j < r.n && j < cap; ++j) out[j] = tok_tile(r, j);
  return r.n;
}
int plan_full(int b, int p0, int p1, int window, int sinks) { return tok_tile_full(b, p0, p1, window, sinks); }
int plan_needs(int tile, int p0, int p1, int window, int sinks) { return tok_span(p0, p1, window, sinks).needs(tile); }
int plan_whole(int tile, int p0, int p1, int window, int sinks) { return tok_span(p0, p1, window, sinks).whole(tile); }
unsigned long long plan_mask(int b, int p, int window, int sinks) { return tok_mask(b, p, window, sinks); }
}
