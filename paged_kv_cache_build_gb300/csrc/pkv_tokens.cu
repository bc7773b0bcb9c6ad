// C-ABI entry points of the token streams (see include/pkv.h). As for frames, the
// host keeps the counters and checks every argument, the capacity and the call
// order before anything is launched; a call that fails has changed nothing.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "pkv_ctx.h"
#include "pkv_tokens.cuh"

using namespace pkv;

namespace {

constexpr int kMaxRows = 1 << 24;    // token rows of one call
constexpr int kMaxGroup = 128;       // query heads per KV head
// Split-KV partials, allocated when the handle's first token stream opens and kept until
// it is destroyed, so that captured calls keep their address; plan_splits cuts no finer
// than they hold.
constexpr size_t kTokenScratchBytes = size_t(64) << 20;

constexpr int kTokenJoins = 16384;   // counters of the splits' joins

bool misaligned(const void* p) { return !p || !aligned16(p); }

// The batch's streams, each named once and a token stream; row offsets that start
// at 0 and do not fall.
pkv_status check_batch(pkv_t h, int n, const int* sids, const int* row_off) {
  if (!h) return fail(h, PKV_ERR_INVALID, "null handle");
  if (n < 1 || n > kMaxTokenBatch || !sids)
    return fail(h, PKV_ERR_INVALID, "a batch names 1..%d streams", kMaxTokenBatch);
  if (pkv_status r = check_device(h)) return r;
  const unsigned long long mark = ++h->batch_no;
  for (int i = 0; i < n; ++i) {
    Stream* st = nullptr;
    if (pkv_status r = get_stream(h, sids[i], &st)) return r;
    if (st->cfg.mode != kModeTokens)
      return fail(h, PKV_ERR_STATE, "stream %d is not a token stream", sids[i]);
    if (h->seen[sids[i]] == mark) return fail(h, PKV_ERR_INVALID, "stream %d twice in one batch", sids[i]);
    h->seen[sids[i]] = mark;
  }
  if (row_off) {
    if (row_off[0] != 0) return fail(h, PKV_ERR_INVALID, "row_off[0] must be 0");
    for (int i = 0; i < n; ++i)
      if (row_off[i + 1] < row_off[i] || row_off[i + 1] > kMaxRows)
        return fail(h, PKV_ERR_INVALID, "row_off must not fall, and stay within %d rows", kMaxRows);
  }
  return PKV_OK;
}

pkv_status check_layer(pkv_t h, int layer) {
  if (layer < 0 || layer >= h->L) return fail(h, PKV_ERR_INVALID, "layer %d out of range", layer);
  return PKV_OK;
}

// A row stride in elements: whole 16-byte vectors, rows that do not overlap.
pkv_status check_stride(pkv_t h, const char* name, long long stride, int row) {
  if (stride % 8 != 0 || stride < row)
    return fail(h, PKV_ERR_INVALID, "%s must be a multiple of 8 of at least %d elements", name, row);
  return PKV_OK;
}

void rows_args(pkv_t h, int layer, TokenRowsArgs* a) {
  std::memset(a, 0, offsetof(TokenRowsArgs, item));
  a->pool = pool_view(h, layer);
  a->free_stack = h->d_free;
  a->top = h->free_top;
  a->err = h->d_err;
}

// What a kernel's CTA costs, in the time of one 64-slot tile: its start and end, and
// (when it leaves partial results) their share of the join. As measured: decode steps
// take 0.25 us a tile and 3 us a CTA, the matrix-unit kernel 0.5 us and 5 us.
struct CtaCost {
  int slots;                     // CTAs that run at once
  int fixed, join;
  int min_piece;                 // tiles below which a range is not cut
  int max_ctas;                  // whose partial results the scratch holds
};

// Splits of the items' key ranges over CTAs, given the tiles that an item's first
// and last block see. All ranges are cut into pieces of one length (at most); of the
// lengths most/1, most/2, .. the one whose waves of CTAs are estimated to end first.
void plan_splits(TokenAttendArgs* a, const int* first, const int* last, const CtaCost& c) {
  int most = 1;
  for (int i = 0; i < a->n; ++i) most = std::max({most, first[i], last[i]});
  int best = most;
  double best_t = 0;
  for (int s = 1; s == 1 || most / s >= c.min_piece; ++s) {
    const int piece = ceil_div(most, s);
    double ctas = 0, work = 0;
    for (int i = 0; i < a->n; ++i) {
      const double pairs = (double)a->item[i].blocks * a->heads;
      const int splits = ceil_div(std::max(first[i], last[i]), piece);
      ctas += pairs * splits;
      work += pairs * (0.5 * (first[i] + last[i]) + splits * (c.fixed + (splits > 1 ? c.join : 0)));
    }
    if (s > 1 && ctas > c.max_ctas) break;
    const double waves = std::max(1.0, std::ceil(ctas / c.slots));
    const double t = std::max(waves * work / ctas, (double)piece + c.fixed);
    if (s == 1 || t < best_t * 0.97) {
      best_t = t;
      best = piece;
    }
    if (ctas > 8.0 * c.slots || s >= 64) break;
  }
  int cta = 0;
  for (int i = 0; i < a->n; ++i) {
    TokenQuery& t = a->item[i];
    t.splits = std::max(1, ceil_div(std::max(first[i], last[i]), best));
    t.cta0 = cta;
    cta += t.blocks * a->heads * t.splits;
  }
  a->ctas = cta;
}

}  // namespace

namespace pkv {

pkv_status token_rollback(pkv_t h, Stream* st, cudaStream_t s) {
  TokenCounts& t = st->tok;
  if (!t.pending) return fail(h, PKV_ERR_STATE, "nothing to roll back");
  const int n = t.len - t.u_pos0, pages = tok_drop_pages(t, n);
  const PushSegment g = seg(st->d_pages, t.n_pages - 1, pages, -1);
  if (pkv_status r = push_pages(h, &g, 1, s)) return r;
  tok_drop(&t, n);
  return PKV_OK;
}

pkv_status token_evict(pkv_t h, Stream* st, cudaStream_t s) {
  TokenCounts& t = st->tok;
  const int g = tok_evict_to(t);
  if (g > t.gap1) {
    const PushSegment sg = seg(st->d_pages, t.gap1, g - t.gap1);
    if (pkv_status r = push_pages(h, &sg, 1, s)) return r;
    t.gap1 = g;
  }
  t.pending = false;
  return PKV_OK;
}

}  // namespace pkv

extern "C" {

pkv_status pkv_stream_open_tokens(pkv_t h, int max_tokens, int window, int sinks, int* stream_id) {
  if (!h || !stream_id) return fail(h, PKV_ERR_INVALID, "null argument");
  if (max_tokens < 1 || max_tokens > (1 << 28))
    return fail(h, PKV_ERR_INVALID, "max_tokens %d outside 1..2^28", max_tokens);
  if (window < 0 || sinks < 0 || (window == 0 && sinks > 0))
    return fail(h, PKV_ERR_INVALID, "window and sinks >= 0 required (no sinks without a window)");
  if (pkv_status r = check_device(h)) return r;
  int sid = -1;
  for (int i = 0; i < h->max_streams && sid < 0; ++i)
    if (!h->streams[i].open) sid = i;
  if (sid < 0) return fail(h, PKV_ERR_OOM, "no free stream id");
  Stream st;
  st.cfg.mode = kModeTokens;
  tok_open(&st.tok, h->Ps, max_tokens, window, std::min(sinks, max_tokens));
  // the page list, and the table buffers of pkv_export_state
  const size_t cap = (size_t)tok_pages(max_tokens, h->Ps);
  st.tbl_cap = (int)std::min<size_t>(cap, (size_t)h->P);
  const size_t words = cap + 2 * (size_t)st.tbl_cap;
  if (!h->d_token_part) PKV_CUDA(h, cudaMalloc(&h->d_token_part, kTokenScratchBytes));
  if (!h->d_joined) {
    unsigned* p = nullptr;
    PKV_CUDA(h, cudaMalloc(&p, kTokenJoins * sizeof(unsigned)));
    SetupStream setup;
    setup.fill(p, 0, kTokenJoins * sizeof(unsigned));
    if (cudaError_t e = setup.wait()) {
      cudaFree(p);
      return cuda_fail(h, e, "stream_open_tokens: clearing the join counters");
    }
    h->d_joined = p;
  }
  // (not cleared: an entry is written before any call reads it)
  PKV_CUDA(h, cudaMalloc(&st.d_mem, words * sizeof(int32_t)));
  st.d_pages = st.d_mem;
  st.d_tbl_idx = st.d_mem + cap;
  st.d_tbl_len = st.d_tbl_idx + st.tbl_cap;
  st.open = true;
  h->streams[sid] = st;
  *stream_id = sid;
  return PKV_OK;
}

pkv_status pkv_append_tokens(pkv_t h, int n, const int* sids, const int* row_off, int layer,
                             const void* k, const void* v, long long k_stride, long long v_stride,
                             void* cuda_stream) {
  if (pkv_status r = check_batch(h, n, sids, row_off)) return r;
  if (!row_off) return fail(h, PKV_ERR_INVALID, "null row_off");
  if (pkv_status r = check_layer(h, layer)) return r;
  const int row = h->H * kHeadDim;
  if (k_stride == 0) k_stride = row;
  if (v_stride == 0) v_stride = row;
  if (pkv_status r = check_stride(h, "k_stride", k_stride, row)) return r;
  if (pkv_status r = check_stride(h, "v_stride", v_stride, row)) return r;
  if (row_off[n] > 0 && (misaligned(k) || misaligned(v)))
    return fail(h, PKV_ERR_INVALID, "k/v must be 16-byte aligned device pointers");
  TokenRowsArgs a;
  rows_args(h, layer, &a);
  a.k = const_cast<uint16_t*>(static_cast<const uint16_t*>(k));
  a.v = const_cast<uint16_t*>(static_cast<const uint16_t*>(v));
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.is_meta = layer == 0 ? 1 : 0;
  a.n = n;
  long long need = 0, units = 0;
  for (int i = 0; i < n; ++i) {
    Stream& st = h->streams[sids[i]];
    const TokenCounts& t = st.tok;
    const int rows = row_off[i + 1] - row_off[i];
    TokenRows& it = a.item[i];
    it.pages = st.d_pages;
    it.unit0 = (int)units;
    it.row0 = row_off[i];
    it.n = rows;
    it.pop0 = (int)need;
    if (layer == 0) {
      if (rows > t.max_tokens - t.len)
        return fail(h, PKV_ERR_INVALID, "stream %d: %d + %d tokens exceed its %d", sids[i], t.len, rows,
                    t.max_tokens);
      it.pos0 = t.len;
      it.old_pages = t.n_pages;
      need += tok_append_need(t, rows);
    } else {
      if (rows == 0) {
        it.pos0 = t.len;
        it.old_pages = t.n_pages;
      } else {
        if (!t.pending) return fail(h, PKV_ERR_STATE, "stream %d: layer > 0 append without one on layer 0", sids[i]);
        if (rows != t.len - t.u_pos0)
          return fail(h, PKV_ERR_INVALID, "stream %d: %d rows, the append on layer 0 had %d", sids[i], rows,
                      t.len - t.u_pos0);
        it.pos0 = t.u_pos0;
        it.old_pages = t.u_old_pages;
      }
    }
    units += rows + tok_zero_slots(t, it.pos0, rows, it.old_pages);
  }
  if (need > h->free_top)
    return fail(h, PKV_ERR_OOM, "free list exhausted (%lld pages needed, %d free)", need, h->free_top);
  if (units == 0) return PKV_OK;
  a.units = (int)units;
  PKV_CUDA(h, launch_token_append(a, as_stream(cuda_stream)));
  if (layer == 0) {
    h->free_top -= (int)need;
    for (int i = 0; i < n; ++i)
      if (a.item[i].n > 0) tok_append(&h->streams[sids[i]].tok, a.item[i].n);
  }
  return PKV_OK;
}

pkv_status pkv_drop_tokens(pkv_t h, int n, const int* sids, const int* counts, void* cuda_stream) {
  if (pkv_status r = check_batch(h, n, sids, nullptr)) return r;
  if (!counts) return fail(h, PKV_ERR_INVALID, "null counts");
  TokenDropArgs a;
  std::memset(&a, 0, offsetof(TokenDropArgs, item));
  a.free_stack = h->d_free;
  a.top = h->free_top;
  a.pool_pages = h->P;
  a.err = h->d_err;
  int base = 0;
  // the last stream's pages first: they were popped last
  for (int i = n - 1; i >= 0; --i) {
    const Stream& st = h->streams[sids[i]];
    const TokenCounts& t = st.tok;
    if (counts[i] < 0 || counts[i] > t.len)
      return fail(h, PKV_ERR_INVALID, "stream %d: %d of its %d tokens to drop", sids[i], counts[i], t.len);
    if (!tok_can_drop(t, counts[i]))
      return fail(h, PKV_ERR_STATE, "stream %d: what its window would see before the dropped tokens is evicted",
                  sids[i]);
    const int pages = tok_drop_pages(t, counts[i]);
    if (pages == 0) continue;
    TokenDropItem& it = a.item[a.n++];
    it.pages = st.d_pages;
    it.start = t.n_pages - 1;
    it.count = pages;
    it.base = base;
    base += pages;
  }
  if (h->free_top + base > h->P) return fail(h, PKV_ERR_STATE, "free stack overflow");
  if (a.n > 0) PKV_CUDA(h, launch_token_drop(a, as_stream(cuda_stream)));
  h->free_top += base;
  for (int i = 0; i < n; ++i)
    if (counts[i] > 0) tok_drop(&h->streams[sids[i]].tok, counts[i]);
  return PKV_OK;
}

pkv_status pkv_read_tokens(pkv_t h, int n, const int* sids, const int* pos0, const int* row_off, int layer,
                           void* k_out, void* v_out, void* cuda_stream) {
  if (pkv_status r = check_batch(h, n, sids, row_off)) return r;
  if (!row_off) return fail(h, PKV_ERR_INVALID, "null row_off");
  if (pkv_status r = check_layer(h, layer)) return r;
  if (row_off[n] == 0) return PKV_OK;
  if (misaligned(k_out) || misaligned(v_out))
    return fail(h, PKV_ERR_INVALID, "k_out/v_out must be 16-byte aligned device pointers");
  TokenRowsArgs a;
  rows_args(h, layer, &a);
  a.k = static_cast<uint16_t*>(k_out);
  a.v = static_cast<uint16_t*>(v_out);
  a.n = n;
  a.units = row_off[n];
  for (int i = 0; i < n; ++i) {
    const Stream& st = h->streams[sids[i]];
    const TokenCounts& t = st.tok;
    const int rows = row_off[i + 1] - row_off[i];
    const int p0 = pos0 ? pos0[i] : t.len - rows;
    if (p0 < 0 || rows > t.len - p0)
      return fail(h, PKV_ERR_INVALID, "stream %d: positions %d.. (%d rows) of %d tokens", sids[i], p0, rows, t.len);
    // evicted: what lies between the sinks' pages and the first live one
    const long long gap0 = (long long)t.keep0 * h->Ps, gap1 = (long long)t.gap1 * h->Ps;
    if (rows > 0 && gap1 > gap0 && p0 < gap1 && (long long)p0 + rows > gap0)
      return fail(h, PKV_ERR_STATE, "stream %d: positions %lld..%lld are evicted", sids[i], gap0, gap1 - 1);
    TokenRows& it = a.item[i];
    it.pages = st.d_pages;
    it.unit0 = it.row0 = row_off[i];
    it.n = rows;
    it.pos0 = p0;
    it.old_pages = INT_MAX;
    it.pop0 = 0;
  }
  PKV_CUDA(h, launch_token_read(a, as_stream(cuda_stream)));
  return PKV_OK;
}

pkv_status pkv_attend_tokens(pkv_t h, const void* q, int q_heads, long long q_stride, const int* row_off,
                             const int* sids, int n, int layer, void* out, int window, int sinks,
                             float sm_scale, void* cuda_stream) {
  if (pkv_status r = check_batch(h, n, sids, row_off)) return r;
  if (!row_off) return fail(h, PKV_ERR_INVALID, "null row_off");
  if (pkv_status r = check_layer(h, layer)) return r;
  if (q_heads < 1 || q_heads % h->H != 0 || q_heads / h->H > kMaxGroup)
    return fail(h, PKV_ERR_INVALID, "q_heads %d must be 1..%d times the cache's %d heads", q_heads, kMaxGroup, h->H);
  if (window < 0 || sinks < 0 || (window == 0 && sinks > 0))
    return fail(h, PKV_ERR_INVALID, "window and sinks >= 0 required (no sinks without a window)");
  const float scale = sm_scale <= 0.f ? 1.0f / std::sqrt((float)h->D) : sm_scale;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!std::isnormal(scale) || !std::isnormal(scale_log2))
    return fail(h, PKV_ERR_INVALID, "sm_scale %g (times log2 e) is no normal fp32 number", sm_scale);
  const int group = q_heads / h->H, row = q_heads * kHeadDim;
  if (q_stride == 0) q_stride = row;
  if (pkv_status r = check_stride(h, "q_stride", q_stride, row)) return r;
  if (row_off[n] == 0) return PKV_OK;
  if ((long long)row_off[n] * q_heads > INT_MAX / 16)
    return fail(h, PKV_ERR_INVALID, "%d rows of %d heads are too many for one call", row_off[n], q_heads);
  if (misaligned(q) || misaligned(out))
    return fail(h, PKV_ERR_INVALID, "q/out must be 16-byte aligned device pointers");
  TokenAttendArgs a;
  std::memset(&a, 0, offsetof(TokenAttendArgs, item));
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.q_stride = q_stride;
  a.heads = h->H;
  a.group = group;
  a.pool = pool_view(h, layer);
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = scale_log2;
  a.err = h->d_err;
  a.joined = h->d_joined;
  int first[kMaxTokenBatch], last[kMaxTokenBatch];
  for (int i = 0; i < n; ++i) {
    const Stream& st = h->streams[sids[i]];
    const TokenCounts& t = st.tok;
    const int rows = row_off[i + 1] - row_off[i];
    if (rows > t.len)
      return fail(h, PKV_ERR_STATE, "stream %d: %d query rows, but only %d tokens", sids[i], rows, t.len);
    if (rows == 0) continue;
    if (!tok_holds(t, tok_window_lo(t.len - rows, window), sinks))
      return fail(h, PKV_ERR_STATE, "stream %d: keys that its queries see are evicted", sids[i]);
    TokenQuery& it = a.item[a.n++];
    it.pages = st.d_pages;
    it.row0 = row_off[i];
    it.n = rows;
    it.pos0 = t.len - rows;
  }
  // one launch per kernel: the streams' rows per KV head decide
  cudaStream_t s = as_stream(cuda_stream);
  const int n_items = a.n;
  TokenQuery all[kMaxTokenBatch];
  std::copy(a.item, a.item + n_items, all);
  long long rows_sum = 0;
  int n_small = 0;
  for (int i = 0; i < n_items; ++i) {
    const long long r = (long long)all[i].n * group;
    if (r <= kTokenFewRows) rows_sum += r, ++n_small;
  }
  const int few_rows = rows_sum <= (long long)kTokenFewRowsAll * n_small ? kTokenFewRows : kTokenFewRowsAll;
  const int max_rows = token_tc_max_rows(h->fp8);
  // one shape for all streams of the matrix-unit kernel, the largest's. On bf16 pages a second
  // launch costs more than the lanes that stay idle: 2 .. 34 new tokens of 18 streams, 25.8
  // against 39.1 us; a chunk of 1500 tokens beside 11 drafts of 20, group 4, 99 against 122 us.
  // On E4M3 pages it depends: the first batch 36.6 against 56.6 us, the second 165 against 155
  // us (there the 512-row shape leaves three of a draft's four lanes without rows).
  int tc_rows = 128;
  for (int i = 0; i < n_items; ++i)
    while (tc_rows < max_rows && (long long)all[i].n * group > tc_rows) tc_rows *= 2;
  for (const int shape : {few_rows, tc_rows}) {
    const int below = shape == few_rows ? 0 : few_rows;
    a.n = 0;
    int most = 0;
    for (int i = 0; i < n_items; ++i) {
      const long long r = (long long)all[i].n * group;
      if (r <= below || (r > shape && shape == few_rows)) continue;
      a.item[a.n++] = all[i];
      most = std::max(most, (int)std::min<long long>(r, shape));
    }
    if (a.n == 0) continue;
    const bool few = shape == few_rows;
    a.rows = !few ? shape : most <= 8 ? 8 : most > 16 && most <= 24 ? 24 : 16;
    for (int i = 0; i < a.n; ++i) {
      TokenQuery& it = a.item[i];
      it.blocks = ceil_div((long long)it.n * group, a.rows);
      const auto block_tiles = [&](int b) {
        const int r0 = b * a.rows, r1 = std::min(r0 + a.rows, it.n * group) - 1;
        return tok_tiles(it.pos0 + r0 / group, it.pos0 + r1 / group, window, sinks).n;
      };
      first[i] = block_tiles(0);
      last[i] = block_tiles(it.blocks - 1);
    }
    const int room = std::min<int>(kTokenScratchBytes / (a.rows * (kHeadDim + 2) * sizeof(float)), kTokenJoins);
    const CtaCost cost = few ? CtaCost{h->num_sms * token_few_ctas_per_sm(), 12, 4, 8, room}
                             : CtaCost{h->num_sms * token_tc_ctas_per_sm(h->fp8, shape), 10, 4, 8, room};
    plan_splits(&a, first, last, cost);
    bool split = false;
    for (int i = 0; i < a.n; ++i) split = split || a.item[i].splits > 1;
    if (split) {
      a.part_o = h->d_token_part;
      a.part_ml = h->d_token_part + (size_t)a.ctas * a.rows * kHeadDim;
    }
    PKV_CUDA(h, few ? launch_token_few(a, s) : launch_token_tc(a, s));
    if (split && !few) PKV_CUDA(h, launch_token_combine(a, s));
  }
  return PKV_OK;
}

pkv_status pkv_token_info(pkv_t h, int sid, int* n_tokens, int* evicted_from, int* evicted_to) {
  Stream* st = nullptr;
  if (pkv_status r = get_stream(h, sid, &st)) return r;
  if (st->cfg.mode != kModeTokens) return fail(h, PKV_ERR_STATE, "stream %d is not a token stream", sid);
  if (n_tokens) *n_tokens = st->tok.len;
  const bool gap = st->tok.gap1 > st->tok.keep0;
  if (evicted_from) *evicted_from = gap ? st->tok.keep0 * h->Ps : 0;
  if (evicted_to) *evicted_to = gap ? st->tok.gap1 * h->Ps : 0;
  return PKV_OK;
}

}  // extern "C"
