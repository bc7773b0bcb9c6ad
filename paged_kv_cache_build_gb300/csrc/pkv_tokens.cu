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
constexpr double kMaxFreq = 1048576.0;   // radians per unit of position

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
// (when it leaves partial results) their share of the join. A tile is what it takes beside the
// SM's other CTAs.
struct CtaCost {
  int slots;                     // CTAs that run at once
  double tile;                   // us
  int fixed, join;
  int min_piece;                 // tiles below which a range is not cut
  int max_ctas;                  // whose partial results the scratch holds
  bool one_wave;                 // look for the shortest ranges whose CTAs all run at once
};

// Splits of the items' key ranges over CTAs, given the tiles that an item's first
// and last block see. All ranges are cut into pieces of one length (at most); of the
// lengths most/1, most/2, .. the one whose waves of CTAs are estimated to end first. Returns
// the estimate in us.
double plan_splits(TokenAttendArgs* a, const int* first, const int* last, const CtaCost& c) {
  // (a batch of many streams is gone through some ten times: no integer divisions in there)
  double range[kMaxTokenBatch], pairs[kMaxTokenBatch], mean[kMaxTokenBatch];
  int most = 1;
  for (int i = 0; i < a->n; ++i) {
    most = std::max({most, first[i], last[i]});
    range[i] = std::max(first[i], last[i]);
    pairs[i] = (double)a->item[i].blocks * a->heads;
    mean[i] = 0.5 * (first[i] + last[i]);
  }
  int best = most;
  double best_t = 0;
  const auto cut = [&](int piece, double* work) {
    // range / piece rounded up: the argument is 0.5 / piece or more from a whole number, and a product
    // with the reciprocal is off by 2^-27 of that at most (ranges have up to 2^22 tiles)
    const double more = piece - 0.5, inv = 1.0 / piece;
    double ctas = 0, sum = 0;
    for (int i = 0; i < a->n; ++i) {
      const int splits = (int)((range[i] + more) * inv);
      ctas += pairs[i] * splits;
      sum += pairs[i] * (mean[i] + splits * (c.fixed + (splits > 1 ? c.join : 0)));
    }
    *work = sum;
    return ctas;
  };
  const auto consider = [&](int piece, double ctas, double work) {
    const double waves = std::max(1.0, std::ceil(ctas / c.slots));
    const double t = std::max(waves * work / ctas, (double)piece + c.fixed);
    if (best_t == 0 || t < best_t * 0.97) {
      best_t = t;
      best = piece;
    }
  };
  double work = 0;
  int whole = 0, parts = 0;                      // lengths whose CTAs all run at once, and do not
  for (int s = 1; s == 1 || most / s >= c.min_piece; ++s) {
    const int piece = ceil_div(most, s);
    const double ctas = cut(piece, &work);
    if (s > 1 && ctas > c.max_ctas) break;
    consider(piece, ctas, work);
    if (ctas <= c.slots) whole = piece;
    else if (parts == 0) parts = piece;
    if (ctas > 8.0 * c.slots || s >= 64) break;
  }
  // Chunks and trees (few streams): also the shortest of those that run at once. (Ragged trees of up
  // to 64 nodes, group 4, over up to 4001 tokens in 16 streams: 39 -> 33 us.)
  if (c.one_wave && parts > 0 && whole > parts + 1) {
    while (whole > parts + 1) {
      const int mid = (whole + parts) / 2;
      (cut(mid, &work) <= c.slots ? whole : parts) = mid;
    }
    const double ctas = cut(whole, &work);
    if (ctas <= c.max_ctas) consider(whole, ctas, work);
  }
  int cta = 0;
  for (int i = 0; i < a->n; ++i) {
    TokenQuery& t = a->item[i];
    t.splits = std::max(1, (std::max(first[i], last[i]) + best - 1) / best);
    t.cta0 = cta;
    cta += t.blocks * a->heads * t.splits;
  }
  a->ctas = cta;
  return best_t * c.tile;
}

// The shares of an attention call in blocks of a kernel's shape (query rows a CTA) with their
// splits; the estimate in us.
double plan_shape(pkv_t h, TokenAttendArgs* a, bool few, int shape, int lanes = 0) {
  a->rows = shape;
  a->lanes = lanes;
  int first[kMaxTokenBatch], last[kMaxTokenBatch];
  for (int i = 0; i < a->n; ++i) {
    TokenQuery& it = a->item[i];
    it.blocks = (it.n * a->group + shape - 1) / shape;   // (fewer than 2^27 rows in all)
    const auto block_tiles = [&](int b) {
      if (a->parents) return tok_tiles(it.pos0, it.pos0 + it.n - 1, a->window, a->sinks).n;
      const int r0 = b * shape, r1 = std::min(r0 + shape, it.n * a->group) - 1;
      return tok_tiles(it.pos0 + r0 / a->group, it.pos0 + r1 / a->group, a->window, a->sinks).n;
    };
    first[i] = block_tiles(0);
    last[i] = block_tiles(it.blocks - 1);
  }
  const int room = std::min<int>(kTokenScratchBytes / (shape * (kHeadDim + 2) * sizeof(float)), kTokenJoins);
  if (few) {
    const CtaCost cost{h->num_sms * token_few_ctas_per_sm(), token_few_tile_us(shape), 12, 4, 8, room, false};
    const double us = plan_splits(a, first, last, cost);
    int blocks = 0, most = 0;
    for (int i = 0; i < a->n; ++i) blocks += a->item[i].blocks, most = std::max(most, a->item[i].blocks);
    if (h->fp8 || most <= 2) return us;
    // bf16 pages: where several blocks read the same keys, a tile is the warps' own time, not the HBM's
    const double tile = std::max(kTokenFewSharedTileUs, cost.tile * a->n / blocks);
    return us / cost.tile * tile + cost.fixed * (cost.tile - tile);
  }
  int most = 0, splits = 1;
  for (int i = 0; i < a->n; ++i) most = std::max(most, a->item[i].n * a->group);
  const CtaCost cost{h->num_sms * token_tc_ctas_per_sm(lanes), token_tc_tile_us(h->fp8, shape, lanes, most),
                     10, 4, 8, room, true};
  const double us = plan_splits(a, first, last, cost) + token_tc_start_us(h->fp8, lanes, a->parents != nullptr);
  for (int i = 0; i < a->n; ++i) splits = std::max(splits, a->item[i].splits);
  return splits > 1 ? us + splits * kTokenSplitUs : us;
}

// Plans the matrix-unit kernel for a's streams: the shape of its CTAs, and the splits.
double plan_tc(pkv_t h, TokenAttendArgs* a) {
  long long most = 0;
  for (int i = 0; i < a->n; ++i) most = std::max(most, (long long)a->item[i].n * a->group);
  // one shape for all streams, the largest's: a second launch costs more than the lanes that
  // stay idle
  int shape = 128;
  while (shape < token_tc_max_rows(h->fp8) && most > shape) shape *= 2;
  // bf16 pages: blocks of 128 read a key once for fewer rows, but leave fewer lanes without rows
  // and end more evenly. Trees of up to 64 nodes, group 4, 256 / 128 rows: 32 streams of up to 2001
  // tokens 44 / 36 us, 8 of 4001 27 / 21 us, 16 of them 36 / 39 us; one of 131072 tokens, group 8,
  // 140 / 150 us.
  if (!h->fp8 && shape == 256) {
    const double narrow = plan_shape(h, a, false, 128, 2), wide = plan_shape(h, a, false, 256, 2);
    return wide <= narrow ? wide : plan_shape(h, a, false, 128, 2);
  }
  // 128 rows: two CTAs of two lanes an SM, or one of four (each with a quarter of the tiles)
  if (shape == 128) {
    const double four = plan_shape(h, a, false, 128, 4), two = plan_shape(h, a, false, 128, 2);
    return two < four ? two : plan_shape(h, a, false, 128, 4);
  }
  return plan_shape(h, a, false, shape, h->fp8 ? 4 : 2);
}

// The rotation as the kernel takes it.
pkv_status rotary_args(pkv_t h, const pkv_rotary* r, RotaryArgs* a) {
  if (!r) return fail(h, PKV_ERR_INVALID, "null rotary");
  if (r->axes < 1 || r->axes > kMaxAxes)
    return fail(h, PKV_ERR_INVALID, "%d position axes, not 1..%d", r->axes, kMaxAxes);
  const int d = r->pair_distance;
  if (d < 1 || d > kHeadDim / 2 || (d & (d - 1)) != 0)
    return fail(h, PKV_ERR_INVALID, "pair_distance %d is no power of two in 1..%d", d, kHeadDim / 2);
  std::memset(a, 0, sizeof(*a));
  a->axes = r->axes;
  a->distance = d;
  for (int i = 0; i < kHeadDim / 2; ++i) {
    if (r->axis[i] < 0 || r->axis[i] >= r->axes)
      return fail(h, PKV_ERR_INVALID, "pair %d: axis %d of %d", i, r->axis[i], r->axes);
    if (!(std::fabs(r->freq[i]) <= kMaxFreq))
      return fail(h, PKV_ERR_INVALID, "pair %d: a frequency of %g (at most %g in magnitude)", i, r->freq[i], kMaxFreq);
    a->turn[i] = rotary_turn(r->freq[i]);
    a->axis[i] = (uint8_t)r->axis[i];
  }
  return PKV_OK;
}

pkv_status check_rows(pkv_t h, int n, const int* sids, const int* row_off) {
  if (pkv_status r = check_batch(h, n, sids, row_off)) return r;
  return row_off ? PKV_OK : fail(h, PKV_ERR_INVALID, "null row_off");
}

// An append, with or without rotation (check_rows first).
pkv_status append_rows(pkv_t h, int n, const int* sids, const int* row_off, int layer, const void* k,
                       const void* v, long long k_stride, long long v_stride, const RotaryArgs* rotary,
                       void* cuda_stream) {
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
  cudaStream_t s = as_stream(cuda_stream);
  PKV_CUDA(h, rotary ? launch_token_append_rotary(a, *rotary, h->num_sms, s) : launch_token_append(a, s));
  if (layer == 0) {
    h->free_top -= (int)need;
    for (int i = 0; i < n; ++i)
      if (a.item[i].n > 0) tok_append(&h->streams[sids[i]].tok, a.item[i].n);
  }
  return PKV_OK;
}

// Attention of the streams' last tokens: in a row, or (parents) as trees (check_rows first).
pkv_status attend_rows(pkv_t h, const void* q, int q_heads, long long q_stride, const int* row_off,
                       const int* sids, int n, int layer, const int32_t* parents, void* out, int window,
                       int sinks, float sm_scale, void* cuda_stream) {
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
  a.parents = parents;
  a.q_stride = q_stride;
  a.heads = h->H;
  a.group = group;
  a.pool = pool_view(h, layer);
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = scale_log2;
  a.err = h->d_err;
  a.joined = h->d_joined;
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
  // the streams' rows per KV head decide on the kernel
  cudaStream_t s = as_stream(cuda_stream);
  const int n_items = a.n;
  long long rows_sum = 0;
  int n_all = 0, n_up_to = 0;                    // of up to kTokenFewRowsAll and kTokenFewRows rows
  for (int i = 0; i < n_items; ++i) {
    const long long r = (long long)a.item[i].n * group;
    if (r <= kTokenFewRowsAll) ++n_all;
    if (r <= kTokenFewRows) rows_sum += r, ++n_up_to;
  }
  const auto give_parts = [&](TokenAttendArgs* t) {
    bool split = false;
    for (int i = 0; i < t->n; ++i) split = split || t->item[i].splits > 1;
    t->part_o = split ? h->d_token_part : nullptr;
    t->part_ml = split ? h->d_token_part + (size_t)t->ctas * t->rows * kHeadDim : nullptr;
  };
  const auto launch_tc = [&](TokenAttendArgs* t) -> pkv_status {
    give_parts(t);
    PKV_CUDA(h, launch_token_tc(*t, s));
    if (t->part_o) PKV_CUDA(h, launch_token_combine(*t, s));
    return PKV_OK;
  };
  const auto launch_few = [&](TokenAttendArgs* t) -> pkv_status {
    give_parts(t);
    PKV_CUDA(h, launch_token_few(*t, s));
    return PKV_OK;
  };
  const auto plan_few = [&](TokenAttendArgs* t) {
    long long most = 0;
    for (int i = 0; i < t->n; ++i) most = std::max(most, (long long)t->item[i].n * group);
    if (most <= 8) return plan_shape(h, t, true, 8);
    // 17 to 24 rows: a block of 24 with three warps, or two of 16 with four, of which the second
    // finds the keys in L2. (21 rows, 24 / 16 + 16, pages not in L2: a stream of 16000 tokens 21.6 / 16.0
    // us, on E4M3 pages 25 / 19; 16 streams of 2000 19.6 / 16.2 us, of 16000 84 / 93, on E4M3 pages
    // 115 / 141; 48 ragged ones of up to 4000 49 / 44 us.)
    if (most > 16 && most <= 24) {
      const double two = plan_shape(h, t, true, 16), one = plan_shape(h, t, true, 24);
      if (one < two) return one;
    }
    return plan_shape(h, t, true, 16);
  };
  if (n_up_to == 0) {
    plan_tc(h, &a);
    return launch_tc(&a);
  }
  if (n_all == n_items) {
    plan_few(&a);
    return launch_few(&a);
  }
  // E4M3 pages: the kernel for few rows has f16 weights, the matrix-unit kernel bf16 ones, so what the
  // former takes of a call of pkv_attend_tokens does not go by speed alone: streams of up to
  // kTokenFewRowsAll rows, and of up to kTokenFewRows where these have no more than
  // kTokenFewRowsAll on average. (What that costs: 16 streams of 500 .. 4001 tokens with 4 .. 48
  // rows 36 against 32 us, with 4 .. 64 rows 46 against 33.)
  const bool f16_weights = h->fp8 && !parents;
  // Streams of both kinds: a launch for each, one behind the other, or (where weights may be bf16) all
  // in the matrix-unit kernel, as the estimates say (and 4 us for the launch). Ragged trees of up to 32
  // nodes, group 4: 16 streams of up to 4001 tokens 35 us in two launches, 25 in one; 32 of 4000 55 and
  // 45; 4 of 8000 29 and 20 us; on E4M3 pages 57 and 45, 90 and 77, 38 and 26 us.
  struct Division {
    TokenAttendArgs small, large;
    double us;
    bool together;
  };
  const double one = f16_weights ? 0.0 : plan_tc(h, &a);
  const auto divide = [&](Division* d, int few_rows) {
    std::memcpy(static_cast<void*>(&d->small), &a, offsetof(TokenAttendArgs, item));
    std::memcpy(static_cast<void*>(&d->large), &a, offsetof(TokenAttendArgs, item));
    d->small.n = d->large.n = 0;
    for (int i = 0; i < n_items; ++i) {
      TokenAttendArgs& t = (long long)a.item[i].n * group <= few_rows ? d->small : d->large;
      t.item[t.n++] = a.item[i];
    }
    const bool both = d->small.n > 0 && d->large.n > 0;
    // (where all are large, that is `one`)
    d->us = d->small.n == 0 && !f16_weights ? one
            : (d->small.n > 0 ? plan_few(&d->small) : 0.0) + (d->large.n > 0 ? plan_tc(h, &d->large) : 0.0) +
                  (both ? 4.0 : 0.0);
    d->together = !f16_weights && (d->small.n == 0 || (both && one <= d->us));
    if (d->together) d->us = one;
  };
  Division by[2], *best = &by[0];
  const bool up_to_64 = f16_weights && rows_sum <= (long long)kTokenFewRowsAll * n_up_to;
  divide(best, up_to_64 ? kTokenFewRows : kTokenFewRowsAll);
  if (!up_to_64 && n_up_to > n_all) {
    // 33 .. 64 rows: up to four blocks of 16 read the keys as often, from L2 but for the first
    divide(&by[1], kTokenFewRows);
    if (by[1].us <= best->us) best = &by[1];
  }
  if (best->together) return launch_tc(&a);
  if (best->small.n > 0)
    if (pkv_status r = launch_few(&best->small)) return r;
  return best->large.n > 0 ? launch_tc(&best->large) : PKV_OK;
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
  if (pkv_status r = check_rows(h, n, sids, row_off)) return r;
  return append_rows(h, n, sids, row_off, layer, k, v, k_stride, v_stride, nullptr, cuda_stream);
}

pkv_status pkv_append_tokens_rotary(pkv_t h, int n, const int* sids, const int* row_off, int layer,
                                    const void* k, const void* v, long long k_stride, long long v_stride,
                                    const void* q, int q_heads, long long q_stride, void* q_out,
                                    const void* positions, const pkv_rotary* rotary, void* cuda_stream) {
  if (pkv_status r = check_rows(h, n, sids, row_off)) return r;
  RotaryArgs a;
  if (pkv_status r = rotary_args(h, rotary, &a)) return r;
  if (q_heads < 0 || q_heads > kMaxGroup * h->H)
    return fail(h, PKV_ERR_INVALID, "q_heads %d outside 0..%d", q_heads, kMaxGroup * h->H);
  const int row = q_heads * kHeadDim;
  if (q_stride == 0) q_stride = row;
  if (pkv_status r = check_stride(h, "q_stride", q_stride, row)) return r;
  if (row_off[n] > 0) {
    if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u) != 0)
      return fail(h, PKV_ERR_INVALID, "positions must be a 4-byte aligned device pointer");
    if (q_heads > 0 && (misaligned(q) || misaligned(q_out)))
      return fail(h, PKV_ERR_INVALID, "q/q_out must be 16-byte aligned device pointers");
    if (q_heads > 0 && q == q_out && q_stride != row)
      return fail(h, PKV_ERR_INVALID, "q_out may be q only where q is contiguous");
  }
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_stride = q_stride;
  a.q_heads = q_heads;
  a.positions = static_cast<const int32_t*>(positions);
  return append_rows(h, n, sids, row_off, layer, k, v, k_stride, v_stride, &a, cuda_stream);
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

pkv_status pkv_keep_tokens(pkv_t h, int n, const int* sids, const int* row_off, const int* keep_off,
                           const void* kept, void* cuda_stream) {
  if (pkv_status r = check_batch(h, n, sids, row_off)) return r;
  if (!row_off || !keep_off) return fail(h, PKV_ERR_INVALID, "null offsets");
  if (keep_off[0] != 0) return fail(h, PKV_ERR_INVALID, "keep_off[0] must be 0");
  TokenKeepArgs a;
  std::memset(static_cast<void*>(&a), 0, offsetof(TokenKeepArgs, item));
  a.pool = pool_view(h, 0);
  a.layer_bytes = (long long)h->P * h->page_bytes;
  a.layers = h->L;
  a.kept = static_cast<const int32_t*>(kept);
  a.free_stack = h->d_free;
  a.top = h->free_top;
  a.err = h->d_err;
  int base = 0;
  // the last stream's pages first, as where they are dropped
  for (int i = n - 1; i >= 0; --i) {
    const Stream& st = h->streams[sids[i]];
    const TokenCounts& t = st.tok;
    const int rows = row_off[i + 1] - row_off[i];
    const long long m = (long long)keep_off[i + 1] - keep_off[i];
    if (m < 0 || m > rows)
      return fail(h, PKV_ERR_INVALID, "stream %d: %lld of %d tokens to keep", sids[i], m, rows);
    if (rows > t.len)
      return fail(h, PKV_ERR_INVALID, "stream %d: the last %d of its %d tokens", sids[i], rows, t.len);
    if (rows == 0) continue;
    if (!tok_can_drop(t, rows - (int)m) || !tok_has_last(t, rows))
      return fail(h, PKV_ERR_STATE, "stream %d: tokens that would stay or be seen are evicted", sids[i]);
    TokenKeepItem& it = a.item[a.n++];
    it.pages = st.d_pages;
    it.pos0 = t.len - rows;
    it.n = rows;
    it.m = (int)m;
    it.kept0 = keep_off[i];
    it.start = t.n_pages - 1;
    it.count = tok_drop_pages(t, rows - (int)m);
    it.base = base;
    base += it.count;
  }
  if (keep_off[n] > 0 && (!kept || (reinterpret_cast<uintptr_t>(kept) & 3u) != 0))
    return fail(h, PKV_ERR_INVALID, "kept must be a 4-byte aligned device pointer");
  if (h->free_top + base > h->P) return fail(h, PKV_ERR_STATE, "free stack overflow");
  if (keep_off[n] > 0 || base > 0) PKV_CUDA(h, launch_token_keep(a, as_stream(cuda_stream)));
  h->free_top += base;
  for (int i = 0; i < n; ++i) {
    const int rows = row_off[i + 1] - row_off[i];
    if (rows > 0) tok_drop(&h->streams[sids[i]].tok, rows - (keep_off[i + 1] - keep_off[i]));
  }
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
  if (pkv_status r = check_rows(h, n, sids, row_off)) return r;
  return attend_rows(h, q, q_heads, q_stride, row_off, sids, n, layer, nullptr, out, window, sinks, sm_scale,
                     cuda_stream);
}

pkv_status pkv_attend_tree(pkv_t h, const void* q, int q_heads, long long q_stride, const int* row_off,
                           const int* sids, int n, int layer, const void* parents, void* out, int window,
                           int sinks, float sm_scale, void* cuda_stream) {
  if (pkv_status r = check_rows(h, n, sids, row_off)) return r;
  if (row_off[n] > 0 && (!parents || (reinterpret_cast<uintptr_t>(parents) & 3u) != 0))
    return fail(h, PKV_ERR_INVALID, "parents must be a 4-byte aligned device pointer");
  for (int i = 0; i < n; ++i)
    if (row_off[i + 1] - row_off[i] > kTreeNodes)
      return fail(h, PKV_ERR_INVALID, "stream %d: a tree of %d nodes, more than %d", sids[i],
                  row_off[i + 1] - row_off[i], kTreeNodes);
  return attend_rows(h, q, q_heads, q_stride, row_off, sids, n, layer, static_cast<const int32_t*>(parents), out,
                     window, sinks, sm_scale, cuda_stream);
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
