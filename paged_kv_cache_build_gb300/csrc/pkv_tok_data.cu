// Token streams: storing new tokens' keys and values (quantised on FP8 pages),
// reading them back, and returning dropped tokens' pages.
//
// Bounds: memory traffic (and, for single tokens, latency). 13754 tokens of 16 heads in 4
// streams on E4M3 pages are written and read back in 35 us, 4.9 TB/s (0.72 of the measured
// copy rate; a block's rounds of loads, quantising and stores overlap only with other
// blocks'). With few tokens a warp moves four consecutive ones of one (K or V, head): 8 lanes
// of 16 bytes a token. Their slots are neighbours in a page, so on E4M3 pages the warp writes
// one run of 256 code bytes and 4 neighbouring exponent bytes.
#include <algorithm>

#include "pkv_tokens.cuh"

namespace pkv {

namespace {

constexpr int kQuad = 4;             // tokens that a warp moves at a time
constexpr int kWarps = 8;

// Few rows: a warp per quad and plane.
template <typename Args>
__global__ void __launch_bounds__(kWarps * 32) token_append_kernel(const __grid_constant__ Args a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane & 7;
  const int H2 = 2 * a.pool.heads, Ps = a.pool.page_size;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int hh = (int)(w % H2);
  const long long unit = w / H2 * kQuad + (lane >> 3);
  if (unit >= a.units) return;                   // the same for the 8 lanes of a token
  const int kv = hh >= a.pool.heads ? 1 : 0, h = hh - kv * a.pool.heads;
  const TokenRows& it = a.item[find_item<TokenRows, &TokenRows::unit0>(a.item, a.n, (int)unit)];
  const int i = (int)unit - it.unit0, pos = it.pos0 + i;
  uint4 val = make_uint4(0u, 0u, 0u, 0u);
  if (i < it.n)
    val = __ldg(reinterpret_cast<const uint4*>((kv ? a.v : a.k) + (it.row0 + i) * (kv ? a.v_stride : a.k_stride) +
                                               h * kHeadDim + c * 8));
  const int pi = pos / Ps, slot = pos - pi * Ps;
  const int page = page_of(a, it, pi);
  if (page < 0) return;
  if (a.is_meta && slot == 0 && hh == 0 && c == 0) it.pages[pi] = page;
  store_row_chunk(a.pool, page, kv, h, slot, c, val);
}

// Two codes (the low bytes) to a bf16 pair times sc, a power of two. Exact: a code has
// 4 significant bits.
__device__ __forceinline__ uint32_t decode2(uint32_t pair, float sc) {
  uint32_t f, r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(f) : "h"((uint16_t)pair));
  float lo, hi;
  asm("{\n .reg .f16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
      : "=f"(lo), "=f"(hi)
      : "r"(f));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi * sc), "f"(lo * sc));
  return r;
}

// Chunk c (values 8 c .. 8 c + 7) of a stored row, as bf16.
__device__ __forceinline__ uint4 load_row_chunk(const PoolView& pv, int page, int kv, int head, int slot,
                                                int c) {
  if (!pv.fp8) {
    const uint16_t* row = pv.base + (long long)page * pv.page_elems +
                          ((long long)(kv * pv.heads + head) * pv.page_size + slot) * kHeadDim;
    return *reinterpret_cast<const uint4*>(row + swizzle_chunk(slot, c) * 8);
  }
  const uint2 codes = *reinterpret_cast<const uint2*>(fp8_row_codes(pv, page, kv, head, slot) + 8 * c);
  const int e = *fp8_row_exp(pv, page, kv, head, slot);
  const float sc = __uint_as_float((uint32_t)(127 + e) << 23);   // 2^e, |e| <= 126
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = decode2((i < 2 ? codes.x : codes.y) >> (16 * (i & 1)), sc);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename Args>
__global__ void __launch_bounds__(kWarps * 32) token_read_kernel(const __grid_constant__ Args a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane & 7;
  const int H2 = 2 * a.pool.heads, Ps = a.pool.page_size;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int hh = (int)(w % H2);
  const long long unit = w / H2 * kQuad + (lane >> 3);
  if (unit >= a.units) return;
  const int kv = hh >= a.pool.heads ? 1 : 0, h = hh - kv * a.pool.heads;
  const TokenRows& it = a.item[find_item<TokenRows, &TokenRows::unit0>(a.item, a.n, (int)unit)];
  const int i = (int)unit - it.unit0, pos = it.pos0 + i, pi = pos / Ps;
  const int page = page_of(a, it, pi);
  if (page < 0) return;
  uint16_t* const dst = (kv ? a.v : a.k) + ((long long)(it.row0 + i) * a.pool.heads + h) * kHeadDim + c * 8;
  *reinterpret_cast<uint4*>(dst) = load_row_chunk(a.pool, page, kv, h, pos - pi * Ps, c);
}

// Many rows: a block takes 32 tokens and works out their places in the pages once; its
// warps go over the (K or V, head) planes, the rows of two planes on their way before
// the first is stored.
constexpr int kManyTokens = 32;

// Places of a block's tokens in plane 0 (K of head 0): code or row, exponent byte, and
// the token's row in the packed tensors (-1: zeros).
struct Places {
  uint8_t* row[kManyTokens];         // null: no token
  uint8_t* exp[kManyTokens];
  int src[kManyTokens];
  int slot[kManyTokens];
};

template <bool READ>
__device__ __forceinline__ void find_places(const TokenRowsArgs& a, Places& p) {
  if (threadIdx.x < kManyTokens) {
    const int unit = blockIdx.x * kManyTokens + threadIdx.x, Ps = a.pool.page_size;
    uint8_t *row = nullptr, *exp = nullptr;
    int src = -1, slot = 0;
    if (unit < a.units) {
      const TokenRows& it = a.item[find_item<TokenRows, &TokenRows::unit0>(a.item, a.n, unit)];
      const int i = unit - it.unit0, pos = it.pos0 + i, pi = pos / Ps;
      const int page = page_of(a, it, pi);
      slot = pos - pi * Ps;
      if (i < it.n) src = it.row0 + i;
      if (page >= 0) {
        uint8_t* const base = reinterpret_cast<uint8_t*>(a.pool.base) + (long long)page * a.pool.page_bytes;
        row = base + (a.pool.fp8 ? fp8_code_off(a.pool.heads, Ps, 0, 0, slot) : (long long)slot * kHeadDim * 2);
        exp = base + fp8_exp_off(a.pool.heads, Ps, 0, 0, slot);
        if (!READ && a.is_meta && slot == 0) it.pages[pi] = page;
      }
    }
    p.row[threadIdx.x] = row;
    p.exp[threadIdx.x] = exp;
    p.src[threadIdx.x] = src;
    p.slot[threadIdx.x] = slot;
  }
  __syncthreads();
}

template <bool FP8>
__global__ void __launch_bounds__(kWarps * 32) token_append_many_kernel(const __grid_constant__ TokenRowsArgs a) {
  __shared__ Places p;
  pdl_wait();
  pdl_trigger();
  find_places<false>(a, p);
  const int lane = threadIdx.x & 31, c = lane & 7, t0 = lane >> 3, H = a.pool.heads;
  const long long plane = (long long)a.pool.page_size * (FP8 ? kHeadDim + 1 : 2 * kHeadDim);
  constexpr int kU = kManyTokens / kQuad;
  for (int hh = threadIdx.x >> 5; hh < 2 * H; hh += kWarps) {
    const int kv = hh >= H ? 1 : 0, h = hh - kv * H;
    const long long stride = kv ? a.v_stride : a.k_stride;
    const uint16_t* const rows = (kv ? a.v : a.k) + h * kHeadDim + c * 8;
    uint4 val[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int src = p.src[u * kQuad + t0];
      val[u] = make_uint4(0u, 0u, 0u, 0u);
      if (src >= 0) val[u] = __ldg(reinterpret_cast<const uint4*>(rows + src * stride));
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int t = u * kQuad + t0;
      uint8_t* const row = p.row[t];
      if (FP8) {
        int e;
        const uint2 codes = quantise8(val[u], &e);
        if (row) *reinterpret_cast<uint2*>(row + hh * plane + 8 * c) = codes;
        if (row && c == 0) p.exp[t][hh * plane] = (uint8_t)(int8_t)e;
      } else if (row) {
        *reinterpret_cast<uint4*>(row + hh * plane + (swizzle_chunk(p.slot[t], c) << 4)) = val[u];
      }
    }
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kWarps * 32) token_read_many_kernel(const __grid_constant__ TokenRowsArgs a) {
  __shared__ Places p;
  pdl_wait();
  pdl_trigger();
  find_places<true>(a, p);
  const int lane = threadIdx.x & 31, H = a.pool.heads;
  const long long plane = (long long)a.pool.page_size * (FP8 ? kHeadDim + 1 : 2 * kHeadDim);
  const long long stride = (long long)H * kHeadDim;
  // lanes of 16 bytes in the page: 4 a row of codes, 8 a row of bf16
  constexpr int kPer = FP8 ? 4 : 8, kRows = 32 / kPer, kU = kManyTokens / kRows;
  const int c = lane % kPer, t0 = lane / kPer;
  constexpr int kPlanes = FP8 ? 2 : 1;         // on their way at a time
  for (int h0 = (threadIdx.x >> 5) * kPlanes; h0 < 2 * H; h0 += kWarps * kPlanes) {
    uint4 val[kPlanes][kU];
    int exps[kPlanes];
#pragma unroll
    for (int q = 0; q < kPlanes; ++q) {        // 2 H planes: pairs are whole
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int t = u * kRows + t0;
        const uint8_t* const row = p.row[t] + (h0 + q) * plane;
        if (p.row[t])
          val[q][u] = *reinterpret_cast<const uint4*>(row + ((FP8 ? c : swizzle_chunk(p.slot[t], c)) << 4));
      }
      if (FP8) exps[q] = p.exp[lane] ? (int)(int8_t)p.exp[lane][(h0 + q) * plane] : 0;
    }
#pragma unroll
    for (int q = 0; q < kPlanes; ++q) {
      const int hh = h0 + q, kv = hh >= H ? 1 : 0, h = hh - kv * H;
      uint16_t* const rows = (kv ? a.v : a.k) + h * kHeadDim + c * (FP8 ? 16 : 8);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int t = u * kRows + t0;
        uint16_t* const dst = rows + p.src[t] * stride;
        if (FP8) {
          const int e = __shfl_sync(0xffffffffu, exps[q], t);
          const float sc = __uint_as_float((uint32_t)(127 + e) << 23);   // 2^e, |e| <= 126
          const uint32_t w[4] = {val[q][u].x, val[q][u].y, val[q][u].z, val[q][u].w};
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = decode2(w[i >> 1] >> (16 * (i & 1)), sc);
          if (p.row[t]) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(dst + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        } else if (p.row[t]) {
          *reinterpret_cast<uint4*>(dst) = val[q][u];
        }
      }
    }
  }
}

template <typename Args>
__global__ void __launch_bounds__(256) token_drop_kernel(const __grid_constant__ Args a) {
  pdl_wait();
  pdl_trigger();
  const TokenDropItem& it = a.item[blockIdx.x];
  for (int i = threadIdx.x; i < it.count; i += blockDim.x) {
    const int p = it.pages[it.start - i];
    if (p < 0 || p >= a.pool_pages) {
      atomicOr(a.err, kErrPageRange);
      continue;
    }
    a.free_stack[a.top + it.base + i] = p;
  }
}

// Accepted drafts move to the front of their tree's slots, in every layer; a block takes one
// (stream, layer, K or V, head), 16 rows a warp at a time, read before any of them is
// written. A row's destination is never behind its source, so what later rounds read is not
// overwritten. The blocks behind those return the dropped pages.
// Bounds: latency (a launch, then the loads of numbers, pages and rows, each behind the one
// before; every step's loads of a lane are on their way together). So a block has as many
// warps as hold the longest list at once, up to 8. Measured: 2.4 us for 4 of 16 nodes of one stream;
// 6.2 us for up to 40 of up to 200 nodes of 64 streams, 8 heads, 2 layers, E4M3 rows (5.3 MB).
constexpr int kKeepRows = 4;         // rows a lane has on their way
template <typename Args>
__global__ void __launch_bounds__(kWarps * 32) token_keep_kernel(const __grid_constant__ Args a, int move_blocks) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= move_blocks) {
    const TokenKeepItem& it = a.item[blockIdx.x - move_blocks];
    for (int i = threadIdx.x; i < it.count; i += blockDim.x) {
      const int p = it.pages[it.start - i];
      if (p < 0 || p >= a.pool.pool_pages) atomicOr(a.err, kErrPageRange);
      else a.free_stack[a.top + it.base + i] = p;
    }
    return;
  }
  const int c = threadIdx.x & 7, t0 = threadIdx.x >> 3, step = blockDim.x >> 3;
  const int H2 = 2 * a.pool.heads, Ps = a.pool.page_size, fp8 = a.pool.fp8;
  const int w = blockIdx.x, planes = a.layers * H2;
  const TokenKeepItem& it = a.item[w / planes];
  const int layer = w % planes / H2, hh = w % H2;
  const int B = fp8_block_rows(Ps);              // a power of two
  const long long plane = (long long)hh * Ps * (fp8 ? kHeadDim + 1 : 2 * kHeadDim);
  uint8_t* const base = reinterpret_cast<uint8_t*>(a.pool.base) + layer * a.layer_bytes + plane;
  const int32_t* const kept = a.kept + it.kept0;
  const bool notes = hh == 0 && layer == 0 && c == 0;
  // the lane's part of a slot's row in its page
  const auto part = [&](int slot) {
    const int rb = slot & (B - 1);
    return fp8 ? (slot - rb) * (kHeadDim + 1) + rb * kHeadDim + 8 * c
               : slot * kHeadDim * 2 + (swizzle_chunk(slot, c) << 4);
  };
  const auto exponent = [&](int slot) {
    const int rb = slot & (B - 1);
    return (slot - rb) * (kHeadDim + 1) + B * kHeadDim + rb;
  };
  for (int r0 = 0; r0 < it.m; r0 += step * kKeepRows) {
    int x[kKeepRows], before[kKeepRows], page[kKeepRows], to_page[kKeepRows];
    uint4 val[kKeepRows];
    int exp[kKeepRows];
#pragma unroll
    for (int u = 0; u < kKeepRows; ++u) {
      const int i = r0 + u * step + t0;
      x[u] = i < it.m ? kept[i] : i;
      before[u] = i < it.m && i > 0 ? kept[i - 1] : -1;
    }
#pragma unroll
    for (int u = 0; u < kKeepRows; ++u) {
      const int i = r0 + u * step + t0;
      const bool inside = x[u] >= i && x[u] < it.n;
      if (i < it.m && notes && (!inside || before[u] >= x[u])) atomicOr(a.err, kErrTree);
      if (i >= it.m || !inside) x[u] = i;        // stays
      page[u] = to_page[u] = 0;
      if (x[u] != i) {
        page[u] = it.pages[(it.pos0 + x[u]) / Ps];
        to_page[u] = it.pages[(it.pos0 + i) / Ps];
      }
    }
#pragma unroll
    for (int u = 0; u < kKeepRows; ++u) {
      const int i = r0 + u * step + t0;
      const bool there = (unsigned)page[u] < (unsigned)a.pool.pool_pages && (unsigned)to_page[u] < (unsigned)a.pool.pool_pages;
      if (!there) {
        if (notes) atomicOr(a.err, kErrPageRange);
        x[u] = i;
      }
      if (x[u] == i) continue;
      const int slot = (it.pos0 + x[u]) % Ps;
      const uint8_t* const from = base + (long long)page[u] * a.pool.page_bytes;
      if (fp8) {
        const uint2 v = *reinterpret_cast<const uint2*>(from + part(slot));
        val[u].x = v.x;
        val[u].y = v.y;
        exp[u] = from[exponent(slot)];
      } else {
        val[u] = *reinterpret_cast<const uint4*>(from + part(slot));
      }
    }
    __syncthreads();                             // read before written
#pragma unroll
    for (int u = 0; u < kKeepRows; ++u) {
      const int i = r0 + u * step + t0;
      if (x[u] == i) continue;
      const int slot = (it.pos0 + i) % Ps;
      uint8_t* const to = base + (long long)to_page[u] * a.pool.page_bytes;
      if (fp8) {
        *reinterpret_cast<uint2*>(to + part(slot)) = make_uint2(val[u].x, val[u].y);
        if (c == 0) to[exponent(slot)] = (uint8_t)exp[u];
      } else {
        *reinterpret_cast<uint4*>(to + part(slot)) = val[u];
      }
    }
    __syncthreads();
  }
}

// Tokens from which a block takes 32 of them: enough blocks to fill the SMs. (Read-back of
// 64 / 512 / 2560 / 4032 tokens of 8 heads on bf16 pages: 2.0 / 2.2 / 3.8 / 4.8 us with a
// warp per quad and plane, 4.7 / 3.6 / 3.6 / 3.7 us with blocks of 32. The rule asks for
// neither heads nor direction, and is off for some. From cold memory, each with a drop's
// launch of some 5 us in the appends, 2432 / 9728 tokens, quads against blocks: 8 heads, bf16
// append 10 / 17 against 18 / 20 us, read 10 / 14 against 11 / 13; E4M3 11 / 20 against
// 13 / 18 and 9 / 18 against 9 / 13; 32 heads, bf16 17 / 38 against 42 / 52 and 16 / 36
// against 18 / 34; E4M3 20 / 50 against 28 / 36 and 18 / 42 against 18 / 28 us.)
constexpr int kManyUnits = 152 * 16;

int row_blocks(const TokenRowsArgs& a) {
  const long long warps = ((long long)a.units + kQuad - 1) / kQuad * 2 * a.pool.heads;
  return (int)((warps + kWarps - 1) / kWarps);
}

using SmallRowsArgs = TokenRowsArgsOf<kSmallTokenBatch>;
using SmallDropArgs = TokenDropArgsOf<kSmallTokenBatch>;
using SmallKeepArgs = TokenKeepArgsOf<kSmallTokenBatch>;

}  // namespace

cudaError_t launch_token_append(const TokenRowsArgs& a, cudaStream_t s) {
  const dim3 threads(kWarps * 32);
  cudaError_t e;
  if (a.units >= kManyUnits) {
    auto* const kernel = a.pool.fp8 ? token_append_many_kernel<true> : token_append_many_kernel<false>;
    e = launch_pdl(kernel, dim3((a.units + kManyTokens - 1) / kManyTokens), threads, 0, s, a);
  } else if (a.n <= kSmallTokenBatch) {
    e = launch_pdl(token_append_kernel<SmallRowsArgs>, dim3(row_blocks(a)), threads, 0, s, small_args(a));
  } else {
    e = launch_pdl(token_append_kernel<TokenRowsArgs>, dim3(row_blocks(a)), threads, 0, s, a);
  }
  count_launches(1);
  return e;
}

cudaError_t launch_token_read(const TokenRowsArgs& a, cudaStream_t s) {
  const dim3 threads(kWarps * 32);
  cudaError_t e;
  if (a.units >= kManyUnits) {
    auto* const kernel = a.pool.fp8 ? token_read_many_kernel<true> : token_read_many_kernel<false>;
    e = launch_pdl(kernel, dim3((a.units + kManyTokens - 1) / kManyTokens), threads, 0, s, a);
  } else if (a.n <= kSmallTokenBatch) {
    e = launch_pdl(token_read_kernel<SmallRowsArgs>, dim3(row_blocks(a)), threads, 0, s, small_args(a));
  } else {
    e = launch_pdl(token_read_kernel<TokenRowsArgs>, dim3(row_blocks(a)), threads, 0, s, a);
  }
  count_launches(1);
  return e;
}

cudaError_t launch_token_drop(const TokenDropArgs& a, cudaStream_t s) {
  const dim3 threads(a.n > 4 ? 32 : 256);
  const cudaError_t e =
      a.n <= kSmallTokenBatch
          ? launch_pdl(token_drop_kernel<SmallDropArgs>, dim3(a.n), threads, 0, s, small_args(a))
          : launch_pdl(token_drop_kernel<TokenDropArgs>, dim3(a.n), threads, 0, s, a);
  count_launches(1);
  return e;
}

cudaError_t launch_token_keep(const TokenKeepArgs& a, cudaStream_t s) {
  int most = 1;
  for (int i = 0; i < a.n; ++i) most = std::max(most, a.item[i].m);
  const int blocks = a.n * a.layers * 2 * a.pool.heads;
  const int warps = std::min(kWarps, (most + kQuad * kKeepRows - 1) / (kQuad * kKeepRows));
  const dim3 grid(blocks + a.n), threads(warps * 32);
  const cudaError_t e =
      a.n <= kSmallTokenBatch
          ? launch_pdl(token_keep_kernel<SmallKeepArgs>, grid, threads, 0, s, small_args(a), blocks)
          : launch_pdl(token_keep_kernel<TokenKeepArgs>, grid, threads, 0, s, a, blocks);
  count_launches(1);
  return e;
}

}  // namespace pkv
