// Token streams: storing new tokens' keys and values (quantised on FP8 pages),
// reading them back, and returning dropped tokens' pages.
//
// Bounds: memory traffic (and, for single tokens, latency). A warp moves four
// consecutive tokens of one (K or V, head): 8 lanes of 16 bytes a token. The
// tokens' slots are neighbours in a page, so on E4M3 pages the warp writes one run
// of 256 code bytes and 4 neighbouring exponent bytes.
#include "pkv_tokens.cuh"

namespace pkv {

namespace {

constexpr int kQuad = 4;             // tokens that a warp moves at a time
constexpr int kWarps = 8;

__device__ __forceinline__ int page_of(const TokenRowsArgs& a, const TokenRows& it, int pi) {
  const int page = a.is_meta && pi >= it.old_pages
                       ? a.free_stack[a.top - 1 - it.pop0 - (pi - it.old_pages)]
                       : it.pages[pi];
  if (page < 0 || page >= a.pool.pool_pages) {
    atomicOr(a.err, kErrPageRange);
    return -1;
  }
  return page;
}

// U quads per warp: the source rows of all of them are loaded before any is stored.
template <int U>
__global__ void __launch_bounds__(kWarps * 32) token_append_kernel(const __grid_constant__ TokenRowsArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane & 7;
  const int H2 = 2 * a.pool.heads, Ps = a.pool.page_size;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int hh = (int)(w % H2);
  const long long unit0 = w / H2 * (kQuad * U) + (lane >> 3);
  const int kv = hh >= a.pool.heads ? 1 : 0, h = hh - kv * a.pool.heads;
  const uint16_t* src = kv ? a.v : a.k;
  const long long stride = kv ? a.v_stride : a.k_stride;
  uint4 val[U];
  int at[U], pos[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long unit = unit0 + u * kQuad;
    at[u] = -1;
    val[u] = make_uint4(0u, 0u, 0u, 0u);
    if (unit >= a.units) continue;
    at[u] = find_item<TokenRows, &TokenRows::unit0>(a.item, a.n, (int)unit);
    const TokenRows& it = a.item[at[u]];
    const int i = (int)unit - it.unit0;
    pos[u] = it.pos0 + i;
    if (i < it.n)
      val[u] = __ldg(reinterpret_cast<const uint4*>(src + (it.row0 + i) * stride + h * kHeadDim + c * 8));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (at[u] < 0) continue;         // the same for the 8 lanes of a token
    const TokenRows& it = a.item[at[u]];
    const int pi = pos[u] / Ps, slot = pos[u] - pi * Ps;
    const int page = page_of(a, it, pi);
    if (page < 0) continue;
    if (a.is_meta && slot == 0 && hh == 0 && c == 0) it.pages[pi] = page;
    store_row_chunk(a.pool, page, kv, h, slot, c, val[u]);
  }
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
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = (uint16_t)((i < 2 ? codes.x : codes.y) >> (16 * (i & 1)));
    uint32_t f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(f) : "h"(pair));
    float lo, hi;
    asm("{\n .reg .f16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
        : "=f"(lo), "=f"(hi)
        : "r"(f));
    // exact: a code has 4 significant bits
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(w[i]) : "f"(hi * sc), "f"(lo * sc));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int U>
__global__ void __launch_bounds__(kWarps * 32) token_read_kernel(const __grid_constant__ TokenRowsArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane & 7;
  const int H2 = 2 * a.pool.heads, Ps = a.pool.page_size;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int hh = (int)(w % H2);
  const long long unit0 = w / H2 * (kQuad * U) + (lane >> 3);
  const int kv = hh >= a.pool.heads ? 1 : 0, h = hh - kv * a.pool.heads;
  uint4 val[U];
  long long row[U];
  int page[U], slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long unit = unit0 + u * kQuad;
    page[u] = -1;
    if (unit >= a.units) continue;
    const TokenRows& it = a.item[find_item<TokenRows, &TokenRows::unit0>(a.item, a.n, (int)unit)];
    const int i = (int)unit - it.unit0;
    const int pos = it.pos0 + i, pi = pos / Ps;
    slot[u] = pos - pi * Ps;
    row[u] = it.row0 + i;
    page[u] = page_of(a, it, pi);
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (page[u] >= 0) val[u] = load_row_chunk(a.pool, page[u], kv, h, slot[u], c);
  uint16_t* dst = kv ? a.v : a.k;
  const long long stride = (long long)a.pool.heads * kHeadDim;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (page[u] >= 0) *reinterpret_cast<uint4*>(dst + row[u] * stride + h * kHeadDim + c * 8) = val[u];
}

__global__ void __launch_bounds__(256) token_drop_kernel(const __grid_constant__ TokenDropArgs a) {
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

// Above this many (token, K or V, head) rows each warp takes several quads.
constexpr long long kManyRows = 152LL * 2 * kWarps * kQuad * 4;

template <int U>
int row_blocks(const TokenRowsArgs& a) {
  const long long warps = ((long long)a.units + kQuad * U - 1) / (kQuad * U) * 2 * a.pool.heads;
  return (int)((warps + kWarps - 1) / kWarps);
}

}  // namespace

cudaError_t launch_token_append(const TokenRowsArgs& a, cudaStream_t s) {
  const bool many = 2LL * a.units * a.pool.heads >= kManyRows;
  const cudaError_t e =
      many ? launch_pdl(token_append_kernel<4>, dim3(row_blocks<4>(a)), dim3(kWarps * 32), 0, s, a)
           : launch_pdl(token_append_kernel<1>, dim3(row_blocks<1>(a)), dim3(kWarps * 32), 0, s, a);
  count_launches(1);
  return e;
}

cudaError_t launch_token_read(const TokenRowsArgs& a, cudaStream_t s) {
  const bool many = 2LL * a.units * a.pool.heads >= kManyRows;
  const cudaError_t e =
      many ? launch_pdl(token_read_kernel<4>, dim3(row_blocks<4>(a)), dim3(kWarps * 32), 0, s, a)
           : launch_pdl(token_read_kernel<1>, dim3(row_blocks<1>(a)), dim3(kWarps * 32), 0, s, a);
  count_launches(1);
  return e;
}

cudaError_t launch_token_drop(const TokenDropArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(token_drop_kernel, dim3(a.n), dim3(a.n > 4 ? 32 : 256), 0, s, a);
  count_launches(1);
  return e;
}

}  // namespace pkv
