// Token streams: storing new tokens with rotary positions. Each row of q and k is 32 pairs of
// values, pair_distance apart, and each pair turns by the angle that its frequency and the
// token's position on its axis give:
//
//   y_a = x_a cos t - x_b sin t,   y_b = x_a sin t + x_b cos t,   t = freq position
//
// k goes to the pages (quantised on E4M3 pages), v beside it as it is, q to q_out.
//
// Angles: freq / 2 pi is kept as a 64-bit fraction of a turn, so position x fraction, cut to
// 64 bits, is the angle without its whole turns for any 32-bit position; fp32 enters only
// behind that. An fp32 product of frequency and position would be off by 2^-24 of the angle: a
// radian's tenth at a million.
//
// E4M3 pages: codes have 4 significant bits, so that an error of fp32's size in a value
// next to the border of two codes would show as a whole step. Values are rotated in fp32, and
// a row in which fp32's error could change a code or the exponent (some in 30,000 values) is
// rotated again in doubles.
//
// Bounds: memory traffic. A warp takes four tokens, whose sines and cosines its lanes hold in
// registers, and goes over planes (heads of q, K and V) of 128 bytes a token.
#include <algorithm>

#include "pkv_ptx.cuh"
#include "pkv_tokens.cuh"

namespace pkv {

namespace {

constexpr int kQuad = 4;             // tokens of a warp
constexpr int kWarps = 8;
constexpr int kFlight = 4;           // planes on their way

// The lane's share of a rotation: elements 8 c .. 8 c + 7 of a token's rows.
struct Turn {
  float cos[8], sin[8];              // sin with the sign of its element (first of a pair: -)
  uint32_t still;                    // bit i: element i's angle is 0, and rotation exact
};

// Element i of chunk c: the pair that it belongs to, and whether it is its second.
__device__ __forceinline__ int pair_of(int c, int i, int distance, bool* second) {
  const int e = 8 * c + i, in = e & (2 * distance - 1);
  *second = in >= distance;
  return (e - in) / 2 + (in & (distance - 1));
}

__device__ __forceinline__ unsigned long long phase_of(const RotaryArgs& r, const int32_t* position, int pair) {
  return (unsigned long long)(long long)position[r.axis[pair]] * r.turn[pair];
}

// The other elements of the lane's eight pairs.
__device__ __forceinline__ void partners(const float (&x)[8], int distance, float (&p)[8]) {
  if (distance >= 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __shfl_xor_sync(0xffffffffu, x[i], distance >> 3);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = distance == 1 ? x[i ^ 1] : distance == 2 ? x[i ^ 2] : x[i ^ 4];
  }
}

// A row whose codes fp32 does not settle: again in doubles, each code from the value rounded
// once. (A double goes to fp32 first: the neighbour on its side where that fell on the border of
// two codes, which has at most 5 significant bits.)
__device__ __noinline__ uint2 quantise_exactly(const RotaryArgs& r, const int32_t* position, int c, const float (&x)[8],
                                               const float (&p)[8], int* e_out) {
  double y[8], big = 0.0;
  for (int i = 0; i < 8; ++i) {
    bool second;
    const int pair = pair_of(c, i, r.distance, &second);
    double sn, cs;
    sincospi((double)(long long)phase_of(r, position, pair) * 0x1p-63, &sn, &cs);
    y[i] = fma((double)x[i], cs, (second ? sn : -sn) * (double)p[i]);
    big = fmax(big, fabs(y[i]));
  }
  const unsigned group = 0xFFu << (threadIdx.x & 24);
  for (int d = 1; d < 8; d <<= 1) big = fmax(big, __shfl_xor_sync(group, big, d));
  int e = 0;
  if (big > 0.0) {
    const double f = frexp(big, &e);
    e += -9 + (f > 0.875 ? 1 : 0);
    e = min(max(e, -126), 126);
  }
  *e_out = e;
  float z[8];
  for (int i = 0; i < 8; ++i) {
    const double v = ldexp(y[i], -e);
    z[i] = (float)v;
    const uint32_t b = __float_as_uint(z[i]);
    if ((b & 0x7FFFFu) == 0u && z[i] != 0.f && (double)z[i] != v)
      z[i] = __uint_as_float(fabs(v) > fabs((double)z[i]) ? b + 1u : b - 1u);
  }
  return make_uint2(fp8_pack2(z[0], z[1]) | (fp8_pack2(z[2], z[3]) << 16),
                    fp8_pack2(z[4], z[5]) | (fp8_pack2(z[6], z[7]) << 16));
}

template <bool FP8, typename Args>
__global__ void __launch_bounds__(kWarps * 32) token_append_rotary_kernel(const __grid_constant__ Args a,
                                                                          const __grid_constant__ RotaryArgs r,
                                                                          int shares) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane & 7;
  const int H = a.pool.heads, Ps = a.pool.page_size, planes = 2 * H + r.q_heads;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long unit = w / shares * kQuad + (lane >> 3);
  if (w / shares * kQuad >= a.units) return;     // the warp's tokens
  const int share = (int)(w % shares);
  const int h0 = (int)((long long)planes * share / shares), h1 = (int)((long long)planes * (share + 1) / shares);
  const bool there = unit < a.units;
  const TokenRows& it = a.item[find_item<TokenRows, &TokenRows::unit0>(a.item, a.n, (int)min(unit, a.units - 1ll))];
  const int i0 = there ? (int)unit - it.unit0 : it.n, pos = it.pos0 + i0;
  const bool row = i0 < it.n;                    // else a slot to be zeroed, or nothing
  const long long src = it.row0 + i0;
  // the token's place in plane 0 of its page
  int slot = 0, page = -1;
  if (there && (h0 < H || h1 > H + r.q_heads)) {
    const int pi = pos / Ps;
    slot = pos - pi * Ps;
    page = page_of(a, it, pi);
    if (a.is_meta && page >= 0 && slot == 0 && h0 == 0 && c == 0) it.pages[pi] = page;
  }
  const int32_t* const position = r.positions + src * r.axes;
  // planes: K, q, V; the last ones do not turn
  const int turning = H + r.q_heads;
  Turn t;
  t.still = 0;
  if (h0 < turning) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bool second;
      const int pair = pair_of(c, i, r.distance, &second);
      const unsigned long long phase = row ? phase_of(r, position, pair) : 0ull;
      if (phase == 0) t.still |= 1u << i;
      float sn;
      sincospif((float)(int)(phase >> 32) * 0x1p-31f, &sn, &t.cos[i]);
      t.sin[i] = second ? sn : -sn;
    }
  }
  uint8_t* const base = reinterpret_cast<uint8_t*>(a.pool.base) + (long long)max(page, 0) * a.pool.page_bytes;
  const long long plane = (long long)Ps * (FP8 ? kHeadDim + 1 : 2 * kHeadDim);
  const long long code = FP8 ? fp8_code_off(H, Ps, 0, 0, slot) + 8 * c
                             : (long long)slot * kHeadDim * 2 + (swizzle_chunk(slot, c) << 4);
  const long long exp = fp8_exp_off(H, Ps, 0, 0, slot);
  for (int hb = h0; hb < h1; hb += kFlight) {
    uint4 val[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int hh = hb + u;
      val[u] = make_uint4(0u, 0u, 0u, 0u);
      if (row && hh < h1) {
        const uint16_t* const from = hh < H         ? a.k + src * a.k_stride + hh * kHeadDim
                                     : hh < turning ? r.q + src * r.q_stride + (hh - H) * kHeadDim
                                                    : a.v + src * a.v_stride + (hh - turning) * kHeadDim;
        val[u] = *reinterpret_cast<const uint4*>(from + 8 * c);
      }
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int hh = hb + u;
      if (hh >= h1) break;
      const uint32_t b[4] = {val[u].x, val[u].y, val[u].z, val[u].w};
      float x[8], y[8], p[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(b[i] << 16);
        x[2 * i + 1] = __uint_as_float(b[i] & 0xFFFF0000u);
      }
      uint4 out = val[u];
      if (hh < turning) {
        partners(x, r.distance, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], t.cos[i], p[i] * t.sin[i]);
        out = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      }
      if (hh >= H && hh < turning) {
        if (row)
          *reinterpret_cast<uint4*>(r.q_out + (src * r.q_heads + hh - H) * kHeadDim + 8 * c) = out;
        continue;
      }
      const int hp = hh < H ? hh : hh - r.q_heads;   // plane of the page
      if constexpr (!FP8) {
        if (page >= 0) *reinterpret_cast<uint4*>(base + hp * plane + code) = out;
      } else {
        // what fp32 may be off by: 2^-20 (|x| + |p|), of a cosine and a sine off by 2^-22 and
        // three roundings
        const bool turned = hh < turning;
        float d[8], lo = 0.f, hi = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!turned) y[i] = x[i];
          d[i] = turned && !((t.still >> i) & 1u) ? (fabsf(x[i]) + fabsf(p[i])) * 0x1p-20f : 0.f;
          lo = fmaxf(lo, fabsf(y[i]) - d[i]);
          hi = fmaxf(hi, fabsf(y[i]) + d[i]);
        }
#pragma unroll
        for (int s = 1; s < 8; s <<= 1) {
          lo = fmaxf(lo, __shfl_xor_sync(0xffffffffu, lo, s));
          hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, s));
        }
        int e = fp8_row_exponent(hi);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t q[4];
        bool unsure = e != fp8_row_exponent(lo);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q[i] = fp8_pack2((y[2 * i] - d[2 * i]) * inv, (y[2 * i + 1] - d[2 * i + 1]) * inv);
          unsure |= q[i] != fp8_pack2((y[2 * i] + d[2 * i]) * inv, (y[2 * i + 1] + d[2 * i + 1]) * inv);
        }
        uint2 codes = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        if (turned && ((__ballot_sync(0xffffffffu, unsure) >> (lane & 24)) & 0xFFu))
          codes = quantise_exactly(r, position, c, x, p, &e);
        if (page >= 0) {
          *reinterpret_cast<uint2*>(base + hp * plane + code) = codes;
          if (c == 0) base[hp * plane + exp] = (uint8_t)(int8_t)e;
        }
      }
    }
  }
}

template <typename Args>
cudaError_t launch_rotary(const Args& a, const RotaryArgs& r, int blocks, int shares, cudaStream_t s) {
  return a.pool.fp8 ? launch_pdl(token_append_rotary_kernel<true, Args>, dim3(blocks), dim3(kWarps * 32), 0, s, a, r, shares)
                    : launch_pdl(token_append_rotary_kernel<false, Args>, dim3(blocks), dim3(kWarps * 32), 0, s, a, r, shares);
}

}  // namespace

cudaError_t launch_token_append_rotary(const TokenRowsArgs& a, const RotaryArgs& r, cudaStream_t s) {
  const long long quads = ((long long)a.units + kQuad - 1) / kQuad;
  const int planes = 2 * a.pool.heads + r.q_heads;
  // few tokens: a plane a warp; else enough warps for the SMs, so that angles are shared
  const long long want = 152 * 48;
  const int shares = (int)std::max<long long>(1, std::min<long long>(planes, want / quads));
  const int blocks = (int)((quads * shares + kWarps - 1) / kWarps);
  const cudaError_t e = a.n <= kSmallTokenBatch ? launch_rotary(small_args(a), r, blocks, shares, s)
                                                : launch_rotary(a, r, blocks, shares, s);
  count_launches(1);
  return e;
}

}  // namespace pkv
