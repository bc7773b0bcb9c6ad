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
// those whose code (or a row whose exponent) fp32's error could change are rotated again in
// doubles: one value in 30,000.
//
// Bounds: memory traffic. A warp takes four tokens, whose sines and cosines its lanes hold in
// registers, and goes over planes (heads of K, q and V) of 128 bytes a token, the next ones on
// their way while it turns these.
#include <algorithm>

#include "pkv_ptx.cuh"
#include "pkv_tokens.cuh"

namespace pkv {

namespace {

constexpr int kQuad = 4;             // tokens of a warp
constexpr int kWarps = 8;
constexpr int kFlight = 4;           // planes on their way
constexpr int kPairs = kHeadDim / 2;

// Element i of chunk c: the pair that it belongs to, and whether it is its second.
__device__ __forceinline__ int pair_of(int c, int i, int distance, bool* second) {
  const int e = 8 * c + i, in = e & (2 * distance - 1);
  *second = in >= distance;
  return (e - in) / 2 + (in & (distance - 1));
}

__device__ __forceinline__ unsigned long long phase_of(const RotaryArgs& r, const int32_t* position, int pair) {
  return (unsigned long long)(long long)position[r.axis[pair]] * r.turn[pair];
}

// The chunk that holds the other elements of the lane's eight pairs (as many bf16 values).
__device__ __forceinline__ uint4 partners(const uint4& v, int distance) {
  if (distance >= 8) {
    const int m = distance >> 3;
    return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, m), __shfl_xor_sync(0xffffffffu, v.y, m),
                      __shfl_xor_sync(0xffffffffu, v.z, m), __shfl_xor_sync(0xffffffffu, v.w, m));
  }
  if (distance == 4) return make_uint4(v.z, v.w, v.x, v.y);
  if (distance == 2) return make_uint4(v.y, v.x, v.w, v.z);
  return make_uint4(__byte_perm(v.x, 0u, 0x1032), __byte_perm(v.y, 0u, 0x1032), __byte_perm(v.z, 0u, 0x1032),
                    __byte_perm(v.w, 0u, 0x1032));
}

__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(b[i] << 16);
    x[2 * i + 1] = __uint_as_float(b[i] & 0xFFFF0000u);
  }
}

// fp8_row_exponent of a largest magnitude by its bits: one more where the fraction is above
// 0.75, a carry.
__device__ __forceinline__ int row_exponent(float amax) {
  const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 135;
  return amax > 0.f ? min(max(e, -126), 126) : 0;
}

// One code of a double within 448, rounded once. (It goes to fp32 first: to the neighbour on its
// side where that fell on the border of two codes, which has at most 5 significant bits.)
__device__ __forceinline__ uint32_t code_of(double v) {
  float z = (float)v;
  const uint32_t b = __float_as_uint(z);
  if ((b & 0x7FFFFu) == 0u && z != 0.f && (double)z != v)
    z = __uint_as_float(fabs(v) > fabs((double)z) ? b + 1u : b - 1u);
  return fp8_pack2(z, 0.f) & 0xFFu;
}

// A rotated row (8 lanes') whose codes fp32 does not settle: the lane's elements whose code may
// differ, or all if the exponent is open, again in doubles. Called by the 8 lanes together.
__device__ __noinline__ uint2 settle(const RotaryArgs& r, const int32_t* position, int c, uint4 vx, uint4 vp, uint2 differ,
                                     bool open, uint2 codes, int* e_io) {
  float x[8], p[8];
  unpack(vx, x);
  unpack(vp, p);
  const auto value = [&](int i) {
    bool second;
    const int pair = pair_of(c, i, r.distance, &second);
    const unsigned long long phase = phase_of(r, position, pair);
    if (phase == 0) return (double)x[i];
    double sn, cs;
    sincospi((double)(long long)phase * 0x1p-63, &sn, &cs);
    return fma((double)x[i], cs, (second ? sn : -sn) * (double)p[i]);
  };
  int e = *e_io;
  if (open) {
    double big = 0.0;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) big = fmax(big, fabs(value(i)));
    const unsigned group = 0xFFu << (threadIdx.x & 24);
    for (int d = 1; d < 8; d <<= 1) big = fmax(big, __shfl_xor_sync(group, big, d));
    e = 0;
    if (big > 0.0) {
      const double f = frexp(big, &e);
      e = min(max(e - 9 + (f > 0.875 ? 1 : 0), -126), 126);
    }
    *e_io = e;
    differ.x = differ.y = ~0u;
  }
  unsigned long long all = codes.x | (unsigned long long)codes.y << 32;
  const unsigned long long which = differ.x | (unsigned long long)differ.y << 32;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    if (((which >> (8 * i)) & 0xFFull) == 0) continue;
    const unsigned long long code = code_of(ldexp(value(i), -e));
    all = (all & ~(0xFFull << (8 * i))) | code << (8 * i);
  }
  return make_uint2((uint32_t)all, (uint32_t)(all >> 32));
}

template <bool FP8, typename Args>
__global__ void __launch_bounds__(kWarps * 32, FP8 ? 3 : 4)
    token_append_rotary_kernel(const __grid_constant__ Args a, const __grid_constant__ RotaryArgs r, int shares) {
  // [token][pair] of each warp; a token's row is 17 float4 apart
  __shared__ __align__(16) float2 turns[kWarps][kQuad][kPairs + 2];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 7, q4 = lane >> 3;
  const int H = a.pool.heads, Ps = a.pool.page_size, planes = 2 * H + r.q_heads;
  const long long w = (long long)blockIdx.x * kWarps + warp;
  const long long unit = w / shares * kQuad + q4;
  if (unit - q4 >= a.units) return;              // the warp's tokens
  const int share = (int)(w % shares);
  const int h0 = (int)((long long)planes * share / shares), h1 = (int)((long long)planes * (share + 1) / shares);
  const bool there = unit < a.units;
  const TokenRows& it = a.item[find_item<TokenRows, &TokenRows::unit0>(a.item, a.n, (int)min(unit, a.units - 1ll))];
  const int i0 = there ? (int)unit - it.unit0 : it.n, pos = it.pos0 + i0;
  const bool row = i0 < it.n;                    // else a slot to be zeroed, or nothing
  const long long src = it.row0 + i0;
  // planes: K, q, V; the last ones do not turn
  const int turning = H + r.q_heads;
  const auto source = [&](int hh) {
    return (hh < H         ? a.k + src * a.k_stride + hh * kHeadDim
            : hh < turning ? r.q + src * r.q_stride + (hh - H) * kHeadDim
                           : a.v + src * a.v_stride + (hh - turning) * kHeadDim) + 8 * c;
  };
  // (the rows' first plane comes while the angles are worked out)
  if (row) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(source(h0)));
  // the token's place in plane 0 of its page
  int slot = 0, page = -1;
  if (there && (h0 < H || h1 > turning)) {
    const int pi = pos / Ps;
    slot = pos - pi * Ps;
    page = page_of(a, it, pi);
    if (a.is_meta && page >= 0 && slot == 0 && h0 == 0 && c == 0) it.pages[pi] = page;
  }
  const int32_t* const position = r.positions + src * r.axes;
  float cs[8], sn[8];                            // sn with its element's sign (first of a pair: -)
  if (h0 < turning) {
    // a pair a lane, for each token; then every lane takes its elements' ones
    const unsigned long long turn = r.turn[lane];
    const int axis = r.axis[lane];
#pragma unroll
    for (int t = 0; t < kQuad; ++t) {
      const bool is_row = __shfl_sync(0xffffffffu, (int)row, 8 * t) != 0;
      const long long at = __shfl_sync(0xffffffffu, src, 8 * t) * r.axes + axis;
      const unsigned long long phase = is_row ? (unsigned long long)(long long)r.positions[at] * turn : 0ull;
      float2 x;
      sincospif((float)(int)(phase >> 32) * 0x1p-31f, &x.y, &x.x);
      turns[warp][t][lane] = x;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bool second;
      const float2 x = turns[warp][q4][pair_of(c, i, r.distance, &second)];
      cs[i] = x.x;
      sn[i] = second ? x.y : -x.y;
    }
  }
  // Planes hh0 .. hh1 - 1, consecutive rows of `rows`, kFlight on their way at a time.
  const auto go = [&](int hh0, int hh1, const uint16_t* rows, auto&& take) {
    for (int hb = hh0; hb < hh1; hb += kFlight) {
      uint4 val[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        val[u] = make_uint4(0u, 0u, 0u, 0u);
        if (row && hb + u < hh1) val[u] = *reinterpret_cast<const uint4*>(rows + (hb + u - hh0) * kHeadDim);
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        if (hb + u < hh1) take(hb + u, val[u]);
    }
  };
  const auto turned = [&](const float (&x)[8], const float (&p)[8], float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], cs[i], p[i] * sn[i]);
  };
  const auto rounded = [&](const uint4& v) {
    const uint4 vp = partners(v, r.distance);
    float x[8], p[8], y[8];
    unpack(v, x);
    unpack(vp, p);
    turned(x, p, y);
    return make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
  };
  uint8_t* const base = reinterpret_cast<uint8_t*>(a.pool.base) + (long long)max(page, 0) * a.pool.page_bytes;
  const long long plane = (long long)Ps * (FP8 ? kHeadDim + 1 : 2 * kHeadDim);
  uint8_t* const code = base + (FP8 ? fp8_code_off(H, Ps, 0, 0, slot) + 8 * c
                                    : (long long)slot * kHeadDim * 2 + (swizzle_chunk(slot, c) << 4));
  const long long exp = fp8_exp_off(H, Ps, 0, 0, slot) - fp8_code_off(H, Ps, 0, 0, slot);   // (of chunk 0)
  const auto store8 = [&](int plane_no, const uint2& codes, int e) {
    if (page < 0) return;
    uint8_t* const to = code + plane_no * plane;
    *reinterpret_cast<uint2*>(to) = codes;
    if (c == 0) to[exp] = (uint8_t)(int8_t)e;
  };

  go(h0, min(h1, H), source(h0), [&](int hh, const uint4& v) {
    if constexpr (!FP8) {
      const uint4 out = rounded(v);
      if (page >= 0) *reinterpret_cast<uint4*>(code + hh * plane) = out;
    } else {
      const uint4 vp = partners(v, r.distance);
      float x[8], p[8], y[8];
      unpack(v, x);
      unpack(vp, p);
      turned(x, p, y);
      // fp32 is off by less than 2^-21 (|x| + |p|): an angle rounded to 2^-25 half turns, a sine
      // and a cosine off by 2^-24, and two roundings
      constexpr float kOff = 0x1p-21f;
      float big = 0.f, most = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        big = fmaxf(big, fabsf(y[i]));
        most = fmaxf(most, fabsf(x[i]));
      }
#pragma unroll
      for (int s = 1; s < 8; s <<= 1) {
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, s));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
      }
      const float off = most * (2.f * kOff);
      int e = row_exponent(big + off);
      const bool open = e != row_exponent(fmaxf(big - off, 0.f));
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23), d = inv * kOff;
      uint32_t lo[4], differ[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s0 = fabsf(x[2 * i]) + fabsf(p[2 * i]), s1 = fabsf(x[2 * i + 1]) + fabsf(p[2 * i + 1]);
        const float z0 = y[2 * i] * inv, z1 = y[2 * i + 1] * inv;
        lo[i] = fp8_pack2(fmaf(-d, s0, z0), fmaf(-d, s1, z1));
        differ[i] = lo[i] ^ fp8_pack2(fmaf(d, s0, z0), fmaf(d, s1, z1));
      }
      uint2 codes = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
      const uint2 other = make_uint2(differ[0] | (differ[1] << 16), differ[2] | (differ[3] << 16));
      const unsigned some = __ballot_sync(0xffffffffu, (other.x | other.y) != 0 || open);
      if ((some >> (lane & 24)) & 0xFFu) codes = settle(r, position, c, v, vp, other, open, codes, &e);
      store8(hh, codes, e);
    }
  });
  const int q0 = max(h0, H);
  uint16_t* const out_row = r.q_out + src * r.q_heads * kHeadDim + 8 * c;
  go(q0, min(h1, turning), source(q0), [&](int hh, const uint4& v) {
    const uint4 out = rounded(v);
    if (row) *reinterpret_cast<uint4*>(out_row + (hh - H) * kHeadDim) = out;
  });
  const int v0 = max(h0, turning);
  go(v0, h1, source(v0), [&](int hh, const uint4& v) {
    if constexpr (FP8) {
      int e;
      const uint2 codes = quantise8(v, &e);
      store8(hh - r.q_heads, codes, e);
    } else if (page >= 0) {
      *reinterpret_cast<uint4*>(code + (hh - r.q_heads) * plane) = v;
    }
  });
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
