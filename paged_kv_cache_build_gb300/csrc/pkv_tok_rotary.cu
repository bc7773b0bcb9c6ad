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
// doubles, one value in some 10,000: by a lane each, behind a warp's K planes, because one takes
// 1 to 2 us (a row of them in place 20 us, and the launch waited for it).
//
// Bounds: memory traffic. A warp takes four tokens, whose sines and cosines its lanes hold in
// registers, and goes over planes (heads of K, q and V) of 128 bytes a token, the next ones on
// their way while it turns these. Measured: 13754 tokens of 16 + 16 + 16 heads with three axes on
// bf16 pages in 28 us (169 MB, 6.0 TB/s, 0.90 of the measured copy rate); 10992 tokens on E4M3 pages
// in 28 us (113 MB, 4.0 TB/s): there the codes' arithmetic takes 62 % of the issue slots, with 18
// warps an SM to hide its latency.
#include <algorithm>

#include "pkv_ptx.cuh"
#include "pkv_tokens.cuh"

namespace pkv {

namespace {

constexpr int kQuad = 4;             // tokens of a warp
constexpr int kWarps = 4;
constexpr int kFlight = 8;           // planes on their way
constexpr int kPairs = kHeadDim / 2;

// Element i of chunk c: the pair that it belongs to, and whether it is its second.
__device__ __forceinline__ int pair_of(int c, int i, int distance, bool* second) {
  const int e = 8 * c + i, in = e & (2 * distance - 1);
  *second = in >= distance;
  return (e - in) / 2 + (in & (distance - 1));
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

// (x0, x1) y + (z0, z1), and without z, in one instruction.
__device__ __forceinline__ float2 fma2(float x0, float x1, float2 y, float2 z) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x0), "f"(x1), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float x0, float x1, float2 y) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x0), "f"(x1), "f"(y.x), "f"(y.y));
  return r;
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
__device__ __forceinline__ double power_of_two(int e) { return __hiloint2double((1023 + e) << 20, 0); }

// Cosine and sine of an angle of phase / 2^64 turns: whole quarters aside, their Taylor series
// within an eighth of a turn, whose next terms are 2^-58 and less. (In place of sincospi, of which a
// call's first use costs a microsecond, its code and constants being nowhere near.)
__device__ __forceinline__ void turn_exactly(unsigned long long phase, double* cs, double* sn) {
  const unsigned quarter = (unsigned)((phase + (1ull << 61)) >> 62) & 3u;
  const double a = (double)(long long)(phase - ((unsigned long long)quarter << 62)) * (6.283185307179586 * 0x1p-64);
  const double q = a * a;
  double s = 1.0 / 355687428096000.0, c = 1.0 / 20922789888000.0;   // 1 / 17!, 1 / 16!
  s = fma(s, q, -1.0 / 1307674368000.0);
  c = fma(c, q, -1.0 / 87178291200.0);
  s = fma(s, q, 1.0 / 6227020800.0);
  c = fma(c, q, 1.0 / 479001600.0);
  s = fma(s, q, -1.0 / 39916800.0);
  c = fma(c, q, -1.0 / 3628800.0);
  s = fma(s, q, 1.0 / 362880.0);
  c = fma(c, q, 1.0 / 40320.0);
  s = fma(s, q, -1.0 / 5040.0);
  c = fma(c, q, -1.0 / 720.0);
  s = fma(s, q, 1.0 / 120.0);
  c = fma(c, q, 1.0 / 24.0);
  s = fma(s, q, -1.0 / 6.0);
  c = fma(c, q, -0.5);
  s = fma(s * q, a, a);
  c = fma(c, q, 1.0);
  const double x = quarter & 1u ? s : c, y = quarter & 1u ? c : s;
  *cs = quarter == 1u || quarter == 2u ? -x : x;
  *sn = quarter & 2u ? -y : y;
}

// Element e of a row as rotated, in doubles: x is its value, p its pair's other one.
__device__ __noinline__ double turned_exactly(const RotaryArgs& r, const int32_t* position, int e, float x, float p) {
  bool second;
  const int pair = pair_of(0, e, r.distance, &second);
  const unsigned long long phase = (unsigned long long)(long long)position[r.axis[pair]] * r.turn[pair];
  if (phase == 0) return (double)x;
  double sn, cs;
  turn_exactly(phase, &cs, &sn);
  return fma((double)x, cs, (second ? sn : -sn) * (double)p);
}

// A value whose code fp32 leaves open, kept until the warp's K planes are done: then a lane each.
struct Open {
  uint32_t values;                   // bf16: the element's (low) and its pair's other one
  int plane;
  uint8_t token, element;            // of the warp's; of the row
  int8_t exponent;
};
constexpr int kOpen = 64;            // of a warp (what does not fit is settled at once)

template <bool FP8, typename Args>
__global__ void __launch_bounds__(kWarps * 32, FP8 ? 5 : 8)
    token_append_rotary_kernel(const __grid_constant__ Args a, const __grid_constant__ RotaryArgs r, int shares) {
  // each warp's: cosines and sines by [token][pair], and planes on their way, a lane's part in
  // its own place
  __shared__ __align__(16) float2 turns[kWarps][kQuad][kPairs + 2];
  __shared__ uint4 ring[kWarps][kFlight][32];
  __shared__ Open open_list[FP8 ? kWarps : 1][FP8 ? kOpen : 1];
  __shared__ int n_open[kWarps];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 7, q4 = lane >> 3;
  const int H = a.pool.heads, Ps = a.pool.page_size, planes = 2 * H + r.q_heads;
  const long long w = (long long)blockIdx.x * kWarps + warp;
  const long long unit = w / shares * kQuad + q4;
  if (unit - q4 >= a.units) return;              // the warp's tokens
  if (lane == 0) n_open[warp] = 0;
  const int share = (int)(w % shares);
  const int h0 = (int)((long long)planes * share / shares), h1 = (int)((long long)planes * (share + 1) / shares);
  const bool there = unit < a.units;
  const TokenRows& it = a.item[find_item<TokenRows, &TokenRows::unit0>(a.item, a.n, (int)min(unit, a.units - 1ll))];
  const int i0 = there ? (int)unit - it.unit0 : it.n, pos = it.pos0 + i0;
  const bool row = i0 < it.n;                    // else a slot to be zeroed, or nothing
  const long long src = row ? it.row0 + i0 : 0;
  // Planes: K, q, V; the last ones do not turn. Each lane has kFlight of its 16 bytes on their way.
  const int turning = H + r.q_heads;
  const uint16_t* from = (h0 < H         ? a.k + src * a.k_stride + h0 * kHeadDim
                          : h0 < turning ? r.q + src * r.q_stride + (h0 - H) * kHeadDim
                                         : a.v + src * a.v_stride + (h0 - turning) * kHeadDim) + 8 * c;
  const uint32_t place = smem_u32(&ring[warp][0][lane]);
  int next = h0;
  const auto fetch = [&]() {
    if (next < h1) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(place + (next - h0) % kFlight * 512),
                   "l"(row ? from : a.k), "r"(row ? 16 : 0)
                   : "memory");
      from += kHeadDim;
      if (++next == H) from = r.q + src * r.q_stride + 8 * c;
      if (next == turning) from = a.v + src * a.v_stride + 8 * c;
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
#pragma unroll 1
  for (int u = 0; u < kFlight; ++u) fetch();
  // the token's place in plane 0 of its page
  int slot = 0, page = -1;
  if (there && (h0 < H || h1 > turning)) {
    const int pi = pos / Ps;
    slot = pos - pi * Ps;
    page = page_of(a, it, pi);
    if (a.is_meta && page >= 0 && slot == 0 && h0 == 0 && c == 0) it.pages[pi] = page;
  }
  const int32_t* const position = r.positions + src * r.axes;
  float2 cs[4], sn[4];                           // sn with its element's sign (first of a pair: -)
  // fp32 is off by less than 2^-21 (|x| + |p|): an angle rounded to 2^-25 half turns, a sine
  // and a cosine off by 2^-24, and two roundings. Angles of 0 turn exactly, which matters: such
  // values may lie on the border of two codes, as many of a text's first token do.
  float off = 0.f;
  if (h0 < turning) {
    // a pair a lane, for each token; then every lane takes its elements' ones
    const unsigned long long turn = r.turn[lane];
    const int axis = r.axis[lane];
#pragma unroll
    for (int t = 0; t < kQuad; ++t) {
      const bool is_row = __shfl_sync(0xffffffffu, (int)row, 8 * t) != 0;
      const long long at = __shfl_sync(0xffffffffu, src, 8 * t) * r.axes + axis;
      const unsigned long long phase = is_row ? (unsigned long long)(long long)r.positions[at] * turn : 0ull;
      float2 x;                                  // (a cosine of 2 marks an angle of exactly 0)
      sincospif((float)(int)(phase >> 32) * 0x1p-31f, &x.y, &x.x);
      if (phase == 0) x.x = 2.f;
      turns[warp][t][lane] = x;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bool second;
      const float2 x = turns[warp][q4][pair_of(c, i, r.distance, &second)];
      if (x.x != 2.f) off = 0x1p-21f;
      const float y = second ? x.y : -x.y;
      if (i & 1) cs[i >> 1].y = fminf(x.x, 1.f), sn[i >> 1].y = y;
      else cs[i >> 1].x = fminf(x.x, 1.f), sn[i >> 1].x = y;
    }
  }
  uint8_t* const base = reinterpret_cast<uint8_t*>(a.pool.base) + (long long)max(page, 0) * a.pool.page_bytes;
  const long long plane = (long long)Ps * (FP8 ? kHeadDim + 1 : 2 * kHeadDim);
  // where the lane's part of the next plane goes: in the page, or (q) in q_out
  uint8_t* to = base + (h0 < H ? h0 : max(h0 - r.q_heads, H)) * plane +
                (FP8 ? fp8_code_off(H, Ps, 0, 0, slot) + 8 * c
                     : (long long)slot * kHeadDim * 2 + (swizzle_chunk(slot, c) << 4));
  const long long exp = fp8_exp_off(H, Ps, 0, 0, slot) - fp8_code_off(H, Ps, 0, 0, slot);   // (of chunk 0)
  uint16_t* q_to = r.q_out + (src * r.q_heads + max(h0 - H, 0)) * kHeadDim + 8 * c;
  // the next plane
  int at = 0;
  const auto take = [&]() {
    uint4 v;
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kFlight - 1) : "memory");
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(place + at % kFlight * 512)
                 : "memory");
    ++at;
    fetch();
    return v;
  };
  const auto turned = [&](const uint4& v, float (&x)[8], float (&p)[8], float2 (&y)[4]) {
    unpack(v, x);
    unpack(partners(v, r.distance), p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = fma2(x[2 * i], x[2 * i + 1], cs[i], mul2(p[2 * i], p[2 * i + 1], sn[i]));
  };
  const auto rounded = [&](const uint4& v) {
    float x[8], p[8];
    float2 y[4];
    turned(v, x, p, y);
    return make_uint4(pack_bf16(y[0].x, y[0].y), pack_bf16(y[1].x, y[1].y), pack_bf16(y[2].x, y[2].y),
                      pack_bf16(y[3].x, y[3].y));
  };
  const auto store8 = [&](const uint2& codes, int e) {
    if (page < 0) return;
    *reinterpret_cast<uint2*>(to) = codes;
    if (c == 0) to[exp] = (uint8_t)(int8_t)e;
  };
  int hh = h0;
#pragma unroll 1
  for (const int end = min(h1, H); hh < end; ++hh, to += plane) {
    const uint4 v = take();
    if constexpr (!FP8) {
      const uint4 out = rounded(v);
      if (page >= 0) *reinterpret_cast<uint4*>(to) = out;
    } else {
      float x[8], p[8], big = 0.f;
      float2 y[4];
      turned(v, x, p, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(y[i].x), fabsf(y[i].y)));
#pragma unroll
      for (int s = 1; s < 8; s <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, s));
      // The exponent (fp8_row_exponent): the bits' one, one more where the fraction is above
      // 0.75, a carry. A pair keeps its length, so |x| + |p| is at most twice the larger of its
      // two values: big is off by 2^-20 of it, 16 of its last places; 20 from a carry it is open.
      const uint32_t b = __float_as_uint(big) + 0x1FFFFFu;
      int e = big > 0.f ? max((int)(b >> 23) - 135, -126) : 0;
      const bool open = ((b + 20u) & 0x7FFFFFu) < 41u;
      if (__any_sync(0xffffffffu, open)) {
        // one value in doubles, or few, says whether the row's largest is above 448 x 2^e, e the
        // smaller of the two
        bool above = false;
        if (open) {
          e = max((int)((b - 20u) >> 23) - 135, -126);
          const double border = 448.0 * power_of_two(e);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (fabsf(i & 1 ? y[i >> 1].y : y[i >> 1].x) > big * (1.f - 0x1p-18f))
              above |= fabs(turned_exactly(r, position, 8 * c + i, x[i], p[i])) > border;
        }
        if ((__ballot_sync(0xffffffffu, above) >> (lane & 24)) & 0xFFu) ++e;
      }
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23), d = inv * off;
      uint32_t lo[4], differ[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s0 = fabsf(x[2 * i]) + fabsf(p[2 * i]), s1 = fabsf(x[2 * i + 1]) + fabsf(p[2 * i + 1]);
        // (a zero's sign goes, so that pairs of zeros are settled)
        const float2 z = fma2(y[i].x, y[i].y, make_float2(inv, inv), make_float2(0.f, 0.f));
        const float2 l = fma2(s0, s1, make_float2(-d, -d), z), h = fma2(s0, s1, make_float2(d, d), z);
        lo[i] = fp8_pack2(l.x, l.y);
        differ[i] = lo[i] ^ fp8_pack2(h.x, h.y);
      }
      uint2 codes = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
      if (differ[0] | differ[1] | differ[2] | differ[3]) {
        // the lane's open elements go to the list, for a lane each behind the K planes
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (((differ[i >> 1] >> (8 * (i & 1))) & 0xFFu) == 0) continue;
          const int k = atomicAdd(&n_open[warp], 1);
          if (k < kOpen) {
            Open o;
            o.values = (__float_as_uint(x[i]) >> 16) | (__float_as_uint(p[i]) & 0xFFFF0000u);
            o.plane = page >= 0 ? hh : -1;
            o.token = (uint8_t)q4;
            o.element = (uint8_t)(8 * c + i);
            o.exponent = (int8_t)e;
            open_list[warp][k] = o;
          } else {
            const double exact = turned_exactly(r, position, 8 * c + i, x[i], p[i]);
            const uint32_t sh = 8 * (i & 3);
            uint32_t& word = i < 4 ? codes.x : codes.y;
            word = (word & ~(0xFFu << sh)) | code_of(exact * power_of_two(-e)) << sh;
          }
        }
      }
      store8(codes, e);
    }
  }
  if constexpr (FP8) {
    // what is open, a lane each
    __syncwarp();
    const int n = min(n_open[warp], kOpen);
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += 32) {
      Open o;
      o.plane = -1;
      o.token = 0;
      if (k0 + lane < n) o = open_list[warp][k0 + lane];
      const long long token = __shfl_sync(0xffffffffu, src, 8 * o.token);
      uint8_t* const its_base = reinterpret_cast<uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(base), 8 * o.token));
      const int its_slot = __shfl_sync(0xffffffffu, slot, 8 * o.token);
      if (o.plane >= 0) {
        const double y = turned_exactly(r, r.positions + token * r.axes, o.element,
                                        __uint_as_float(o.values << 16), __uint_as_float(o.values & 0xFFFF0000u));
        its_base[o.plane * plane + fp8_code_off(H, Ps, 0, 0, its_slot) + o.element] =
            (uint8_t)code_of(y * power_of_two(-o.exponent));
      }
    }
  }
#pragma unroll 1
  for (const int end = min(h1, turning); hh < end; ++hh, q_to += kHeadDim) {
    const uint4 out = rounded(take());
    if (row) *reinterpret_cast<uint4*>(q_to) = out;
  }
#pragma unroll 1
  for (; hh < h1; ++hh, to += plane) {
    const uint4 v = take();
    if constexpr (FP8) {
      int e;
      const uint2 codes = quantise8(v, &e);
      store8(codes, e);
    } else if (page >= 0) {
      *reinterpret_cast<uint4*>(to) = v;
    }
  }
}

template <typename Args>
cudaError_t launch_rotary(const Args& a, const RotaryArgs& r, int blocks, int shares, cudaStream_t s) {
  return a.pool.fp8 ? launch_pdl(token_append_rotary_kernel<true, Args>, dim3(blocks), dim3(kWarps * 32), 0, s, a, r, shares)
                    : launch_pdl(token_append_rotary_kernel<false, Args>, dim3(blocks), dim3(kWarps * 32), 0, s, a, r, shares);
}

}  // namespace

cudaError_t launch_token_append_rotary(const TokenRowsArgs& a, const RotaryArgs& r, int num_sms, cudaStream_t s) {
  const long long quads = ((long long)a.units + kQuad - 1) / kQuad;
  const int planes = 2 * a.pool.heads + r.q_heads;
  // Equal shares of the planes for so many warps a quad. Angles cost a warp what 5 to 10 planes do, so
  // shares have kSharePlanes of them or more, but where that leaves an SM fewer than kFewWarps warps: there
  // latency counts (a plane a warp at the least). More warps than many_warps an SM bring nothing.
  // (Tokens x planes on bf16 pages, with 8 / 24 / 96 warps an SM: 300 x 48 4.9 / 6.2 / 6.7 us, 1000 x 48
  // 6.4 / 7.2 / 14.1, 3000 x 48 11.3 / 8.3 / 15.9, 10992 x 6 7.3 / 7.5 / 14.4, 13754 x 48 31.0 / 30.8 / 28.5; on
  // E4M3 pages 8.0 / 10.5 / 10.5, 10.6 / 11.3 / 18.8, 19.5 / 14.4 / 24.6, 11.2 / 11.3 / 21.6, 43.9 / 44.1 / 51.3.)
  constexpr int kSharePlanes = 12, kFewWarps = 8;
  const int many_warps = a.pool.fp8 ? 24 : 96;
  const long long few = std::min<long long>(planes, num_sms * kFewWarps / quads);
  const long long many = std::min<long long>(planes / kSharePlanes, (long long)num_sms * many_warps / quads);
  const int shares = (int)std::max({1ll, few, many});
  const int blocks = (int)((quads * shares + kWarps - 1) / kWarps);
  const cudaError_t e = a.n <= kSmallTokenBatch ? launch_rotary(small_args(a), r, blocks, shares, s)
                                                : launch_rotary(a, r, blocks, shares, s);
  count_launches(1);
  return e;
}

}  // namespace pkv
