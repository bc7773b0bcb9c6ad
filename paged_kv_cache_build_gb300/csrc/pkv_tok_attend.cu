// Causal attention of a token stream's last tokens over its pages, for few query
// rows per KV head: single tokens, drafted tokens to verify, short chunks. With a
// window, a query at position p sees j > p - window and j < sinks; always j <= p. TREE: the rows
// are the nodes of a drafted tree (pkv_attend_tree); what each sees of the tree's slots is walked
// out of the parents while the first tiles come (a tree of 16 nodes over 776 tokens 7.6 us,
// as a chain in the causal kernel 7.0).
//
//   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),   s_j = log2(e) sm_scale q . k_j
//
// in one pass over the keys, with the running maximum m. The query heads that share
// a KV head are rows of the same CTA, so a key is read once for all of them.
//
// Bounds: memory traffic; every visible K and V row is read once from HBM. One
// producer warp keeps a ring of 64-slot tiles filled by bulk copies (the pages are
// stored as ready operands, so a block of slots is one copy of K and one of V); each
// of four (three) warps takes every fourth (third) tile whole, holds its own m, sum and O,
// and they are joined at the end. Long tables are split over CTAs; the one that ends last
// of a row block's splits joins their partial results. The products run on warp-level matrix
// instructions with the 8, 16 or 24 query rows on the N side: S^T = K Q^T and
// O^T += V^T P^T.
// Measured: 32 streams of up to 8192 tokens, 32 query heads on 8, in 51.2 us on bf16 pages
// (6.0 TB/s, 0.89 of the measured copy rate) and in 38.2 us on E4M3 pages (4.1 TB/s: there
// the conversions' and the softmax' instruction latencies on eight warps an SM bound it; more
// warps with fewer registers, or two warps a tile, were no faster).
//
// bf16 pages: P is rounded to bf16 (2^-9 relative) for the second product. E4M3
// pages: codes are exact in f16, so both products run in f16 on the codes: q is
// scaled by a power of two per row into [1, 2) and rounded to f16 (exact but for
// elements 2^-14 below the row's largest), the K row's exponent is added to the
// score, and the V row's exponent is folded into P, which keeps a reference of its
// own: w_j = 2^(s_j + e_j - R), R the running maximum of s_j + e_j minus 15 (so that f16
// holds w from 2^15 down to 2^-24), O = 2^(R - m) sum_j w_j code_j. Rows of zeros are left
// out of R; any other row has a code of 224 or more (but for magnitudes near bf16's least),
// so what f16 loses is 2^-39 of a row's largest contribution.
#include "pkv_ptx.cuh"
#include "pkv_tokens.cuh"

#include <atomic>
#include <type_traits>

namespace pkv {

namespace {

// Consumer warps (and one producer). Up to 16 rows: four, at 168 registers a thread. 24 rows:
// three, so that two CTAs' warps have 255 (a fourth warp makes them spill: 4 % slower).
template <int NT>
constexpr int kWarps = NT <= 2 ? 4 : 3;
template <int NT>
constexpr int kThreads = (kWarps<NT> + 1) * 32;

template <bool FP8>
constexpr int kTileBytes = FP8 ? kTokTile * (kHeadDim + 1) : kTokTile * kHeadDim * 2;   // K or V
// Two CTAs an SM with about 96 KB of tiles each. (A third one on E4M3 pages, at 128
// registers, measured the same.)
constexpr int kCtasPerSm = 2;
template <bool FP8>
constexpr int kRing = FP8 ? 11 : 6;

struct NoTree {};

template <int NT, bool FP8, bool TREE>
struct __align__(1024) FewSmem {
  union {
    struct {
      uint8_t k[kRing<FP8>][kTileBytes<FP8>];
      uint8_t v[kRing<FP8>][kTileBytes<FP8>];
    };
    float o[kWarps<NT>][NT * 8][kHeadDim];           // after the last tile: the warps' O
  };
  float ml[kWarps<NT>][NT * 8][2];
  uint64_t full[kRing<FP8>];
  uint64_t empty[kRing<FP8>];
  std::conditional_t<TREE, TreeSmem<NT * 8>, NoTree> tree;
  int abort;
  int last;
};

__device__ __forceinline__ void mma_16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t pair) {   // the low two bytes
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(pair));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;\n" : "+r"(x));
  return x;
}
__device__ __forceinline__ float max8(float x) {   // over the 8 lanes of a query column
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

// Values d .. d + 3 of a row whose splits' partial results start at row pr0:
// o = sum_s 2^(m_s - M) o_s, l = sum_s 2^(m_s - M) l_s, M = max_s m_s, in order.
template <int kFold, typename Args>
__device__ __forceinline__ float4 join_splits(const Args& a, long long pr0, int splits, int d,
                                              float* l_out) {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < splits; s0 += kFold) {
    float2 ml[kFold];
    float4 ov[kFold];
#pragma unroll
    for (int k = 0; k < kFold; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      ov[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + k < splits) {
        const long long pr = pr0 + (long long)(s0 + k) * a.rows;
        ml[k] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + pr * 2));
        ov[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + pr * kHeadDim + d));
      }
    }
#pragma unroll
    for (int k = 0; k < kFold; ++k) {
      if (ml[k].y == 0.f) continue;              // every key masked (a sum that is no number is kept)
      const float m_new = fmaxf(m, ml[k].x);
      const float c = fast_exp2(m - m_new), w = fast_exp2(ml[k].x - m_new);
      l = l * c + w * ml[k].y;
      o.x = o.x * c + w * ov[k].x;
      o.y = o.y * c + w * ov[k].y;
      o.z = o.z * c + w * ov[k].z;
      o.w = o.w * c + w * ov[k].w;
      m = m_new;
    }
  }
  *l_out = l;
  return o;
}
// Values d .. d + 3 of the CTA's row r, divided by the row's sum.
template <typename Args>
__device__ __forceinline__ void write_row(const Args& a, const TokenQuery& t, const TokenWork& w, int r, int d,
                                          const float4& o, float l) {
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int rr = w.r0 + r;
  uint16_t* dst = a.out + ((long long)(t.row0 + rr / a.group) * a.heads * a.group + w.head * a.group +
                           rr % a.group) * kHeadDim + d;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

template <int NT, bool FP8, bool TREE, typename Args>
__global__ void __launch_bounds__(kThreads<NT>, kCtasPerSm) token_few_kernel(const __grid_constant__ Args a) {
  extern __shared__ uint8_t smem_raw[];
  FewSmem<NT, FP8, TREE>& sm = *reinterpret_cast<FewSmem<NT, FP8, TREE>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int kS = kRing<FP8>;
  static_assert(kS > kWarps<NT>, "the order of the stages' releases");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  __syncthreads();
  const TokenWork w = token_work<TREE>(a, blockIdx.x);
  const TokenQuery& t = a.item[w.item];
  const TokTiles tiles = tok_tiles(w.p0, w.p1, a.window, a.sinks);
  const int j0 = (int)((long long)tiles.n * w.split / t.splits);
  const int j1 = (int)((long long)tiles.n * (w.split + 1) / t.splits);
  const int nT = j1 - j0;
  const int Ps = a.pool.page_size;
  volatile int* abort = &sm.abort;
  pdl_wait();
  pdl_trigger();

  if (warp == kWarps<NT>) {
    // ---------------------------------------------------------------- producer
    // The page blocks of the next 32 / per tiles, one per lane: their addresses are
    // worked out together, and a tile then costs a wait and its lanes' copies.
    const int rows = min(Ps, kTokTile);                  // slots per block
    const int per = kTokTile / rows, group = 32 / per;
    const uint32_t block_bytes = (uint32_t)kTileBytes<FP8> / per;
    constexpr long long kRowBytes = FP8 ? kHeadDim + 1 : 2 * kHeadDim;
    const long long plane = (long long)Ps * kRowBytes;   // of a head's K or V in a page
    const uint32_t dst = (lane % per) * block_bytes;     // the lane's block in a tile
    int issued = 0;
    for (int base = 0; base < nT && issued == base; base += group) {
      const uint8_t* src = nullptr;
      if (base + lane / per < nT) {
        const int f = tok_tile(tiles, j0 + base + lane / per) * kTokTile + (lane % per) * rows;
        int page = t.pages[tok_block_entry(f, rows, w.p0, w.p1, a.window, a.sinks, Ps)];
        if (page < 0 || page >= a.pool.pool_pages) {
          atomicOr(a.err, kErrPageRange);
          page = 0;
        }
        src = reinterpret_cast<const uint8_t*>(a.pool.base) + (long long)page * a.pool.page_bytes +
              w.head * plane + (f % Ps) * kRowBytes;
      }
      const int end = min(nT, base + group);
      for (int j = base; j < end; ++j) {
        const int s = j % kS;
        if (!mbar_wait(&sm.empty[s], ((j / kS) & 1) ^ 1, abort, a.err)) break;
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[s], 2u * kTileBytes<FP8>);
        __syncwarp();
        if (lane / per == j - base) {
          const uint32_t bar = smem_u32(&sm.full[s]);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
                "[%3];\n" ::"r"(smem_u32(kv ? sm.v[s] : sm.k[s]) + dst),
                "l"(src + kv * a.pool.heads * plane), "r"(block_bytes), "r"(bar)
                : "memory");
        }
        issued = j + 1;
      }
    }
    // no copy may still be landing when the ring is used for the join
    if (lane == 0)
      for (int j = max(0, issued - kS); j < issued; ++j)
        mbar_wait(&sm.full[j % kS], (j / kS) & 1, abort, a.err, false);
  }

  const int g = lane >> 2, tq = lane & 3;
  float m[NT][2], l[NT][2], o[4][NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d][n][0] = o[d][n][1] = o[d][n][2] = o[d][n][3] = 0.f;
  }
  float ref[NT][2];                              // E4M3: R + 15
#pragma unroll
  for (int n = 0; n < NT; ++n) ref[n][0] = ref[n][1] = -INFINITY;

  if (warp < kWarps<NT>) {
    // Q^T as B operands (query g of each 8), rows behind the last one as zeros.
    // E4M3: the K codes of a row are read 16 bytes a lane, so the d of (step kk,
    // lane tq, i) is 16 tq + 4 kk + i; bf16: the operand's own order.
    uint32_t qb[NT][4][2];
    float sl2[NT][2];                            // score scale of queries 2 tq, 2 tq + 1
    int pos[NT][2];                              // trees: the row in the block instead
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = n * 8 + g;
      const int rr = w.r0 + r;
      const uint16_t* src = a.q + (t.row0 + rr / a.group) * a.q_stride +
                            (w.head * a.group + rr % a.group) * kHeadDim;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qb[n][kk][i] = r < w.rows ? __ldg(reinterpret_cast<const uint32_t*>(
                                          src + (FP8 ? 16 * tq + 4 * kk + 2 * i : 16 * kk + 8 * i + 2 * tq)))
                                    : 0u;
      int e = 0;
      if constexpr (FP8) {
        float big = 0.f;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            big = fmaxf(big, fabsf(__uint_as_float(qb[n][kk][i] << 16)));
            big = fmaxf(big, fabsf(__uint_as_float(qb[n][kk][i] & 0xFFFF0000u)));
          }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^e <= big < 2^(e + 1), |e| <= 126 so that both scales are normal
        e = (int)(__float_as_uint(big) >> 23) - 127;
        e = big == 0.f ? 0 : (e < -126 ? -126 : (e > 126 ? 126 : e));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qb[n][kk][i] = pack_f16(__uint_as_float(qb[n][kk][i] << 16) * inv,
                                    __uint_as_float(qb[n][kk][i] & 0xFFFF0000u) * inv);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int er = __shfl_sync(0xffffffffu, e, (2 * tq + i) * 4);
        sl2[n][i] = a.scale_log2 * __uint_as_float((uint32_t)(127 + er) << 23);
        const int rq = min(n * 8 + 2 * tq + i, w.rows - 1);
        pos[n][i] = TREE ? rq : t.pos0 + (w.r0 + rq) / a.group;
      }
    }
    if constexpr (TREE) {
      // what the rows see of the tree, if the CTA has a tile that some of them do not see whole
      if (a.window > 0 || (nT > 0 && tok_tile(tiles, j1 - 1) * kTokTile + kTokTile > t.pos0)) {
        load_parents(sm.tree, a.parents + t.row0, t.n, threadIdx.x, kWarps<NT> * 32, a.err);
        __syncwarp();
        asm volatile("bar.sync 1, %0;\n" ::"n"(kWarps<NT> * 32) : "memory");
        if (threadIdx.x < w.rows)
          walk_tree(sm.tree, threadIdx.x, (w.r0 + threadIdx.x) / a.group, t.pos0, a.window, a.sinks);
        __syncwarp();
        asm volatile("bar.sync 1, %0;\n" ::"n"(kWarps<NT> * 32) : "memory");
      }
    }

    for (int j = warp; j < nT; j += kWarps<NT>) {
      const int s = j % kS;
      // A stage passes between warps, and copies may land out of order: a parity
      // names the phase only once the one before it is over. The stage's last tile,
      // j - kS, is over when its warp has released it; the wait for that is exact,
      // because tile j - kWarps<NT>, which this warp has used, was issued after tile
      // j - kS, and so after tile j - 2 kS was released.
      if (j >= kS && !mbar_wait(&sm.empty[s], ((j / kS) & 1) ^ 1, abort, a.err)) break;
      if (!mbar_wait(&sm.full[s], (j / kS) & 1, abort, a.err)) break;
      const int b = tok_tile(tiles, j0 + j) * kTokTile;
      const uint8_t* kt = sm.k[s];
      const uint8_t* vt = sm.v[s];
      const int B = Ps >= kTokTile ? kTokTile : Ps;    // rows of an E4M3 block
      float sc[4][NT][4];                        // S^T: slot (16 sg +) g | g + 8, query 2 tq | + 1
      float ve[4][2];                            // E4M3: exponents of the V rows g, g + 8
      float prod = 1.f;                          // E4M3: of the exponents; 0 if one of them is 0
#pragma unroll
      for (int sg = 0; sg < 4; ++sg) {
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[sg][n][0] = sc[sg][n][1] = sc[sg][n][2] = sc[sg][n][3] = 0.f;
        if constexpr (FP8) {
          uint4 c[2];
          float ke[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 16 * sg + 8 * i + g, rb = r & (B - 1), blk = (r - rb) * (kHeadDim + 1);
            c[i] = *reinterpret_cast<const uint4*>(kt + blk + rb * kHeadDim + 16 * tq);
            ke[i] = __uint_as_float((uint32_t)(127 + (int8_t)kt[blk + B * kHeadDim + rb]) << 23);
            ve[sg][i] = (float)(int8_t)vt[blk + B * kHeadDim + rb];
            prod *= ve[sg][i];
          }
          const uint32_t c0[4] = {c[0].x, c[0].y, c[0].z, c[0].w};
          const uint32_t c1[4] = {c[1].x, c[1].y, c[1].z, c[1].w};
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t ka[4] = {codes_to_f16(c0[kk]), codes_to_f16(c1[kk]), codes_to_f16(c0[kk] >> 16),
                                    codes_to_f16(c1[kk] >> 16)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816_f16(sc[sg][n], ka, qb[n][kk][0], qb[n][kk][1]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[sg][n][e] *= ke[e >> 1];
        } else {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            uint32_t ka[4];
            ldsm_x4(sw_addr(smem_u32(kt), sg * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * kk + (lane >> 4)),
                    ka[0], ka[1], ka[2], ka[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(sc[sg][n], ka, qb[n][kk][0], qb[n][kk][1]);
          }
        }
      }
      if constexpr (FP8) {
        // A row of zeros is stored with exponent 0 (others have it for magnitudes of 224 and
        // more only). It brings nothing to O, so it must not raise R: its exponent is -inf.
        // (Looking for it costs 1.5 to 2 % of a call of single tokens; a product of the
        // exponents less than eight comparisons.)
        if (__any_sync(0xffffffffu, prod == 0.f)) {
          uint32_t zeros = 0;                    // bit 2 sg + i
#pragma unroll 1
          for (int u = 0; u < 8; ++u) {
            const int r = 8 * u + g, rb = r & (B - 1);
            const uint4 c = *reinterpret_cast<const uint4*>(vt + (r - rb) * (kHeadDim + 1) + rb * kHeadDim + 16 * tq);
            uint32_t any = (c.x | c.y | c.z | c.w) & 0x7F7F7F7Fu;
            any |= __shfl_xor_sync(0xffffffffu, any, 1);
            any |= __shfl_xor_sync(0xffffffffu, any, 2);
            if (any == 0u) zeros |= 1u << u;
          }
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if ((zeros >> u) & 1u) ve[u >> 1][u & 1] = -INFINITY;
        }
      }
      const bool full = TREE ? tree_tile_full(b, t.pos0, t.n, a.window, a.sinks)
                             : tok_tile_full(b, w.p0, w.p1, a.window, a.sinks);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int sg = 0; sg < 4; ++sg) {
            sc[sg][n][i] *= sl2[n][i];
            sc[sg][n][2 + i] *= sl2[n][i];
          }
          if (!full) {
            uint64_t bits;
            if constexpr (TREE)
              bits = tree_mask(b, t.pos0, sm.tree.depth[pos[n][i]], sm.tree.words[pos[n][i]], a.window, a.sinks);
            else
              bits = tok_mask(b, pos[n][i], a.window, a.sinks);
#pragma unroll
            for (int sg = 0; sg < 4; ++sg)
#pragma unroll
              for (int hi = 0; hi < 2; ++hi)
                if (!((bits >> (16 * sg + 8 * hi + g)) & 1ull)) sc[sg][n][2 * hi + i] = -INFINITY;
          }
          float mx = -INFINITY, rx = -INFINITY;
#pragma unroll
          for (int sg = 0; sg < 4; ++sg)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              const float x = sc[sg][n][2 * hi + i];
              mx = fmaxf(mx, x);
              if constexpr (FP8) rx = fmaxf(rx, x + ve[sg][hi]);
            }
          const float m_new = fmaxf(m[n][i], max8(mx));
          const float m_use = m_new == -INFINITY ? 0.f : m_new;
          const float alpha = fast_exp2(m[n][i] - m_use);
          m[n][i] = m_new;
          float o_alpha = alpha, r_use = 0.f;
          if constexpr (FP8) {
            const float r_new = fmaxf(ref[n][i], max8(rx));
            r_use = r_new == -INFINITY ? 0.f : r_new;
            o_alpha = fast_exp2(ref[n][i] - r_use);
            ref[n][i] = r_new;
          }
          float sum = 0.f;
#pragma unroll
          for (int sg = 0; sg < 4; ++sg)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              float& x = sc[sg][n][2 * hi + i];
              sum += fast_exp2(x - m_use);
              x = FP8 ? fast_exp2(x + ve[sg][hi] - (r_use - 15.f)) : fast_exp2(x - m_use);
            }
          l[n][i] = l[n][i] * alpha + sum;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            o[d][n][i] *= o_alpha;
            o[d][n][2 + i] *= o_alpha;
          }
        }
      // O^T += V^T P^T, 16 slots at a time
#pragma unroll
      for (int sg = 0; sg < 4; ++sg) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi)
            pb[n][hi] = transpose8(FP8 ? pack_f16(sc[sg][n][2 * hi], sc[sg][n][2 * hi + 1])
                                       : pack_bf16(sc[sg][n][2 * hi], sc[sg][n][2 * hi + 1]));
        if constexpr (FP8) {
          // Transposed 16-bit loads bring byte pairs (d, d + 1) of slots 2 tq, 2 tq + 1:
          // matrix i of the four is slots 8 (i & 1) .., 16 bytes i >> 1 of the half row.
          // Row g of the operand is d = 2 g, row g + 8 is d = 2 g + 1 of the 16.
          const int r = 16 * sg + (lane & 7) + ((lane >> 3) & 1) * 8, rb = r & (B - 1);
          const uint32_t row = smem_u32(vt) + (r - rb) * (kHeadDim + 1) + rb * kHeadDim + 16 * (lane >> 4);
#pragma unroll
          for (int d2 = 0; d2 < 2; ++d2) {
            uint32_t x[4];
            ldsm_x4_t(row + 32 * d2, x[0], x[1], x[2], x[3]);
#pragma unroll
            for (int dd = 0; dd < 2; ++dd) {
              const uint32_t lo = __byte_perm(x[2 * dd], 0u, 0x3120);       // slots 2 tq, + 1
              const uint32_t hi = __byte_perm(x[2 * dd + 1], 0u, 0x3120);   // and 8 further
              const uint32_t va[4] = {codes_to_f16(lo), codes_to_f16(lo >> 16), codes_to_f16(hi),
                                      codes_to_f16(hi >> 16)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_16816_f16(o[2 * d2 + dd][n], va, pb[n][0], pb[n][1]);
            }
          }
        } else {
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            uint32_t va[4];
            ldsm_x4_t(sw_addr(smem_u32(vt), sg * 16 + (lane & 7) + (lane >> 4) * 8, 2 * d + ((lane >> 3) & 1)),
                      va[0], va[1], va[2], va[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(o[d][n], va, pb[n][0], pb[n][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[s]);
    }
  }
  __syncthreads();                               // every tile is used: the ring is free

  // ---- join the warps
  if (warp < kWarps<NT>) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[n][i];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int r = n * 8 + 2 * tq + i;
        // E4M3: O moves to the reference m (in two steps: the factor alone may underflow)
        const float half = FP8 && m[n][i] != -INFINITY ? fast_exp2(0.5f * (ref[n][i] - 15.f - m[n][i])) : 1.f;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi)
            sm.o[warp][r][FP8 ? 16 * d + 2 * g + hi : 16 * d + g + 8 * hi] = o[d][n][2 * hi + i] * half * half;
        if (g == 0) {
          sm.ml[warp][r][0] = m[n][i];
          sm.ml[warp][r][1] = sum;
        }
      }
  }
  __syncthreads();
  // 16 lanes a row, 4 values a lane
  for (int x = threadIdx.x; x < w.rows * 16; x += kThreads<NT>) {
    const int r = x >> 4, d = (x & 15) * 4;
    float mm = -INFINITY;
#pragma unroll
    for (int i = 0; i < kWarps<NT>; ++i) mm = fmaxf(mm, sm.ml[i][r][0]);
    float ll = 0.f;
    float4 ov = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kWarps<NT>; ++i) {
      const float f = mm == -INFINITY ? 0.f : fast_exp2(sm.ml[i][r][0] - mm);
      const float4 p = *reinterpret_cast<const float4*>(&sm.o[i][r][d]);
      ll += f * sm.ml[i][r][1];
      ov.x += f * p.x;
      ov.y += f * p.y;
      ov.z += f * p.z;
      ov.w += f * p.w;
    }
    if (t.splits == 1) {
      write_row(a, t, w, r, d, ov, ll);
    } else {
      const long long pr = (long long)blockIdx.x * a.rows + r;
      __stcg(reinterpret_cast<float4*>(a.part_o + pr * kHeadDim + d), ov);
      if (d == 0) __stcg(reinterpret_cast<float2*>(a.part_ml + pr * 2), make_float2(mm, ll));
    }
  }
  if (t.splits == 1) return;
  // ---- the CTA that ends last of its splits joins them, in their order
  __threadfence();
  __syncthreads();
  const int cta0 = blockIdx.x - w.split;
  if (threadIdx.x == 0) {
    const unsigned before = atomicAdd(a.joined + cta0, 1u);
    sm.last = before == (unsigned)t.splits - 1u;
    if (sm.last) a.joined[cta0] = 0;             // for the next call
  }
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  for (int x = threadIdx.x; x < w.rows * 16; x += kThreads<NT>) {
    const int r = x >> 4, d = (x & 15) * 4;
    float l = 0.f;
    const float4 o = join_splits<12>(a, (long long)cta0 * a.rows + r, t.splits, d, &l);
    write_row(a, t, w, r, d, o, l);
  }
}

// For the matrix-unit kernel's splits: 8 threads a (token, query head), 8 values each.
// The partial results come from L2; loads of four splits are on their way at a time.
constexpr int kJoinFold = 4;
__global__ void __launch_bounds__(256, 4) token_combine_kernel(const __grid_constant__ TokenAttendArgs a, int pairs) {
  pdl_wait();
  pdl_trigger();
  const int gid = blockIdx.x * blockDim.x + threadIdx.x;
  const int pair = gid >> 3, d = (gid & 7) * 8;
  if (pair >= pairs) return;
  const int H = a.heads * a.group;
  const int tok = pair / H, qh = pair - tok * H, row = a.item[0].row0 + tok;
  const TokenQuery& t = a.item[find_item<TokenQuery, &TokenQuery::row0>(a.item, a.n, row)];
  const int splits = t.splits;
  if (row >= t.row0 + t.n || splits == 1) return;
  const int head = qh / a.group;
  const int r = (row - t.row0) * a.group + qh - head * a.group;
  const int block = r / a.rows;
  const int cta = t.cta0 + ((t.blocks - 1 - block) * a.heads + head) * splits;
  const long long pr0 = (long long)cta * a.rows + (r - block * a.rows);
  const float2* const ml = reinterpret_cast<const float2*>(a.part_ml) + pr0;
  const float* const part = a.part_o + pr0 * kHeadDim + d;
  float m = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < splits; s0 += kJoinFold) {
    float4 x[kJoinFold][2];
    float2 y[kJoinFold];
#pragma unroll
    for (int k = 0; k < kJoinFold; ++k) {
      y[k] = make_float2(-INFINITY, 0.f);
      x[k][0] = x[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + k < splits) {
        const long long at = (long long)(s0 + k) * a.rows;
        y[k] = __ldcg(ml + at);
        x[k][0] = __ldcg(reinterpret_cast<const float4*>(part + at * kHeadDim));
        x[k][1] = __ldcg(reinterpret_cast<const float4*>(part + at * kHeadDim + 4));
      }
    }
    float m_new = m;
#pragma unroll
    for (int k = 0; k < kJoinFold; ++k) m_new = fmaxf(m_new, y[k].x);
    const float ref = m_new == -INFINITY ? 0.f : m_new, c = fast_exp2(m - ref);
    m = m_new;
    l *= c;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= c;
#pragma unroll
    for (int k = 0; k < kJoinFold; ++k) {
      if (s0 + k >= splits) break;
      const float w = fast_exp2(y[k].x - ref);   // 0: the split's tiles are masked for the row
      l += w * y[k].y;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o[4 * i] += w * x[k][i].x;
        o[4 * i + 1] += w * x[k][i].y;
        o[4 * i + 2] += w * x[k][i].z;
        o[4 * i + 3] += w * x[k][i].w;
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint4*>(a.out + ((long long)row * H + qh) * kHeadDim + d) =
      make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                 pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
}

template <int NT, bool FP8, bool TREE, typename Args>
cudaError_t launch_few_args(const Args& a, cudaStream_t s) {
  constexpr int smem = (int)sizeof(FewSmem<NT, FP8, TREE>) + 1024;
  static_assert((smem + 1024) * kCtasPerSm <= 228 * 1024, "shared memory per SM");
  static std::atomic<unsigned long long> configured{0};   // a bit per device
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev >= 64 || !(configured.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(token_few_kernel<NT, FP8, TREE, Args>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured.fetch_or(bit);
  }
  const cudaError_t e = launch_pdl(token_few_kernel<NT, FP8, TREE, Args>, dim3(a.ctas), dim3(kThreads<NT>), smem, s, a);
  count_launches(1);
  return e;
}
template <int NT, bool FP8, bool TREE>
cudaError_t launch_few(const TokenAttendArgs& a, cudaStream_t s) {
  return a.n <= kSmallTokenBatch ? launch_few_args<NT, FP8, TREE>(small_args(a), s)
                                 : launch_few_args<NT, FP8, TREE>(a, s);
}
template <bool FP8, bool TREE>
cudaError_t launch_few_rows(const TokenAttendArgs& a, cudaStream_t s) {
  return a.rows == 8    ? launch_few<1, FP8, TREE>(a, s)
         : a.rows == 16 ? launch_few<2, FP8, TREE>(a, s)
                        : launch_few<3, FP8, TREE>(a, s);
}

}  // namespace

int token_few_ctas_per_sm() { return kCtasPerSm; }

cudaError_t launch_token_few(const TokenAttendArgs& a, cudaStream_t s) {
  if (a.parents) return a.pool.fp8 ? launch_few_rows<true, true>(a, s) : launch_few_rows<false, true>(a, s);
  return a.pool.fp8 ? launch_few_rows<true, false>(a, s) : launch_few_rows<false, false>(a, s);
}

cudaError_t launch_token_combine(const TokenAttendArgs& a, cudaStream_t s) {
  const TokenQuery& last = a.item[a.n - 1];
  // (rows x query heads fit 2^27: pkv_attend_tokens)
  const int pairs = (last.row0 + last.n - a.item[0].row0) * a.heads * a.group;
  const cudaError_t e = launch_pdl(token_combine_kernel, dim3((pairs + 31) / 32), dim3(256), 0, s, a, pairs);
  count_launches(1);
  return e;
}

}  // namespace pkv
