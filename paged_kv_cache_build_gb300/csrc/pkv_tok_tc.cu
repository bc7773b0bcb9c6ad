// Causal attention of a token stream's last tokens over its pages on the
// 5th-generation tensor cores (tcgen05 + TMEM): chunks of a prompt, where a KV head
// has many query rows (tokens x query heads of the group).
//
//   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),   s_j = log2(e) sm_scale q . k_j
//
// Bounds: at head_dim 64 a 128 x 128 step is 512 cycles of the matrix unit (256 for
// each product) and 512 of the SM's 32 exponentials a cycle, so the softmax must run
// beside the products without a pause. A CTA has two lanes of 128 query rows, each
// with four softmax warps (a thread per row) and its own O in TMEM; the scores of
// their steps go round three TMEM buffers of 128 columns, so that a lane's next S
// is ready when it has written its P. The lanes are two blocks of 128 rows (MT = 2),
// or, for up to 128 rows, one block over every second step of the keys (MT = 1),
// joined at the end.
//
// The CTAs stay: each takes (row block, KV head, split) items from a counter until
// none is left, so that an item's queries, pages and first scores are under way while
// the one before it ends.
//
// Warps: 0-7 softmax (lane = warp / 4); 8 issues QK, 9 and 10 the lanes' PV: a warp
// that issues products spends most of its time in waits and in filling the matrix
// unit's queue, and one for all of them left the unit idle half the time; 11 the
// producer, which fills a ring of 128-slot K and V steps by bulk copies (pages are
// stored as ready operands); 12 the planner, which takes the items and loads their
// queries; on E4M3 pages the producer fills a ring of codes, and warps 13 on convert
// them into the operand ring (code * 2^e is exact in bf16).
//
// x counts the steps of both lanes in turn; step x uses S buffer x % 3, and P(x) is
// written over the first half of S(x). QK(x) waits for PV(x - 3), PV(x) for P(x).
// m is a reference that need not be the running maximum, for it
// cancels: it moves to the row's maximum on the first step and when a row's sum of a
// step exceeds 2^64, so that most steps take one pass over S. P is rounded to bf16
// (2^-9 relative) for the matrix unit; sums are taken before that rounding, in fp32.
// Every wait is bounded; one that gives up sets the device error word.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "pkv_ptx.cuh"
#include "pkv_tokens.cuh"

namespace pkv {

namespace {

constexpr int kLanes = 2;
constexpr int kStep = 2 * kTokTile;            // slots per step
constexpr int kSoftmaxWarps = 4 * kLanes;
constexpr int kIssueQK = kSoftmaxWarps;
constexpr int kIssuePV = kIssueQK + 1;
constexpr int kProducer = kIssuePV + kLanes;
constexpr int kPlanner = kProducer + 1;
constexpr int kConvert0 = kPlanner + 1;
template <bool FP8>
constexpr int kConvertWarps = FP8 ? 7 : 0;
template <bool FP8>
constexpr int kThreads = FP8 ? 32 * 20 : 32 * 16;
static_assert(kConvert0 + kConvertWarps<true> == 20, "whole warpgroups");
// Registers at launch, of which the others leave some to the softmax warpgroups.
template <bool FP8>
constexpr int kLaunchRegs = FP8 ? 96 : 128;
constexpr int kSoftmaxRegs = 168;
template <bool FP8>
constexpr int kOtherRegs = FP8 ? 48 : 88;
template <bool FP8>
constexpr bool kRegsFit = kSoftmaxRegs * kSoftmaxWarps + kOtherRegs<FP8> * (kThreads<FP8> / 32 - kSoftmaxWarps) <=
                          kLaunchRegs<FP8> * (kThreads<FP8> / 32);
static_assert(kRegsFit<false> && kRegsFit<true>, "the register split is within the launch's registers");
template <bool FP8>
constexpr int kRing = FP8 ? 3 : 4;
constexpr int kCodeRing = 3;
constexpr int kCodeBytes = kTokTile * (kHeadDim + 1);   // of K or V in a 64-slot tile
// TMEM: S buffer i at 128 i, O of lane i at 384 + 64 i
constexpr int kSBufs = 3;
constexpr uint32_t kTmemO = 384, kTmemCols = 512;
constexpr int kMaxFlags = 2048;                // steps whose flags are worked out beforehand
constexpr float kSumLimit = 18446744073709551616.0f;   // 2^64

// An item, as the roles read it.
struct Plan {
  int valid;                     // 0: no item is left
  int index;                     // its number: where its partial results go
  TokenWork work;
  TokTiles tiles;
  int j0, n_tiles;               // its 64-slot tiles; step i has tiles 2 i and 2 i + 1
  int row0, pos0, n_pages, splits;
  const int32_t* pages;
  TokSpan span[kLanes];          // what the lanes' rows see
};

template <int MT, bool FP8>
struct __align__(1024) TcSmem {
  uint8_t q[2][MT][128 * 128];
  uint8_t k[kRing<FP8>][kStep * 128];
  uint8_t v[kRing<FP8>][kStep * 128];
  float o[MT == 1 ? kHeadDim : 1][128];   // lane 1's part, for the join
  float ml[128][2];
  uint8_t code[FP8 ? kCodeRing : 1][FP8 ? 4 * kCodeBytes : 16];   // tile 0: K, V; tile 1: K, V
  uint64_t kv_full[kRing<FP8>];
  uint64_t kv_empty[kRing<FP8>];
  uint64_t code_full[kCodeRing];
  uint64_t code_empty[kCodeRing];
  uint64_t s_full[kSBufs];
  uint64_t p_full[kLanes][kSBufs];   // of the lane's step in the buffer
  uint64_t pv_done[kSBufs];
  uint64_t o_done[kLanes][2];    // the lane's PVs, in turn
  uint64_t plan_full[2];
  uint64_t plan_empty[2];
  uint64_t join_full[4];         // per row quarter
  uint64_t join_empty[4];
  uint64_t done[kLanes + 1];     // an issuer's products are all done (lanes' PV, QK)
  Plan plan[2];
  uint8_t flags[2][kMaxFlags];   // per step: see step_flags
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void fma2(float& a, float& b, float x, float y, float s, float c) {
  asm("{\n .reg .b64 d, m, k;\n mov.b64 d, {%2, %3};\n mov.b64 m, {%4, %4};\n mov.b64 k, {%5, %5};\n"
      " fma.rn.f32x2 d, d, m, k;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(a), "=f"(b)
      : "f"(x), "f"(y), "f"(s), "f"(c));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  asm("{\n .reg .b64 d, m;\n mov.b64 d, {%0, %1};\n mov.b64 m, {%2, %3};\n add.rn.f32x2 d, d, m;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

// An arrival without a branch around it.
__device__ __forceinline__ void mbar_arrive_if(uint64_t* bar, bool yes) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %1, 0;\n"
      " @p mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"((int)yes)
      : "memory");
}

// Four E4M3 codes to bf16 pairs times 2^e: a code's bits, shifted to bf16's places,
// are its value times 2^-120 (subnormal codes become bf16 subnormals), so one exact
// product with 2^(120 + e) remains, or two where that is no bf16 number (e > 7).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t w, bool high, uint32_t scale) {
  const uint32_t x = __byte_perm(w, 0u, high ? 0x3424 : 0x1404);   // the codes in the high bytes
  return mul_bf16x2((x & 0x80008000u) | ((x >> 4) & 0x07F007F0u), scale);
}

// What the lanes see of step i: bits 2 l: lane l needs it; 2 l + 1: it sees it whole.
__device__ __forceinline__ int step_flags(const TokTiles& tiles, int j0, int n_tiles, int i, const TokSpan& s0,
                                          const TokSpan& s1) {
  const int t0 = tok_tile(tiles, j0 + 2 * i);
  const bool two = 2 * i + 1 < n_tiles;
  const int t1 = two ? tok_tile(tiles, j0 + 2 * i + 1) : 0;
  const auto lane = [&](const TokSpan& s) {
    return (s.needs(t0) || (two && s.needs(t1)) ? 1 : 0) | (two && s.whole(t0) && s.whole(t1) ? 2 : 0);
  };
  return lane(s0) | lane(s1) << 2;
}

// A wait of a whole warp, with one outcome for all of it: control flow stays uniform.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  if (__all_sync(0xffffffffu, mbar_test(smem_u32(bar), parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
}

template <int MT, bool FP8>
__global__ void __launch_bounds__(kThreads<FP8>, 1) token_tc_kernel(const __grid_constant__ TokenAttendArgs a) {
  extern __shared__ uint8_t smem_raw[];
  TcSmem<MT, FP8>& sm = *reinterpret_cast<TcSmem<MT, FP8>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int kS = kRing<FP8>;
  // warp-uniform, and known to be
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(&sm.kv_full[s], FP8 ? kConvertWarps<FP8> : 1);
      mbar_init(&sm.kv_empty[s], MT);
    }
    for (int s = 0; s < kCodeRing; ++s) {
      mbar_init(&sm.code_full[s], 1);
      mbar_init(&sm.code_empty[s], FP8 ? kConvertWarps<FP8> : 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&sm.s_full[i], 1);
      for (int l = 0; l < kLanes; ++l) mbar_init(&sm.p_full[l][i], 4);
      mbar_init(&sm.pv_done[i], 1);
    }
    for (int l = 0; l < kLanes; ++l)
      for (int i = 0; i < 2; ++i) mbar_init(&sm.o_done[l][i], 1);
    for (int l = 0; l <= kLanes; ++l) mbar_init(&sm.done[l], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.plan_full[i], 1);
      // softmax, QK (its commit), PV, producer, converters
      mbar_init(&sm.plan_empty[i], kSoftmaxWarps + 1 + kLanes + 1 + kConvertWarps<FP8>);
    }
    for (int q = 0; q < 4; ++q) {
      mbar_init(&sm.join_full[q], 1);
      mbar_init(&sm.join_empty[q], 1);
    }
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kIssueQK) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  volatile int* abort = &sm.abort;
  const int G = a.group;
  const auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  // the n-th item's plan, once it is there; null: none is left, or a wait gave up
  const auto next_plan = [&](int n) -> const Plan* {
    if (!mbar_wait_warp(&sm.plan_full[n & 1], (n >> 1) & 1, abort, a.err)) return nullptr;
    const Plan* p = &sm.plan[n & 1];
    return uniform(p->valid) ? p : nullptr;
  };
  // x counts an item's lane steps: an even number, so that the lanes take turns from
  // item to item (MT = 1: a last one may be empty)
  const auto lane_steps = [](int steps) { return MT == 2 ? 2 * steps : (steps + 1) & ~1; };
  pdl_wait();
  pdl_trigger();

  if (warp >= kProducer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs<FP8>));
    if (warp == kPlanner) {
      // -------------------------------------------------------------- planner
      int index = blockIdx.x;
      for (int n = 0;; ++n) {
        int next = 0;
        if (lane == 0 && index < a.ctas) next = gridDim.x + (int)atomicAdd(a.tickets, 1u);
        if (!mbar_wait_warp(&sm.plan_empty[n & 1], ((n >> 1) & 1) ^ 1, abort, a.err)) break;
        Plan& p = sm.plan[n & 1];
        if (index >= a.ctas) {
          if (lane == 0) p.valid = 0;
          __syncwarp();
          mbar_arrive_if(&sm.plan_full[n & 1], lane == 0);
          break;
        }
        const TokenWork w = token_work(a, index);
        const TokenQuery& t = a.item[w.item];
        const TokTiles tiles = tok_tiles(w.p0, w.p1, a.window, a.sinks);
        const int steps = (tiles.n + 1) / 2;
        const int j0 = 2 * (int)((long long)steps * w.split / t.splits);
        const int n_tiles = min(tiles.n, 2 * (int)((long long)steps * (w.split + 1) / t.splits)) - j0;
        TokSpan span[kLanes];
#pragma unroll
        for (int l = 0; l < kLanes; ++l) {
          const int r0 = w.r0 + (MT == 2 ? 128 * l : 0), rows = min(128, w.r0 + w.rows - r0);
          span[l] = tok_span(t.pos0 + r0 / G, t.pos0 + (r0 + max(rows, 1) - 1) / G, a.window, a.sinks);
          if (rows <= 0) {             // nothing is needed, nothing whole
            span[l].hi = -1;
            span[l].f1 = 0;
          }
        }
        if (lane == 0) {
          p.valid = 1;
          p.index = index;
          p.work = w;
          p.tiles = tiles;
          p.j0 = j0;
          p.n_tiles = n_tiles;
          p.row0 = t.row0;
          p.pos0 = t.pos0;
          p.n_pages = t.n_pages;
          p.splits = t.splits;
          p.pages = t.pages;
          for (int l = 0; l < kLanes; ++l) p.span[l] = span[l];
        }
        for (int i = lane; 2 * i < n_tiles && i < kMaxFlags; i += 32)
          sm.flags[n & 1][i] = (uint8_t)step_flags(tiles, j0, n_tiles, i, span[0], span[1]);
        // Q rows as swizzled operand tiles, 4 rows of 8 chunks at a time; rows behind
        // the last one as zeros
        int tok = (w.r0 + (lane >> 3)) / G, mem = (w.r0 + (lane >> 3)) % G;
        const int dt = 4 / G, dm = 4 % G, c = lane & 7;
        for (int r = lane >> 3; r < MT * 128; r += 4) {
          const bool there = r < w.rows;
          const uint16_t* src = a.q + (there ? (t.row0 + tok) * a.q_stride + (w.head * G + mem) * kHeadDim + c * 8 : 0);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                           smem_u32(&sm.q[n & 1][r >> 7][(r & 127) * 128 + (swizzle_chunk(r & 7, c) << 4)])),
                       "l"(src), "r"(there ? 16 : 0)
                       : "memory");
          tok += dt;
          mem += dm;
          if (mem >= G) {
            mem -= G;
            ++tok;
          }
        }
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        fence_proxy_async();
        __syncwarp();
        mbar_arrive_if(&sm.plan_full[n & 1], lane == 0);
        index = uniform(next);
      }
      // the CTA that ends last puts the counters back
      if (lane == 0 && atomicAdd(a.tickets + 1, 1u) == gridDim.x - 1) {
        a.tickets[0] = 0;
        a.tickets[1] = 0;
      }
    } else if (warp == kProducer) {
      // ------------------------------------------------------------- producer
      const int Ps = a.pool.page_size;
      // The page blocks of the next 32 / per steps, one per lane: their addresses are
      // worked out together, and a step then costs a wait and its lanes' copies.
      const int rows = min(Ps, kTokTile);                // slots per block
      const int half_blocks = kTokTile / rows, per = 2 * half_blocks, group = 32 / per;
      constexpr uint32_t kOperand = FP8 ? kCodeBytes : kTokTile * 128;   // bytes of K or V in a tile
      constexpr int kRingN = FP8 ? kCodeRing : kS;
      uint64_t* const full = FP8 ? sm.code_full : sm.kv_full;
      uint64_t* const empty = FP8 ? sm.code_empty : sm.kv_empty;
      const uint32_t block_bytes = kOperand / half_blocks;
      constexpr long long kRowBytes = FP8 ? kHeadDim + 1 : 2 * kHeadDim;
      const long long plane = (long long)Ps * kRowBytes; // of a head's K or V in a page
      // the lane's block: of the step's tile `half`, its pp-th
      const int half = lane % per / half_blocks, pp = lane % half_blocks;
      int g = 0;                                         // steps of all items so far
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Plan* p = next_plan(n);
        if (!p) break;
        const int nT = p->n_tiles, j0 = p->j0, nS = (nT + 1) / 2;
        const TokTiles tiles = p->tiles;
        for (int base = 0; ok && base < nS; base += group) {
          const uint8_t* src = nullptr;
          if (base + lane / per < nS) {
            // a last step of one tile takes it twice: the second is masked
            const int j = min(2 * (base + lane / per) + half, nT - 1);
            const int f = tok_tile(tiles, j0 + j) * kTokTile + pp * rows;
            // blocks behind the last page repeat it: their slots are masked
            const int e = f / Ps;
            int page = p->pages[min(e, p->n_pages - 1)];
            if (page < 0 || page >= a.pool.pool_pages) {
              atomicOr(a.err, kErrPageRange);
              page = 0;
            }
            src = reinterpret_cast<const uint8_t*>(a.pool.base) + (long long)page * a.pool.page_bytes +
                  p->work.head * plane + (f - e * Ps) * kRowBytes;
          }
          const int end = min(nS, base + group);
          for (int i = base; i < end; ++i, ++g) {
            const int s = g % kRingN;
            ok = mbar_wait_warp(&empty[s], ((g / kRingN) & 1) ^ 1, abort, a.err);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], 4u * kOperand);
            __syncwarp();
            if (lane / per == i - base) {
              const uint32_t bar = smem_u32(&full[s]);
#pragma unroll
              for (int kv = 0; kv < 2; ++kv) {
                uint8_t* dst = FP8 ? sm.code[s] + (2 * half + kv) * kCodeBytes
                                   : (kv ? sm.v[s] : sm.k[s]) + half * kTokTile * 128;
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
                    "[%3];\n" ::"r"(smem_u32(dst + pp * block_bytes)),
                    "l"(src + kv * a.pool.heads * plane), "r"(block_bytes), "r"(bar)
                    : "memory");
              }
            }
          }
        }
        __syncwarp();
        mbar_arrive_if(&sm.plan_empty[n & 1], lane == 0);
      }
      // no copy may still be landing when the CTA ends
      if (lane == 0)
        for (int i = max(0, g - kRingN); i < g; ++i)
          mbar_wait(&full[i % kRingN], (i / kRingN) & 1, abort, a.err, false);
    } else if constexpr (FP8) {
      // ----------------------------------------------- E4M3 steps to operands
      // 4 lanes a row, 16 codes a lane; 8 rows of K or of V a warp at a time
      const int B = min(kTokTile, a.pool.page_size);     // rows of a code block
      const int cw = warp - kConvert0;
      int g = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Plan* p = next_plan(n);
        if (!p) break;
        const int nS = (p->n_tiles + 1) / 2;
        for (int i = 0; i < nS; ++i, ++g) {
          const int c8 = g % kCodeRing, s = g % kS;
          ok = mbar_wait_warp(&sm.code_full[c8], (g / kCodeRing) & 1, abort, a.err) &&
               mbar_wait_warp(&sm.kv_empty[s], ((g / kS) & 1) ^ 1, abort, a.err);
          if (!ok) break;
#pragma unroll 2
          for (int u = cw; u < 4 * kTokTile / 8; u += kConvertWarps<FP8>) {
            const int op = u >> 3;                       // tile 0: K, V; tile 1: K, V
            const int r = (u & 7) * 8 + (lane >> 2), q4 = lane & 3;
            const uint8_t* blk = sm.code[c8] + op * kCodeBytes + (r & ~(B - 1)) * (kHeadDim + 1);
            const int rb = r & (B - 1);
            const uint4 c = *reinterpret_cast<const uint4*>(blk + rb * kHeadDim + 16 * q4);
            const int e = (int8_t)blk[B * kHeadDim + rb];
            const uint32_t s1 = (uint32_t)(127 + 120 + min(e, 7)) << 7;
            const uint32_t sc = s1 | (s1 << 16);
            uint32_t o[8] = {codes_to_bf16(c.x, false, sc), codes_to_bf16(c.x, true, sc),
                             codes_to_bf16(c.y, false, sc), codes_to_bf16(c.y, true, sc),
                             codes_to_bf16(c.z, false, sc), codes_to_bf16(c.z, true, sc),
                             codes_to_bf16(c.w, false, sc), codes_to_bf16(c.w, true, sc)};
            if (e > 7) {
              const uint32_t s2 = (uint32_t)(127 + e - 7) << 7;
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = mul_bf16x2(o[k], s2 | (s2 << 16));
            }
            uint8_t* row = ((op & 1) ? sm.v[s] : sm.k[s]) + (64 * (op >> 1) + r) * 128;
            *reinterpret_cast<uint4*>(row + (swizzle_chunk(r, 2 * q4) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(row + (swizzle_chunk(r, 2 * q4 + 1) << 4)) =
                make_uint4(o[4], o[5], o[6], o[7]);
          }
          fence_proxy_async();
          __syncwarp();
          mbar_arrive_if(&sm.kv_full[s], lane == 0);
          mbar_arrive_if(&sm.code_empty[c8], lane == 0);
        }
        mbar_arrive_if(&sm.plan_empty[n & 1], lane == 0);
      }
    }
  } else if (warp >= kIssueQK) {
    // ------------------------------------------------------------ MMA issuers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs<FP8>));
    const uint32_t tmem = (uint32_t)uniform((int)sm.tmem_base);
    const uint32_t k0 = smem_u32(sm.k[0]), v0 = smem_u32(sm.v[0]);
    const auto flags = [&](const Plan* p, int n, int i) {
      if (i < kMaxFlags) return uniform(sm.flags[n & 1][i]);
      return uniform(step_flags(p->tiles, p->j0, p->n_tiles, i, p->span[0], p->span[1]));
    };
    int g0 = 0;                                  // steps of the items before
    bool ok = true;
    if (warp == kIssueQK) {
      constexpr uint32_t kIdQK = idesc_bf16(128, kStep, false);
      int buf = 0;
      uint32_t phase = 1;                        // of the buffer's last PV (none yet: passes)
      for (int n = 0; ok; ++n) {
        const Plan* p = next_plan(n);
        if (!p) break;
        const int nS = (uniform(p->n_tiles) + 1) / 2, nX = lane_steps(nS);
        const uint32_t q0 = smem_u32(sm.q[n & 1][0]);
        for (int x = 0; x < nX; ++x) {
          const int i = MT == 2 ? x >> 1 : x, l = x & 1, s = (g0 + i) % kS;
          const int f = i < nS ? flags(p, n, i) >> (2 * (MT == 2 ? l : 0)) : 0;
          if ((MT == 1 ? i < nS : l == 0) &&
              !(ok = mbar_wait_warp(&sm.kv_full[s], ((g0 + i) / kS) & 1, abort, a.err)))
            break;
          if (!(ok = mbar_wait_warp(&sm.pv_done[buf], phase, abort, a.err))) break;
          if (f & 1) {
            tc_fence_after();
            const uint64_t qa = sdesc(q0 + (MT == 2 ? l * (128 * 128) : 0)), kb = sdesc(k0 + s * (kStep * 128));
#pragma unroll
            for (int kk = 0; kk < kHeadDim / 16; ++kk)
              tc_mma_warp(tmem + kStep * buf, qa + 2 * kk, kb + 2 * kk, kIdQK, kk > 0);
          }
          tc_commit_warp(&sm.s_full[buf]);
          if (++buf == kSBufs) {
            buf = 0;
            phase ^= 1;
          }
        }
        tc_commit_warp(&sm.plan_empty[n & 1]);   // the item's Q has been read
        g0 += nS;
      }
      tc_commit_warp(&sm.done[kLanes]);
      mbar_wait(&sm.done[kLanes], 0, abort, a.err, false);
    } else {
      constexpr uint32_t kIdPV = idesc_bf16(128, kHeadDim, true);
      const int l = warp - kIssuePV;
      int buf = l, n_lane = 0;                   // the lane's steps so far
      uint32_t phase[kSBufs] = {0, 0, 0};
      for (int n = 0; ok; ++n) {
        const Plan* p = next_plan(n);
        if (!p) break;
        const int nS = (uniform(p->n_tiles) + 1) / 2, nX = lane_steps(nS);
        uint32_t some = 0;
        for (int x = l; x < nX; x += 2) {
          // everything that does not need P comes before the wait for it
          const int i = MT == 2 ? x >> 1 : x, s = (g0 + i) % kS;
          const bool there = MT == 2 || i < nS;
          const bool needed = there && (flags(p, n, i) >> (2 * (MT == 2 ? l : 0))) & 1;
          if (there && !(ok = mbar_wait_warp(&sm.kv_full[s], ((g0 + i) / kS) & 1, abort, a.err))) break;
          const uint32_t ph = buf == 0 ? phase[0] : buf == 1 ? phase[1] : phase[2];
          if (!(ok = mbar_wait_warp(&sm.p_full[l][buf], ph, abort, a.err))) break;
          if (needed) {
            tc_fence_after();
            const uint64_t vb = sdesc(v0 + s * (kStep * 128));
            const uint32_t t_p = tmem + kStep * buf, t_o = tmem + kTmemO + 64 * l;
#pragma unroll
            for (int kk = 0; kk < kStep / 16; ++kk)
              tc_mma_ts_warp(t_o, t_p + 8 * kk, vb + 128 * kk, kIdPV, kk > 0 ? 1u : some);
            some = 1;
          }
          tc_commit_warp(&sm.pv_done[buf]);
          if (there) tc_commit_warp(&sm.kv_empty[s]);
          tc_commit_warp(&sm.o_done[l][n_lane++ & 1]);
          if (buf == 0) phase[0] ^= 1;
          else if (buf == 1) phase[1] ^= 1;
          else phase[2] ^= 1;
          buf = buf + 2 >= kSBufs ? buf + 2 - kSBufs : buf + 2;
        }
        mbar_arrive_if(&sm.plan_empty[n & 1], lane == 0);
        g0 += nS;
      }
      tc_commit_warp(&sm.done[l]);
      mbar_wait(&sm.done[l], 0, abort, a.err, false);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
    const int li = warp >> 2, m_blk = MT == 2 ? li : 0;
    const int wq = warp & 3, r = wq * 32 + lane;           // row of the lane's 128
    const uint32_t tmem = sm.tmem_base + ((uint32_t)(wq * 32) << 16);
    const uint32_t t_o = tmem + kTmemO + 64 * li;
    const float sl2 = a.scale_log2;
    int buf = li;
    uint32_t phase = 0;
    int n_lane = 0;                                        // the lane's steps of the items before
    bool alive = true;
    for (int item = 0; alive; ++item) {
      const Plan* const plan = next_plan(item);
      if (!plan) break;
      const uint8_t* const flags = sm.flags[item & 1];
      const int rows = min(128, plan->work.rows - 128 * m_blk);   // <= 0: the lane has none
      const int rr = plan->work.r0 + 128 * m_blk + min(r, max(rows, 1) - 1);
      const int p = plan->pos0 + rr / G;
      const int nT = plan->n_tiles, j0 = plan->j0;
      const int nX = lane_steps((nT + 1) / 2);
      float m_run = -INFINITY, l_run = 0.f;
      bool some = false;
      const auto step = [&](int x) {             // the lane's flags of step x
        const int i = MT == 2 ? x >> 1 : x;
        if (2 * i >= nT) return 0;
        if (i < kMaxFlags) return (int)flags[i] >> (2 * m_blk);
        return step_flags(plan->tiles, j0, nT, i, plan->span[m_blk], plan->span[m_blk]);
      };
      int f_next = li < nX ? step(li) : 0;
      for (int x = li; x < nX; x += 2) {
        const uint32_t t_s = tmem + kStep * buf;
        const int i = MT == 2 ? x >> 1 : x;
        const int f = f_next;
        const bool whole = f & 2;
        if (!(alive = mbar_wait_warp(&sm.s_full[buf], phase, abort, a.err))) break;
        if (f & 1) {
          tc_fence_after();
          uint32_t pk[kStep / 2];
          float sum0, sum1;
          const auto tile_bits = [&](int j) {    // the row's view of the item's j-th tile
            return j < nT ? tok_mask(tok_tile(plan->tiles, j0 + j) * kTokTile, p, a.window, a.sinks) : 0ull;
          };
          // P and its sum against the reference m_run
          const auto exponentiate = [&](auto masked) {
            const float m_ref = m_run == -INFINITY ? 0.f : m_run;
            uint64_t bits[2] = {0, 0};
            if constexpr (masked) {
              bits[0] = tile_bits(2 * i);
              bits[1] = tile_bits(2 * i + 1);
            }
            sum0 = sum1 = 0.f;
            float v[2][32];
            PKV_TMEM_LD32(t_s, reinterpret_cast<uint32_t*>(v[0]));
#pragma unroll
            for (int c = 0; c < kStep; c += 32) {
              float (&u)[32] = v[(c >> 5) & 1];
              tmem_wait_ld();
              if (c + 32 < kStep) PKV_TMEM_LD32(t_s + c + 32, reinterpret_cast<uint32_t*>(v[((c >> 5) & 1) ^ 1]));
              if constexpr (masked) {
                const uint32_t part = (uint32_t)(bits[c >> 6] >> (c & 63));
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!((part >> k) & 1u)) u[k] = -INFINITY;
              }
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                float e0, e1;
                fma2(e0, e1, u[k], u[k + 1], sl2, -m_ref);
                e0 = fast_exp2(e0);
                e1 = fast_exp2(e1);
                pk[(c + k) >> 1] = pack_bf16(e0, e1);
                add2(sum0, sum1, e0, e1);
              }
            }
          };
          // a second pass, after the rows that need it have moved their reference
#pragma unroll 1
          for (int pass = 0;; ++pass) {
            if (whole) exponentiate(std::false_type{});
            else exponentiate(std::true_type{});
            const bool redo = m_run == -INFINITY || !(sum0 + sum1 <= kSumLimit);
            if (pass == 1 || !__any_sync(0xffffffffu, redo)) break;
            // the row's maximum becomes its reference (S is still in TMEM)
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kStep; c += 16) {
              float v[16];
              PKV_TMEM_LD16(t_s + c, reinterpret_cast<uint32_t*>(v));
              tmem_wait_ld();
              const uint32_t part = (uint32_t)(tile_bits(2 * i + c / kTokTile) >> (c & 63));
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if ((part >> k) & 1u) mx = fmaxf(mx, v[k]);
            }
            mx *= sl2;
            float alpha = 1.f;
            bool rescale = false;
            if (redo && mx > m_run) {
              if (m_run != -INFINITY) {
                alpha = fast_exp2(m_run - mx);
                l_run *= alpha;
                rescale = true;
              }
              m_run = mx;
            }
            if (__any_sync(0xffffffffu, rescale)) {
              // O moves to the new reference, once PV(x - 2) is done. Its parity names
              // its phase: PV(x - 6), the one before on that barrier, is over, since
              // S(x) is; the one after it waits for this step's P.
              const int n = n_lane + (x >> 1) - 1;
              if (x >= 2 && !(alive = mbar_wait_warp(&sm.o_done[li][n & 1], (n >> 1) & 1, abort, a.err))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < kHeadDim; c += 16) {
                uint32_t o[16];
                PKV_TMEM_LD16(t_o + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                PKV_TMEM_ST16(t_o + c, o);
              }
              tmem_wait_st();
            }
          }
          l_run += sum0 + sum1;
          PKV_TMEM_ST32(t_s, pk);
          PKV_TMEM_ST32(t_s + 32, (pk + 32));
          if (x + 2 < nX) f_next = step(x + 2);
          tmem_wait_st();
          some = true;
          tc_fence_before();
        } else if (x + 2 < nX) {
          f_next = step(x + 2);
        }
        __syncwarp();
        mbar_arrive_if(&sm.p_full[li][buf], lane == 0);
        // buffer and phase of x + 2
        buf += 2;
        if (buf >= kSBufs) {
          buf -= kSBufs;
          phase ^= 1;
        }
      }
      if (!alive) break;
      // ---- the item's end: every PV of the lane, and with it O, is done
      // (the last but one is waited for first: it tells the phases of the last apart)
      n_lane += nX / 2;
      for (int n = max(n_lane - 2, n_lane - nX / 2); n < n_lane && alive; ++n)
        alive = mbar_wait_warp(&sm.o_done[li][n & 1], (n >> 1) & 1, abort, a.err);
      if (!alive) break;
      tc_fence_after();
      const long long pr = (long long)plan->index * a.rows + 128 * m_blk + r;
      const bool split = plan->splits > 1;
      uint16_t* const out =
          a.out + ((long long)(plan->row0 + rr / G) * a.heads * G + plan->work.head * G + rr % G) * kHeadDim;
      const bool writes = r < rows;
      // the plan is used up
      __syncwarp();
      mbar_arrive_if(&sm.plan_empty[item & 1], lane == 0);
      if (MT == 1 && li == 1) {
        // lane 1 leaves its O, m and l to lane 0
        if (!(alive = mbar_wait_warp(&sm.join_empty[wq], (item & 1) ^ 1, abort, a.err))) break;
#pragma unroll
        for (int c = 0; c < kHeadDim; c += 16) {
          uint32_t o[16];
          PKV_TMEM_LD16(t_o + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) sm.o[MT == 1 ? c + k : 0][r] = some ? __uint_as_float(o[k]) : 0.f;
        }
        sm.ml[r][0] = m_run;
        sm.ml[r][1] = l_run;
        __syncwarp();
        mbar_arrive_if(&sm.join_full[wq], lane == 0);
        tc_fence_before();
        continue;
      }
      float f0 = 1.f, f1 = 0.f;
      if (MT == 1) {
        if (!(alive = mbar_wait_warp(&sm.join_full[wq], item & 1, abort, a.err))) break;
        const float m1 = sm.ml[r][0], mm = fmaxf(m_run, m1), ref = mm == -INFINITY ? 0.f : mm;
        f0 = fast_exp2(m_run - ref);
        f1 = fast_exp2(m1 - ref);
        l_run = l_run * f0 + sm.ml[r][1] * f1;
        m_run = mm;
      }
      const float inv = split ? 1.f : (l_run > 0.f ? 1.f / l_run : 0.f);
#pragma unroll
      for (int c = 0; c < kHeadDim; c += 16) {
        uint32_t o[16];
        PKV_TMEM_LD16(t_o + c, o);
        tmem_wait_ld();
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          f[k] = some ? __uint_as_float(o[k]) : 0.f;
          if (MT == 1) f[k] = f[k] * f0 + sm.o[c + k][r] * f1;
          f[k] *= inv;
        }
        if (writes) {
          if (!split) {
#pragma unroll
            for (int k = 0; k < 16; k += 8)
              *reinterpret_cast<uint4*>(out + c + k) =
                  make_uint4(pack_bf16(f[k], f[k + 1]), pack_bf16(f[k + 2], f[k + 3]),
                             pack_bf16(f[k + 4], f[k + 5]), pack_bf16(f[k + 6], f[k + 7]));
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<float4*>(a.part_o + pr * kHeadDim + c + k) =
                  make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
          }
        }
      }
      if (split && writes) *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m_run, l_run);
      tc_fence_before();                         // O has been read: the next item may write it
      if (MT == 1) {
        __syncwarp();
        mbar_arrive_if(&sm.join_empty[wq], lane == 0);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssueQK) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(sm.tmem_base), "r"(kTmemCols));
  }
}

template <int MT, bool FP8>
cudaError_t launch_tc(const TokenAttendArgs& a, int num_sms, cudaStream_t s) {
  constexpr int smem = (int)sizeof(TcSmem<MT, FP8>) + 1024;
  static_assert(smem <= 232448, "shared memory of a CTA");
  static std::atomic<unsigned long long> configured{0};   // a bit per device
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev >= 64 || !(configured.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(token_tc_kernel<MT, FP8>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // a warpgroup that asks for more registers than the launch brought would wait for ever
    cudaFuncAttributes attr;
    if (cudaError_t e2 = cudaFuncGetAttributes(&attr, token_tc_kernel<MT, FP8>)) return e2;
    if (attr.numRegs < kLaunchRegs<FP8>) return cudaErrorInvalidConfiguration;
    if (dev < 64) configured.fetch_or(bit);
  }
  const cudaError_t e = launch_pdl(token_tc_kernel<MT, FP8>, dim3(a.ctas < num_sms ? a.ctas : num_sms),
                                   dim3(kThreads<FP8>), smem, s, a);
  count_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_token_tc(const TokenAttendArgs& a, int num_sms, cudaStream_t s) {
  if (a.pool.fp8) return a.rows == 128 ? launch_tc<1, true>(a, num_sms, s) : launch_tc<2, true>(a, num_sms, s);
  return a.rows == 128 ? launch_tc<1, false>(a, num_sms, s) : launch_tc<2, false>(a, num_sms, s);
}

}  // namespace pkv
