// Causal attention of a token stream's last tokens over its pages on the
// 5th-generation tensor cores (tcgen05 + TMEM): chunks of a prompt, where a KV head
// has many query rows (tokens x query heads of the group).
//
//   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),   s_j = log2(e) sm_scale q . k_j
//
// Bounds: at head_dim 64 a 128 x 64 tile of scores takes 2 x 128 matrix-unit cycles (4096
// multiply-adds a cycle) and 256 cycles of the SM's 32 exponentials a cycle, so neither may
// pause for the other. What makes them pause is latency: S must come back from the matrix
// unit and P go to it. So an SM runs four independent pipelines ("lanes"), each 128 query
// rows with its own S and O in TMEM, its own issuing warp and its own four softmax warps (a
// thread per row); while one waits for its products the others exponentiate. A CTA's lanes
// are MT blocks of 128 rows times kLanes / MT interleaved parts of the key tiles, joined at
// the end. Measured: 1374 queries of 32 heads over 43968 keys of 8 in 481 us on bf16 pages,
// 1.01 PFLOP/s (0.53 of the measured cuBLAS rate), and in 627 us on E4M3 pages, where the
// warps that convert tiles set the pace.
//
// Warps: softmax (lane = warp / 4), the lanes' MMA issuers, the producer, which fills a ring
// of 64-slot K and V tiles by bulk copies (pages are stored as ready operands); on E4M3 pages
// it fills a ring of codes, and three or seven warps convert them into the operand ring
// (code * 2^e is exact in bf16).
//
// A lane's cycle: QK into S, softmax (P = 2^(S - m) as bf16 over the first half of S), PV
// into O, and QK of the next tile behind it. Its issuing warp stays converged (see
// tc_mma_warp) and has waited for the next tile's K and V before it waits for P. m is a
// reference that need not be the running maximum, for it cancels: it moves to the row's
// maximum on the first tile and when a row's sum of a tile exceeds 2^10, so that most
// tiles take one pass over S. P is rounded to bf16 (2^-9 relative) for the matrix unit;
// sums are taken before that rounding, in fp32.
// Every wait is bounded; one that gives up sets the device error word.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "pkv_ptx.cuh"
#include "pkv_tokens.cuh"

namespace pkv {

namespace {

constexpr int kBN = kTokTile;
// bf16 pages, 256 rows: two CTAs of two lanes an SM, so that one's start and end run beside
// the other's products (prefill of 8192 tokens, 16 heads: 145 us, 152 with one CTA of 512
// rows; ragged batch of 12 chunks 245 against 270 us). Else one CTA of four lanes: E4M3 pages,
// which it converts once for all of them, and 128 rows, which take little time beside the
// pages' (16 x 4031 keys: 32 us, 37 with two CTAs).
template <int MT, bool FP8>
constexpr int kLanes = FP8 || MT == 1 ? 4 : 2;
template <int MT, bool FP8>
constexpr int kCtasPerSm = 4 / kLanes<MT, FP8>;
template <int MT, bool FP8>
constexpr int kSoftmaxWarps = 4 * kLanes<MT, FP8>;
template <int MT, bool FP8>
constexpr int kIssuer0 = kSoftmaxWarps<MT, FP8>;
template <int MT, bool FP8>
constexpr int kProducer = kIssuer0<MT, FP8> + kLanes<MT, FP8>;
template <int MT, bool FP8>
constexpr int kConvert0 = kProducer<MT, FP8> + 1;
// The conversion sets E4M3 pages' pace: with one or two row blocks seven warps do it (16
// streams of 8030 keys, 120 rows: 97 us, 160 with three), with four there are registers for
// three only.
template <int MT, bool FP8>
constexpr int kConvertWarps = kLanes<MT, FP8> == 2 ? 1 : FP8 && MT < 4 ? 7 : 3;   // (bf16: idle, whole warpgroups)
template <int MT, bool FP8>
constexpr int kThreads = 32 * (kConvert0<MT, FP8> + kConvertWarps<MT, FP8>);
// Registers a thread at launch; the softmax warpgroups then take what the others give up.
template <int MT, bool FP8>
constexpr int kLaunchRegs = FP8 && MT < 4 ? 72 : 80;
template <int MT, bool FP8>
constexpr int kOtherRegs = FP8 && MT < 4 ? 40 : 32;
template <int MT, bool FP8>
constexpr int kSoftmaxRegs = FP8 && MT < 4 ? 96 : 104;
template <int MT, bool FP8>
constexpr bool kRegsFit =
    kSoftmaxRegs<MT, FP8> * kSoftmaxWarps<MT, FP8> +
        kOtherRegs<MT, FP8> * (kThreads<MT, FP8> / 32 - kSoftmaxWarps<MT, FP8>) <=
    kLaunchRegs<MT, FP8> * (kThreads<MT, FP8> / 32);
template <int MT, bool FP8>
constexpr int kQThreads = 32 * kProducer<MT, FP8>;   // softmax warps and issuers
// The ring's stages belong to one part of the tiles each: a multiple of kLanes / MT.
template <int MT, bool FP8>
constexpr int kRing = kLanes<MT, FP8> == 2 ? 4 : MT == 4 ? 6 : 8;
constexpr int kCodeRing = 4;
constexpr int kCodeBytes = kBN * (kHeadDim + 1);
// TMEM: S of lane i at 64 i, O at 64 (kLanes + i)
template <int MT, bool FP8>
constexpr uint32_t kTmemCols = 128 * kLanes<MT, FP8>;
constexpr float kSumLimit = 1024.0f;           // values up to 2^90 cannot take O past fp32's end

template <int MT, bool FP8>
struct __align__(1024) TcSmem {
  uint8_t q[MT][128 * 128];
  union {
    struct {
      uint8_t k[kRing<MT, FP8>][kBN * 128];
      uint8_t v[kRing<MT, FP8>][kBN * 128];
    };
    float o[kLanes<MT, FP8> - MT + (MT == kLanes<MT, FP8>)][kHeadDim][128];   // parts 1.. of the tiles, for the join
  };
  uint8_t code[FP8 ? kCodeRing : 1][FP8 ? 2 * kCodeBytes : 16];
  float ml[kLanes<MT, FP8>][128][2];
  uint64_t kv_full[kRing<MT, FP8>];
  uint64_t kv_empty[kRing<MT, FP8>];
  uint64_t code_full[kCodeRing];
  uint64_t code_empty[kCodeRing];
  uint64_t s_full[kLanes<MT, FP8>];
  uint64_t p_full[kLanes<MT, FP8>];
  uint64_t done[kLanes<MT, FP8>];
  // the CTA's work, kept here for the roles to read what they need of it
  TokenWork work;
  TokTiles tiles;
  int j0, j1;                    // its tiles
  int row0, pos0, splits;
  const int32_t* pages;
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

// A bounded wait (seconds)
__device__ __forceinline__ bool tok_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err,
                                         bool honor_abort = true) {
  return mbar_wait(bar, parity, abort, err, honor_abort, 1u << 21);
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

// A lane's rows: 128 m .. of the CTA's (none: n <= 0), and the tiles that they see.
struct LaneRows {
  int n;
  TokSpan span;
};
__device__ __forceinline__ LaneRows lane_rows(const TokenAttendArgs& a, const TokenWork& w, int pos0, int m) {
  LaneRows l;
  l.n = min(128, w.rows - 128 * m);
  const int r0 = w.r0 + 128 * m;
  l.span = tok_span(pos0 + r0 / a.group, pos0 + (r0 + l.n - 1) / a.group, a.window, a.sinks);
  if (l.n <= 0) l.span.hi = -1;
  return l;
}

template <int MT, bool FP8>
__global__ void __launch_bounds__(kThreads<MT, FP8>, kCtasPerSm<MT, FP8>)
    token_tc_kernel(const __grid_constant__ TokenAttendArgs a) {
  extern __shared__ uint8_t smem_raw[];
  TcSmem<MT, FP8>& sm = *reinterpret_cast<TcSmem<MT, FP8>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int kS = kRing<MT, FP8>;
  constexpr int kParts = kLanes<MT, FP8> / MT;
  static_assert(kS % kParts == 0, "a stage's tiles belong to one part");
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(&sm.kv_full[s], FP8 ? kConvertWarps<MT, FP8> : 1);
      mbar_init(&sm.kv_empty[s], MT);
    }
    for (int s = 0; s < kCodeRing; ++s) {
      mbar_init(&sm.code_full[s], 1);
      mbar_init(&sm.code_empty[s], kConvertWarps<MT, FP8>);
    }
    for (int i = 0; i < kLanes<MT, FP8>; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.done[i], 1);
    }
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kIssuer0<MT, FP8>) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols<MT, FP8>));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  if (threadIdx.x == 32) {
    const TokenWork w = token_work(a, blockIdx.x);
    const TokenQuery& t = a.item[w.item];
    const TokTiles tiles = tok_tiles(w.p0, w.p1, a.window, a.sinks);
    sm.work = w;
    sm.tiles = tiles;
    sm.j0 = (int)((long long)tiles.n * w.split / t.splits);
    sm.j1 = (int)((long long)tiles.n * (w.split + 1) / t.splits);
    sm.row0 = t.row0;
    sm.pos0 = t.pos0;
    sm.splits = t.splits;
    sm.pages = t.pages;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  volatile int* abort = &sm.abort;
  const TokenWork& w = sm.work;
  const int G = a.group;
  static_assert(kRegsFit<MT, FP8>, "the register split is within the launch's registers");
  pdl_wait();
  pdl_trigger();

  if (warp < kProducer<MT, FP8>) {
    // Q rows as swizzled operand tiles, all on their way at once; rows behind the last
    // one as zeros
    // (row r + kQThreads<MT, FP8> / 8 is dt tokens and dm members of the group further)
    constexpr int kStepRows = kQThreads<MT, FP8> / 8;
    const int c = threadIdx.x & 7, dt = kStepRows / G, dm = kStepRows - dt * G;
    int r = threadIdx.x >> 3, tok = (w.r0 + r) / G, mem = w.r0 + r - tok * G;
    for (; r < MT * 128; r += kStepRows) {
      const bool there = r < w.rows;
      const uint16_t* src = a.q;
      if (there) src += (sm.row0 + tok) * a.q_stride + (w.head * G + mem) * kHeadDim + c * 8;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                       smem_u32(&sm.q[r >> 7][(r & 127) * 128 + (swizzle_chunk(r & 7, c) << 4)])),
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
    asm volatile("bar.sync 1, %0;\n" ::"r"(kQThreads<MT, FP8>) : "memory");
  }

  if (warp == kProducer<MT, FP8>) {
    // ---------------------------------------------------------------- producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs<MT, FP8>));
    const int Ps = a.pool.page_size;
    const int nT = sm.j1 - sm.j0, j0 = sm.j0, p0 = w.p0, p1 = w.p1, head = w.head;
    const TokTiles tiles = sm.tiles;
    const int32_t* pages = sm.pages;
    // The page blocks of the next 32 / per tiles, one per lane: their addresses are
    // worked out together, and a tile then costs a wait and its lanes' copies.
    const int rows = min(Ps, kBN);                       // slots per block
    const int per = kBN / rows, group = 32 / per;
    constexpr uint32_t kOperand = FP8 ? kCodeBytes : kBN * 128;   // bytes of K or V in a tile
    constexpr int kRingN = FP8 ? kCodeRing : kS;
    uint64_t* const full = FP8 ? sm.code_full : sm.kv_full;
    uint64_t* const empty = FP8 ? sm.code_empty : sm.kv_empty;
    const uint32_t block_bytes = kOperand / per;
    constexpr long long kRowBytes = FP8 ? kHeadDim + 1 : 2 * kHeadDim;
    const long long plane = (long long)Ps * kRowBytes;   // of a head's K or V in a page
    const uint32_t place = (lane % per) * block_bytes;   // the lane's block in a tile
    int issued = 0;
    for (int base = 0; base < nT && issued == base; base += group) {
      const uint8_t* src = nullptr;
      if (base + lane / per < nT) {
        const int f = tok_tile(tiles, j0 + base + lane / per) * kBN + (lane % per) * rows;
        int page = pages[tok_block_entry(f, rows, p0, p1, a.window, a.sinks, Ps)];
        if (page < 0 || page >= a.pool.pool_pages) {
          atomicOr(a.err, kErrPageRange);
          page = 0;
        }
        src = reinterpret_cast<const uint8_t*>(a.pool.base) + (long long)page * a.pool.page_bytes +
              head * plane + (f % Ps) * kRowBytes;
      }
      const int end = min(nT, base + group);
      for (int j = base; j < end; ++j) {
        const int s = j % kRingN;
        if (!tok_wait(&empty[s], ((j / kRingN) & 1) ^ 1, abort, a.err)) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], 2u * kOperand);
        __syncwarp();
        if (lane / per == j - base) {
          const uint32_t bar = smem_u32(&full[s]);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            uint8_t* dst = FP8 ? sm.code[s] + kv * kCodeBytes : (kv ? sm.v[s] : sm.k[s]);
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
                "[%3];\n" ::"r"(smem_u32(dst) + place),
                "l"(src + kv * a.pool.heads * plane), "r"(block_bytes), "r"(bar)
                : "memory");
          }
        }
        issued = j + 1;
      }
    }
    // no copy may still be landing when the CTA joins or ends
    if (lane == 0)
      for (int j = max(0, issued - kRingN); j < issued; ++j)
        tok_wait(&full[j % kRingN], (j / kRingN) & 1, abort, a.err, false);
  } else if (warp >= kConvert0<MT, FP8>) {
    // ------------------------------------------------- E4M3 tiles to operands
    // 4 lanes a row, 16 codes a lane; 8 rows of K or of V a warp at a time
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs<MT, FP8>));
    const int B = min(kBN, a.pool.page_size);    // rows of a code block
    const int nT = FP8 ? sm.j1 - sm.j0 : 0;
    const int cw = warp - kConvert0<MT, FP8>;
    int u0 = cw;                                 // takes turns with the tile's larger shares
    for (int j = 0; j < nT; ++j) {
      const int c8 = j % kCodeRing, s = j % kS;
      if (!tok_wait(&sm.code_full[c8], (j / kCodeRing) & 1, abort, a.err)) break;
      if (!tok_wait(&sm.kv_empty[s], ((j / kS) & 1) ^ 1, abort, a.err)) break;
#pragma unroll (MT == 4 ? 3 : 2)
      for (int u = u0; u < 2 * kBN / 8; u += kConvertWarps<MT, FP8>) {
        const int kv = u >= kBN / 8 ? 1 : 0;
        const int r = (u - kv * (kBN / 8)) * 8 + (lane >> 2), q4 = lane & 3;
        const uint8_t* blk = sm.code[c8] + kv * kCodeBytes + (r & ~(B - 1)) * (kHeadDim + 1);
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
          for (int i = 0; i < 8; ++i) o[i] = mul_bf16x2(o[i], s2 | (s2 << 16));
        }
        uint8_t* row = (kv ? sm.v[s] : sm.k[s]) + r * 128;
        *reinterpret_cast<uint4*>(row + (swizzle_chunk(r, 2 * q4) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(row + (swizzle_chunk(r, 2 * q4 + 1) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      u0 = u0 + 1 < kConvertWarps<MT, FP8> ? u0 + 1 : 0;
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.kv_full[s]);
        mbar_arrive(&sm.code_empty[c8]);
      }
    }
  } else if (warp >= kIssuer0<MT, FP8>) {
    // ------------------------------------------------------------- MMA issuer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs<MT, FP8>));
    {
      const int li = warp - kIssuer0<MT, FP8>;
      const TokSpan span = lane_rows(a, sm.work, sm.pos0, li % MT).span;
      const int nT = sm.j1 - sm.j0, j0 = sm.j0;
      const TokTiles tiles = sm.tiles;
      const uint32_t tmem = sm.tmem_base;
      constexpr uint32_t kIdQK = idesc_bf16(128, kBN, false);
      constexpr uint32_t kIdPV = idesc_bf16(128, kHeadDim, true);
      const uint64_t qa = sdesc(smem_u32(&sm.q[li % MT][0]));
      const uint32_t t_s = tmem + 64 * li, t_o = t_s + 64 * kLanes<MT, FP8>;
      uint32_t phase = 0;
      bool ok = true, busy = false;              // busy: a tile's P is to come
      uint32_t some = 0;                         // O holds something
      int cur = 0;                               // its stage
      for (int j = li / MT;;) {
        // the next tile that the lane needs, and its K and V, before the wait for P
        bool next = false;
        int s = 0;
        for (; j < nT; j += kParts) {
          const bool needs = span.needs(tok_tile(tiles, j0 + j));
          if (busy && !needs) break;               // tiles that it skips: after this PV
          s = j % kS;
          if (!(ok = tok_wait(&sm.kv_full[s], (j / kS) & 1, abort, a.err))) break;
          if (needs) {
            next = true;
            break;
          }
          if (lane == 0) mbar_arrive(&sm.kv_empty[s]);
        }
        if (!ok) break;
        if (busy) {
          if (!tok_wait(&sm.p_full[li], phase, abort, a.err)) break;
          phase ^= 1;
          tc_fence_after();
          const uint64_t vb = sdesc(smem_u32(sm.v[cur]));
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            tc_mma_ts_warp(t_o, t_s + 8 * kk, vb + 128 * kk, kIdPV, kk > 0 ? 1u : some);
          some = 1;
          tc_commit_warp(&sm.kv_empty[cur]);
        }
        if (!next) {
          if (j >= nT) break;
          busy = false;
          continue;
        }
        // (the matrix unit keeps the order: S overwrites P after PV has read it, and the
        // next S announces this PV, too)
        tc_fence_after();
        const uint64_t kb = sdesc(smem_u32(sm.k[s]));
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk) tc_mma_warp(t_s, qa + 2 * kk, kb + 2 * kk, kIdQK, kk > 0);
        tc_commit_warp(&sm.s_full[li]);
        busy = true;
        cur = s;
        j += kParts;
      }
      tc_commit_warp(&sm.done[li]);
      tok_wait(&sm.done[li], 0, abort, a.err, false);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs<MT, FP8>));
    const int li = warp >> 2, m_blk = li % MT, part = li / MT;
    const int wq = warp & 3, r = wq * 32 + lane;           // row of the lane's 128
    const LaneRows rows = lane_rows(a, sm.work, sm.pos0, m_blk);
    const int p = sm.pos0 + (w.r0 + 128 * m_blk + min(r, max(rows.n, 1) - 1)) / G;
    const uint32_t tmem = sm.tmem_base;
    const uint32_t t_lane = (uint32_t)(wq * 32) << 16;
    const uint32_t t_s = tmem + t_lane + 64 * li, t_o = t_s + 64 * kLanes<MT, FP8>;
    const float sl2 = a.scale_log2;
    float m_run = -INFINITY, l_run = 0.f;
    uint32_t n = 0;
    bool alive = true;
    const TokTiles tiles = sm.tiles;
    const int j1 = sm.j1;
    for (int j = sm.j0 + part; j < j1; j += kParts) {
      const int tile = tok_tile(tiles, j);
      if (!rows.span.needs(tile)) continue;
      const bool whole = rows.span.whole(tile);
      if (!tok_wait(&sm.s_full[li], n & 1, abort, a.err)) {
        alive = false;
        break;
      }
      tc_fence_after();
      uint32_t pk[kBN / 2];
      float sum0, sum1, alpha = 1.f;
      bool rescale = false;
      // P and its sum against the reference m_run
      const auto exponentiate = [&](auto masked) {
        const float m_ref = m_run == -INFINITY ? 0.f : m_run;
        uint64_t bits = 0;
        if constexpr (masked) bits = tok_mask(tile * kBN, p, a.window, a.sinks);
        sum0 = sum1 = 0.f;
        float v[2][16];
        PKV_TMEM_LD16(t_s, reinterpret_cast<uint32_t*>(v[0]));
#pragma unroll
        for (int c = 0; c < kBN; c += 16) {
          float (&u)[16] = v[(c >> 4) & 1];
          tmem_wait_ld();
          if (c + 16 < kBN) PKV_TMEM_LD16(t_s + c + 16, reinterpret_cast<uint32_t*>(v[((c >> 4) & 1) ^ 1]));
          if constexpr (masked) {
            const uint32_t part = (uint32_t)(bits >> c);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!((part >> i) & 1u)) u[i] = -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float x, y;
            fma2(x, y, u[i], u[i + 1], sl2, -m_ref);
            x = fast_exp2(x);
            y = fast_exp2(y);
            pk[(c + i) >> 1] = pack_bf16(x, y);
            add2(sum0, sum1, x, y);
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
        const uint64_t bits = tok_mask(tile * kBN, p, a.window, a.sinks);
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kBN; c += 16) {
          float v[16];
          PKV_TMEM_LD16(t_s + c, reinterpret_cast<uint32_t*>(v));
          tmem_wait_ld();
          const uint32_t part = (uint32_t)(bits >> c);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if ((part >> i) & 1u) mx = fmaxf(mx, v[i]);
        }
        mx *= sl2;
        if (redo && mx > m_run) {
          if (m_run != -INFINITY) {
            alpha = fast_exp2(m_run - mx);
            l_run *= alpha;
            rescale = true;
          }
          m_run = mx;
        }
      }
      l_run += sum0 + sum1;
      PKV_TMEM_ST32(t_s, pk);
      tmem_wait_st();
      if (__any_sync(0xffffffffu, rescale)) {
        // S of this tile means that the lane's earlier products are done
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 16) {
          uint32_t o[16];
          PKV_TMEM_LD16(t_o + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          PKV_TMEM_ST16(t_o + c, o);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      mbar_arrive_if(&sm.p_full[li], lane == 0);
      ++n;
    }
    alive = alive && tok_wait(&sm.done[li], 0, abort, a.err);
    tc_fence_after();
    if (kParts > 1) {
      // ---- join the parts of the tiles: parts 1.. leave O, m and l to part 0
      asm volatile("bar.sync 2, %0;\n" ::"r"(kSoftmaxWarps<MT, FP8> * 32) : "memory");   // the ring is free
      if (part > 0) {
#pragma unroll
        for (int c = 0; c < kHeadDim; c += 16) {
          uint32_t o[16];
          PKV_TMEM_LD16(t_o + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) sm.o[li - MT][c + i][r] = n > 0 ? __uint_as_float(o[i]) : 0.f;
        }
        sm.ml[li][r][0] = m_run;
        sm.ml[li][r][1] = l_run;
      }
      asm volatile("bar.sync 2, %0;\n" ::"r"(kSoftmaxWarps<MT, FP8> * 32) : "memory");
    }
    if (alive && part == 0 && wq * 32 < rows.n) {
      float f0 = 1.f, fp[kParts];
      if (kParts > 1) {
        float mm = m_run;
#pragma unroll
        for (int i = 1; i < kParts; ++i) mm = fmaxf(mm, sm.ml[li + i * MT][r][0]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        f0 = fast_exp2(m_run - ref);
        l_run *= f0;
#pragma unroll
        for (int i = 1; i < kParts; ++i) {
          fp[i] = fast_exp2(sm.ml[li + i * MT][r][0] - ref);
          l_run += fp[i] * sm.ml[li + i * MT][r][1];
        }
        m_run = mm;
      }
      const bool split = sm.splits > 1;
      const float inv = split ? 1.f : (l_run > 0.f ? 1.f / l_run : 0.f);
      const int rr = w.r0 + 128 * m_blk + r;
      const long long pr = (long long)blockIdx.x * a.rows + 128 * m_blk + r;
      // the row's place in out, or in the partial results
      uint8_t* const row_out =
          split ? reinterpret_cast<uint8_t*>(a.part_o + pr * kHeadDim)
                : reinterpret_cast<uint8_t*>(
                      a.out + ((long long)(sm.row0 + rr / G) * a.heads * G + w.head * G + rr % G) * kHeadDim);
      // A thread has a row, but a warp writes rows of 128 bytes by 8 lanes each (a store of
      // 32 lanes to 32 rows costs 32 cycles): through the row block's Q tile, which no
      // product reads any more. bf16 rows go in one pass, fp32 partials in two.
      uint8_t* const stage = sm.q[m_blk] + wq * 32 * 128;
      const int n_rows = min(32, rows.n - wq * 32);
      for (int half = 0; half < (split ? 2 : 1); ++half) {
#pragma unroll 1
        for (int c = 0; c < (split ? 32 : kHeadDim); c += 16) {
          const int col = 32 * half + c;
          uint32_t o[16];
          PKV_TMEM_LD16(t_o + col, o);
          tmem_wait_ld();
          float f[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            f[i] = n > 0 ? __uint_as_float(o[i]) : 0.f;
            if (kParts > 1) {
              f[i] *= f0;
#pragma unroll
              for (int k = 1; k < kParts; ++k) f[i] += fp[k] * sm.o[k * MT + m_blk - MT][col + i][r];
            }
            f[i] *= inv;
          }
          if (!split) {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              *reinterpret_cast<uint4*>(stage + lane * 128 + (swizzle_chunk(lane, (c + i) >> 3) << 4)) =
                  make_uint4(pack_bf16(f[i], f[i + 1]), pack_bf16(f[i + 2], f[i + 3]),
                             pack_bf16(f[i + 4], f[i + 5]), pack_bf16(f[i + 6], f[i + 7]));
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(stage + lane * 128 + (swizzle_chunk(lane, (c + i) >> 2) << 4)) =
                  make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 4 * i + (lane >> 3);
          uint8_t* const to = reinterpret_cast<uint8_t*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row_out), row));
          const uint4 val = *reinterpret_cast<const uint4*>(stage + row * 128 + (swizzle_chunk(row, lane & 7) << 4));
          if (row < n_rows) *reinterpret_cast<uint4*>(to + 128 * half + 16 * (lane & 7)) = val;
        }
        __syncwarp();
      }
      if (split && r < rows.n) *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m_run, l_run);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer0<MT, FP8>) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(sm.tmem_base),
                 "r"(kTmemCols<MT, FP8>));
  }
}

template <int MT, bool FP8>
cudaError_t launch_tc(const TokenAttendArgs& a, cudaStream_t s) {
  constexpr int smem = (int)sizeof(TcSmem<MT, FP8>) + 1024;
  static_assert((smem + 1024) * kCtasPerSm<MT, FP8> <= 228 * 1024, "shared memory per SM");
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
    if (attr.numRegs < kLaunchRegs<MT, FP8>) return cudaErrorInvalidConfiguration;
    if (dev < 64) configured.fetch_or(bit);
  }
  const cudaError_t e = launch_pdl(token_tc_kernel<MT, FP8>, dim3(a.ctas), dim3(kThreads<MT, FP8>), smem, s, a);
  count_launches(1);
  return e;
}

}  // namespace

int token_tc_max_rows(bool fp8) { return fp8 ? 512 : 256; }

int token_tc_ctas_per_sm(bool fp8, int rows) { return !fp8 && rows == 256 ? kCtasPerSm<2, false> : 1; }

cudaError_t launch_token_tc(const TokenAttendArgs& a, cudaStream_t s) {
  if (a.pool.fp8)
    return a.rows == 128   ? launch_tc<1, true>(a, s)
           : a.rows == 256 ? launch_tc<2, true>(a, s)
                           : launch_tc<4, true>(a, s);
  return a.rows == 128 ? launch_tc<1, false>(a, s) : launch_tc<2, false>(a, s);
}

}  // namespace pkv
