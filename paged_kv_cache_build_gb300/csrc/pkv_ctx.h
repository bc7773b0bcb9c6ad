// The handle, its streams, and the host helpers that the library's entry points
// share (definitions in pkv_host.cu).
#pragma once

#include <cuda_runtime.h>

#include <string>
#include <vector>

#include "../../include/pkv.h"
#include "pkv_internal.cuh"
#include "pkv_token_plan.h"

namespace pkv {

constexpr int kModeTokens = 2;   // a token stream (pkv_stream_open_tokens)

struct Stream {
  bool open = false;
  pkv_stream_cfg cfg{};
  // device lists (one allocation)
  int32_t* d_mem = nullptr;
  int32_t* d_scale = nullptr;
  int32_t* d_window = nullptr;
  int32_t* d_special = nullptr;
  int32_t* d_chunks = nullptr;   // [sliding_window_num][ppc]
  int32_t* d_tbl_idx = nullptr;
  int32_t* d_tbl_len = nullptr;
  int tbl_cap = 0;
  // frame-mode counters
  int f_sp = 0;
  int n_scale = 0, win_head = 0, win_count = 0, n_special = 0, sp_len = 0, kept = 0;
  bool pending = false;
  bool u_to_scale = false, u_new_sp = false;
  int u_sp_before = 0, u_sp_off = 0, u_patch_pos = 0;
  // chunked-mode counters (by ring slot)
  int ppc = 0;
  int c_head = 0, n_chunks = 0;
  bool c_open = false;
  int c_len[kMaxChunks] = {0}, c_pages[kMaxChunks] = {0}, c_frames[kMaxChunks] = {0};
  int u_n_new = 0, u_old_pages = 0, u_pos0 = 0, u_slot = 0;
  bool u_new_chunk = false;
  // token streams: the page list and its counters
  int32_t* d_pages = nullptr;
  TokenCounts tok;
};

}  // namespace pkv

struct pkv_ctx {
  int P = 0, Ps = 0, H = 0, D = 0, L = 0, max_streams = 0;
  long long page_elems = 0;      // bf16 elements per page (bf16 pools)
  int fp8 = 0;                   // 1: E4M3 pages with row exponents
  long long page_bytes = 0;      // bytes per page (either format)
  uint16_t* d_pool = nullptr;
  int32_t* d_free = nullptr;
  int* d_err = nullptr;
  int free_top = 0;
  std::vector<pkv::Stream> streams;
  float* d_scratch = nullptr;
  size_t scratch_bytes = 0;
  int scratch_allocs = 0;        // times the split-KV scratch was (re)allocated
  int device = 0;                // the device current at pkv_create_ex
  float* noalloc_scratch = nullptr;   // device address of the static scratch on `device`
  void* d_select = nullptr;      // page skipping: query means, page estimates, kept list
  float* d_km = nullptr;         // bf16 pages: mean key per (layer, page, head, d)
  int* d_km_len = nullptr;       // its tags per (layer, page): valid length, or -1
  int select_kept = -1;          // entries in that kept list (the last call's); -1: none yet
  int num_sms = 0;
  float* d_token_part = nullptr; // token attention: partial results of split calls
  unsigned* d_joined = nullptr;  // token attention: counters of the splits' joins, 0 between calls
  std::vector<unsigned long long> seen;   // per stream id: the last batch that named it
  unsigned long long batch_no = 0;
  std::string last_error;
};

namespace pkv {

#define PKV_CUDA(h, call)                                  \
  do {                                                     \
    cudaError_t e_ = (call);                               \
    if (e_ != cudaSuccess) return cuda_fail((h), e_, #call); \
  } while (0)

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Layer `layer`'s page set (a byte offset, so that it holds for either format).
inline uint16_t* layer_base(pkv_t h, int layer) {
  return reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(h->d_pool) +
                                     (long long)layer * h->P * h->page_bytes);
}

// What an entry point writes to the device before it returns, on a stream of its own
// that it waits for: the caller's streams need not be ordered behind the default one,
// which may be busy. Operations after a failed one do nothing; wait() returns the first
// error.
class SetupStream {
 public:
  SetupStream() : e_(cudaStreamCreateWithFlags(&s_, cudaStreamNonBlocking)) {}
  ~SetupStream() {
    if (s_) cudaStreamDestroy(s_);
  }
  SetupStream(const SetupStream&) = delete;
  void fill(void* p, int byte, size_t bytes) {
    if (e_ == cudaSuccess) e_ = cudaMemsetAsync(p, byte, bytes, s_);
  }
  void copy_in(void* p, const void* host, size_t bytes) {
    if (e_ == cudaSuccess) e_ = cudaMemcpyAsync(p, host, bytes, cudaMemcpyHostToDevice, s_);
  }
  cudaError_t wait() {
    if (e_ == cudaSuccess) e_ = cudaStreamSynchronize(s_);
    return e_;
  }

 private:
  cudaStream_t s_ = nullptr;
  cudaError_t e_;
};

// Records the message and returns the status.
pkv_status fail(pkv_t h, pkv_status st, const char* fmt, ...);
pkv_status cuda_fail(pkv_t h, cudaError_t e, const char* what);
PoolView pool_view(pkv_t h, int layer);
pkv_status get_stream(pkv_t h, int sid, Stream** out);
// Refuses a current device other than the handle's.
pkv_status check_device(pkv_t h);
pkv_status push_pages(pkv_t h, const PushSegment* segs, int n_seg, cudaStream_t s);
PushSegment seg(const int32_t* src, int start, int count, int step = 1, int ring = 0);

// Token streams (pkv_tokens.cu).
pkv_status token_rollback(pkv_t h, Stream* st, cudaStream_t s);
pkv_status token_evict(pkv_t h, Stream* st, cudaStream_t s);

}  // namespace pkv
