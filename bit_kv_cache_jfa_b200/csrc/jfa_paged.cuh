// jfa_paged.cuh — the paged 4-bit cache shared by its kernels (append, read
// back, attention, page moves).
//
// A page holds 64 tokens: one K4V4 record (the layout of jfa_common.cuh,
// 9728 bytes) per KV head, [n_pages][H_kv][9728].  The table gives each
// sequence's pages in order; a page is written once, when its 64 tokens are
// complete, so sequences may share it.  The newest 1..64 tokens of a sequence
// stay in bf16 in its tail, [batch][H_kv][64][128]; 16-byte chunk c of slot t
// sits at chunk position c ^ (t & 7), so that a copy of consecutive slots is a
// tensor-core operand without shared-memory bank conflicts as it lands.
//
// Lengths and tables are read on the device, so that a captured graph follows
// them as they grow.
#pragma once

#include "jfa_internal.cuh"

namespace jfa {

constexpr int kPgRec = JFA_PAGE_RECORD_BYTES;
constexpr int kPgRow = kD * 2;             // bytes of a bf16 row
constexpr int kPgTailBytes = kTail * kPgRow;  // one of K, V of a (sequence, KV head)
static_assert(kPgRec == 512 + 4096 + 1024 + 4096, "K4V4 record");

// Byte offset of chunk c (16 bytes) of tail slot t inside its (sequence, KV head).
JFA_HD int tail_chunk(int t, int c) { return t * kPgRow + ((c ^ (t & 7)) << 4); }

// A pair of bf16 numbers: its values, and the pair of two values.
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Workspace: the error flag, a ticket per (sequence, KV head) (zero between
// calls) and the attention's partials: two per CTA, and one per warp.
constexpr int kPgMaxCtas = 192;
constexpr int kPgWarps = 12;
constexpr int kPgPart = kMaxG * kPartStride;  // floats of one partial: per head m, l, pad2, acc[128]
struct PagedWs {
  size_t off_flag, off_ticket, off_cta, off_warp, total;
};
inline PagedWs paged_ws(int batch, int hkv) {
  PagedWs w;
  w.off_flag = 0;
  w.off_ticket = 256;
  w.off_cta = w.off_ticket + ((size_t)batch * hkv * 4 + 255) / 256 * 256;
  w.off_warp = w.off_cta + (size_t)kPgMaxCtas * 2 * kPgPart * 4;
  w.total = w.off_warp + (size_t)kPgMaxCtas * kPgWarps * kPgPart * 4;
  return w;
}

// A sequence's length as the kernels use it: 0 (and the flag) when it is
// negative or past what the table's row can hold beside the tail.
__device__ __forceinline__ int checked_len(int n, int max_pages, uint32_t* flag) {
  if (n < 0 || n > (long long)max_pages * kKG + kTail) {
    set_flag(flag, JFA_DEVERR_BAD_INDEX);
    return 0;
  }
  return n;
}

// Exclusive prefix sums of one value per thread b < JFA_MAX_BATCH over a block
// of at least JFA_MAX_BATCH threads: pre[0..JFA_MAX_BATCH], the total last.
// Every thread of the block calls it.
__device__ __forceinline__ void batch_prefix(int val, int* pre, int* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int x = tid < kMaxBatch ? val : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31 && w < kMaxBatch / 32) warp_sums[w] = x;
  __syncthreads();
  if (tid < kMaxBatch) {
    int before = 0;
#pragma unroll
    for (int i = 0; i < kMaxBatch / 32; ++i) before += i < w ? warp_sums[i] : 0;
    pre[tid + 1] = before + x;
    if (tid == 0) pre[0] = 0;
  }
  __syncthreads();
}

// The row whose range [pre[row], pre[row + 1]) holds x (0 <= x < pre[256]).
__device__ __forceinline__ int batch_find(const int* pre, int x) {
  int lo = 0, hi = kMaxBatch;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
static_assert(kMaxBatch == 256, "batch_find halves 256 rows in 8 steps");

int launch_paged_append(const jfa_paged& c, const uint16_t* k_new, int64_t k_tok, int64_t k_head,
                        const uint16_t* v_new, int64_t v_tok, int64_t v_head, const int32_t* cu,
                        int n_total, uint8_t* ws, cudaStream_t st);
int launch_paged_gather(const jfa_paged& c, const int32_t* cu, const int32_t* start, int n_total,
                        uint16_t* k_out, uint16_t* v_out, uint8_t* ws, cudaStream_t st);
int launch_paged_fork(const jfa_paged& c, const int32_t* pairs, int n, uint8_t* ws, cudaStream_t st);
int launch_paged_move(const jfa_paged& c, const int32_t* moves, int n, const int32_t* remap,
                      uint8_t* ws, cudaStream_t st);
int launch_paged_attend(const jfa_paged& c, const uint16_t* q, int64_t q_row, float scale, int window,
                        int sinks, uint8_t* ws, uint16_t* out, float* lse, cudaStream_t st);
int launch_qk_norm_rope(const jfa_rope& r, cudaStream_t st);

}  // namespace jfa
