// paged_cache.cu — the paged 4-bit cache apart from its attention: append
// (quantize complete groups into pages, keep the rest in the bf16 tails),
// read-back as bf16 rows, fork and page moves.
#include "jfa_paged.cuh"
#include "jfa_quant.cuh"

namespace jfa {

constexpr int kPcThreads = 256;
constexpr int kPcPitch = kD + 8;  // bf16 per staged row: 272 bytes, so that the 8 rows a
                                  // fragment reads fall into different banks

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
struct PagedAppendParams {
  jfa_paged c;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int32_t* cu;
  uint32_t* flag;
  int64_t k_tok, k_head, v_tok, v_head;
  int n_total, n_each;
};

// Code of x in a group of zero point z and scale s, both in fp32, inv = 1/s:
// the rule's fp64 quotient (jfa_quant.cuh) wherever the fp32 one is too near
// a border between two codes to decide.  The fp32 quotient's error is below
// 3 * 2^-24 relative, 3e-6 at 15.
__device__ __forceinline__ uint32_t code4(float x, float z, float s, float inv) {
  const float r = (x - z) * inv;
  const float t = rintf(r);
  if (fabsf(r - t) > 0.49999f) return quant_code((double)x, (double)z, (double)s, 4);
  return (uint32_t)fminf(fmaxf(t, 0.f), 15.f);
}

struct GroupParams {
  float z, s, inv;
};
__device__ __forceinline__ GroupParams group_params(float mn, float mx, uint16_t& sb, uint16_t& zb) {
  double z, s;
  quant_params((double)mn, (double)mx, 4, zb, sb, z, s);
  GroupParams g;
  g.z = (float)z;
  g.s = (float)s;
  g.inv = s > 0.0 ? 1.0f / g.s : 0.f;  // scale 0: every code 0
  return g;
}

// The rows of sequence `row` among the new ones: the first and how many.  A
// range longer than its sequence is padded in front.
__device__ __forceinline__ void new_rows(const PagedAppendParams& p, int row, int len, int& a, int& n) {
  a = p.cu ? p.cu[row] : row * p.n_each;
  n = p.cu ? p.cu[row + 1] - a : p.n_each;
  if (n > len) {
    a += n - len;
    n = len;
  }
}

// A CTA per (unit, KV head); a unit is one page of a row to be packed.  The
// first unit of a row that gets tokens (there is one even when no page is
// complete) also rewrites the row's tail, after it has read what it packs of
// the old one; the later pages of the row hold new tokens only.
//
// Memory traffic is the bound for prompts (512 B of rows in and 152 B of
// record out per token and KV head); a decode step's append (one row a
// sequence) is bound by its launch and two dependent loads.  The codes are
// formed from fp32 quotients, eight to a 32-bit word of the record, each
// thread storing 16 bytes of key and of value codes.
__global__ void __launch_bounds__(kPcThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  __shared__ int pre[kMaxBatch + 1];
  __shared__ int wsum[kMaxBatch / 32];
  __shared__ __align__(16) uint16_t xk[kKG][kPcPitch];
  __shared__ __align__(16) uint16_t xv[kKG][kPcPitch];
  __shared__ float ks[kD], kz[kD], kinv[kD];
  __shared__ float vs[kKG][4], vz[kKG][4], vinv[kKG][4];
  __shared__ float2 mm[4][kD];
  const int tid = threadIdx.x, h = blockIdx.y;
  pdl_wait();
  // The attention that follows may become resident now.  Not before the wait:
  // a next kernel that reads earlier kernels' results ahead of its own wait
  // finds those complete.
  pdl_launch_dependents();
  int units = 0;
  if (tid < p.c.batch) {
    const int len = checked_len(p.c.seq_lens[tid], p.c.max_pages, p.flag);
    const int c0 = p.cu ? p.cu[tid] : 0, c1 = p.cu ? p.cu[tid + 1] : 0;
    if (c0 < 0 || c1 < c0 || c1 > p.n_total) {
      set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
    } else {
      int a, n_new;
      new_rows(p, tid, len, a, n_new);
      if (n_new > 0) units = max(1, (split_point(len) - split_point(len - n_new)) / kKG);
    }
  }
  batch_prefix(units, pre, wsum);
  const int x = blockIdx.x;
  if (x >= pre[kMaxBatch]) return;
  const int row = batch_find(pre, x), j = x - pre[row];
  const int n1 = p.c.seq_lens[row];
  int a, n_new;
  new_rows(p, row, n1, a, n_new);
  const int n0 = n1 - n_new;
  const int nq0 = split_point(n0), nq1 = split_point(n1);
  const size_t seg = (size_t)row * p.c.num_kv_heads + h;
  uint8_t* tail[2] = {reinterpret_cast<uint8_t*>(p.c.tail_k) + seg * kPgTailBytes,
                      reinterpret_cast<uint8_t*>(p.c.tail_v) + seg * kPgTailBytes};
  const uint16_t* fresh[2] = {p.k_new + (int64_t)a * p.k_tok + h * p.k_head,
                              p.v_new + (int64_t)a * p.v_tok + h * p.v_head};
  const int64_t tok[2] = {p.k_tok, p.v_tok};

  if (nq1 > nq0) {
    const int g = nq0 / kKG + j, t0 = g * kKG;
    const int page = p.c.table[(size_t)row * p.c.max_pages + g];
    const bool page_ok = page >= 0 && page < p.c.n_pages;
    if (!page_ok && tid == 0) set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
    // the group's rows: from the old tail below n0, else new
    {
      uint4 w[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = (tid >> 4) + 16 * i, ch = tid & 15, tau = t0 + t;
#pragma unroll
        for (int m = 0; m < 2; ++m)
          w[m][i] = tau < n0 ? *reinterpret_cast<const uint4*>(tail[m] + tail_chunk(tau - nq0, ch))
                             : *reinterpret_cast<const uint4*>(fresh[m] + (int64_t)(tau - n0) * tok[m] + 8 * ch);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = (tid >> 4) + 16 * i, ch = tid & 15;
        *reinterpret_cast<uint4*>(&xk[t][8 * ch]) = w[0][i];
        *reinterpret_cast<uint4*>(&xv[t][8 * ch]) = w[1][i];
      }
    }
    __syncthreads();
    // keys: range of a channel pair over 16 tokens; values: of a (token, 32 channels)
    {
      const int cp = tid & 63, q = tid >> 6;
      float2 lo = make_float2(INFINITY, INFINITY), hi = make_float2(-INFINITY, -INFINITY);
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&xk[16 * q + t][2 * cp]);
        const float e0 = __uint_as_float(w << 16), e1 = __uint_as_float(w & 0xFFFF0000u);
        lo.x = fminf(lo.x, e0);
        hi.x = fmaxf(hi.x, e0);
        lo.y = fminf(lo.y, e1);
        hi.y = fmaxf(hi.y, e1);
      }
      mm[q][2 * cp] = make_float2(lo.x, hi.x);
      mm[q][2 * cp + 1] = make_float2(lo.y, hi.y);
    }
    bool bad = false;
    uint8_t* rec = static_cast<uint8_t*>(p.c.pages) +
                   ((size_t)(page_ok ? page : 0) * p.c.num_kv_heads + h) * kPgRec;
    {
      const int t = tid >> 2, jj = tid & 3;
      float lo = INFINITY, hi = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(&xv[t][32 * jj + 8 * i]);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float e0 = __uint_as_float(ww[e] << 16), e1 = __uint_as_float(ww[e] & 0xFFFF0000u);
          lo = fminf(lo, fminf(e0, e1));
          hi = fmaxf(hi, fmaxf(e0, e1));
        }
      }
      uint16_t sb, zb;
      const GroupParams gp = group_params(lo, hi, sb, zb);
      bad |= !finite_h(sb) || !finite_h(zb);
      vs[t][jj] = gp.s;
      vz[t][jj] = gp.z;
      vinv[t][jj] = gp.inv;
      if (page_ok) {
        *reinterpret_cast<uint16_t*>(rec + off_vs(4) + vs_scale_off(t, jj)) = sb;
        *reinterpret_cast<uint16_t*>(rec + off_vs(4) + vs_zero_off(t, jj)) = zb;
      }
    }
    __syncthreads();
    if (tid < kD) {
      float lo = mm[0][tid].x, hi = mm[0][tid].y;
#pragma unroll
      for (int q = 1; q < 4; ++q) {
        lo = fminf(lo, mm[q][tid].x);
        hi = fmaxf(hi, mm[q][tid].y);
      }
      uint16_t sb, zb;
      const GroupParams gp = group_params(lo, hi, sb, zb);
      bad |= !finite_h(sb) || !finite_h(zb);
      ks[tid] = gp.s;
      kz[tid] = gp.z;
      kinv[tid] = gp.inv;
      if (page_ok) {
        *reinterpret_cast<uint16_t*>(rec + off_ks() + ks_scale_off(tid)) = sb;
        *reinterpret_cast<uint16_t*>(rec + off_ks() + ks_zero_off(tid)) = zb;
      }
    }
    if (bad) set_flag(p.flag, JFA_DEVERR_NONFINITE_QUANT);
    __syncthreads();
    // codes: a thread forms four consecutive words (16 bytes) of each section
    // (kc_bits and vc_loc give the places)
    {
      const int mt = tid >> 6, lane = (tid >> 1) & 31, w0 = (tid & 1) * 4, gid = lane >> 2, tig = lane & 3;
      uint32_t word[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int w = w0 + i;
        uint32_t out = 0u;
#pragma unroll
        for (int hs = 0; hs < 2; ++hs) {  // slots w and w + 8: channels 64 apart
          const int c = 16 * (w >> 1) + 2 * tig + 8 * (w & 1) + 64 * hs;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t pr = *reinterpret_cast<const uint32_t*>(&xk[16 * mt + gid + 8 * r][c]);
            out |= code4(__uint_as_float(pr << 16), kz[c], ks[c], kinv[c]) << (4 * hs + 8 * r);
            out |= code4(__uint_as_float(pr & 0xFFFF0000u), kz[c + 1], ks[c + 1], kinv[c + 1])
                   << (4 * hs + 8 * r + 16);
          }
        }
        word[i] = out;
      }
      if (page_ok)
        *reinterpret_cast<uint4*>(rec + off_kc() + tid * 16) = make_uint4(word[0], word[1], word[2], word[3]);
    }
    {
      const int kk = tid >> 6, half = (tid >> 5) & 1, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
      uint32_t word[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int w8 = 4 * half + i, hi8 = w8 & 1;
        uint32_t out = 0u;
#pragma unroll
        for (int hs = 0; hs < 2; ++hs) {  // m-tiles w8 / 2 and w8 / 2 + 4
          const int mt = (w8 >> 1) + 4 * hs, jj = mt >> 1;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = 16 * kk + 2 * tig + 8 * hi8 + e;
#pragma unroll
            for (int chi = 0; chi < 2; ++chi)
              out |= code4(bf(xv[t][16 * mt + gid + 8 * chi]), vz[t][jj], vs[t][jj], vinv[t][jj])
                     << (4 * hs + 8 * chi + 16 * e);
          }
        }
        word[i] = out;
      }
      if (page_ok)
        *reinterpret_cast<uint4*>(rec + off_vc(4) + tid * 16) = make_uint4(word[0], word[1], word[2], word[3]);
    }
  }
  // the new tail: after a packed page it restarts at nq1, all of it new
  // (slots past it keep what they held)
  if (j == 0) {
    const int from = nq1 > nq0 ? nq1 : n0;
    for (int i = tid; i < (n1 - from) * 32; i += kPcThreads) {
      const int m = i & 1, ch = (i >> 1) & 15, tau = from + (i >> 5);
      *reinterpret_cast<uint4*>(tail[m] + tail_chunk(tau - nq1, ch)) =
          *reinterpret_cast<const uint4*>(fresh[m] + (int64_t)(tau - n0) * tok[m] + 8 * ch);
    }
  }
}

int launch_paged_append(const jfa_paged& c, const uint16_t* k_new, int64_t k_tok, int64_t k_head,
                        const uint16_t* v_new, int64_t v_tok, int64_t v_head, const int32_t* cu,
                        int n_total, uint8_t* ws, cudaStream_t st) {
  PagedAppendParams p;
  p.c = c;
  p.k_new = k_new;
  p.v_new = v_new;
  p.cu = cu;
  p.flag = reinterpret_cast<uint32_t*>(ws + paged_ws(c.batch, c.num_kv_heads).off_flag);
  p.k_tok = k_tok;
  p.k_head = k_head;
  p.v_tok = v_tok;
  p.v_head = v_head;
  p.n_total = n_total;
  p.n_each = n_total / c.batch;
  // a row of n tokens packs at most n / 64 pages beside its first unit
  const int rows = c.batch < n_total ? c.batch : n_total;
  return launch_pdl(paged_append_kernel, dim3(rows + n_total / kKG, c.num_kv_heads), dim3(kPcThreads), 0, st, p) ==
                 cudaSuccess
             ? JFA_OK
             : JFA_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// read-back
// ---------------------------------------------------------------------------
struct PagedGatherParams {
  jfa_paged c;
  const int32_t* cu;
  const int32_t* start;
  uint16_t* k_out;
  uint16_t* v_out;
  uint32_t* flag;
  int n_total;
};

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// A CTA per (64-token group of a row's range, KV head): the record through
// shared memory (or the tail's rows), each half warp writing whole 256-byte
// rows.  HBM-bound: 152 B in and 512 B out per token and KV head.
__global__ void __launch_bounds__(kPcThreads) paged_gather_kernel(const __grid_constant__ PagedGatherParams p) {
  __shared__ int pre[kMaxBatch + 1];
  __shared__ int wsum[kMaxBatch / 32];
  __shared__ __align__(16) uint8_t rec[kPgRec];
  const int tid = threadIdx.x, h = blockIdx.y;
  pdl_wait();
  int units = 0;
  if (tid < p.c.batch) {
    const int a = p.cu[tid], cnt = p.cu[tid + 1] - a, s = p.start ? p.start[tid] : 0;
    if (cnt != 0) {
      const int n = checked_len(p.c.seq_lens[tid], p.c.max_pages, p.flag);
      if (a < 0 || cnt < 0 || a > p.n_total - cnt || s < 0 || s > n - cnt)
        set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
      else
        units = (s + cnt - 1) / kKG - s / kKG + 1;
    }
  }
  batch_prefix(units, pre, wsum);
  const int x = blockIdx.x;
  if (x >= pre[kMaxBatch]) return;
  const int row = batch_find(pre, x);
  const int a = p.cu[row], cnt = p.cu[row + 1] - a, s = p.start ? p.start[row] : 0;
  const int n = p.c.seq_lens[row], nq = split_point(n);
  const int g = s / kKG + x - pre[row], t0 = g * kKG;
  const int lo = max(s, t0) - t0, hi = min(s + cnt, t0 + kKG) - t0;  // tokens of the group to write
  const int ch = tid & 15;
  const int64_t pitch = (int64_t)p.c.num_kv_heads * kD;
  const int64_t first = ((int64_t)a + t0 - s) * pitch + (int64_t)h * kD + 8 * ch;  // of token t0 (may lie before the rows)
  uint16_t* ko = p.k_out + first;
  uint16_t* vo = p.v_out + first;
  if (t0 >= nq) {
    const size_t seg = (size_t)row * p.c.num_kv_heads + h;
    const uint8_t* tk = reinterpret_cast<const uint8_t*>(p.c.tail_k) + seg * kPgTailBytes;
    const uint8_t* tv = reinterpret_cast<const uint8_t*>(p.c.tail_v) + seg * kPgTailBytes;
    for (int t = tid >> 4; t < hi; t += 16) {
      if (t < lo) continue;
      *reinterpret_cast<uint4*>(ko + t * pitch) = *reinterpret_cast<const uint4*>(tk + tail_chunk(t, ch));
      *reinterpret_cast<uint4*>(vo + t * pitch) = *reinterpret_cast<const uint4*>(tv + tail_chunk(t, ch));
    }
    return;
  }
  const int page = p.c.table[(size_t)row * p.c.max_pages + g];
  if (page < 0 || page >= p.c.n_pages) {
    if (tid == 0) set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.c.pages) +
                                                    ((size_t)page * p.c.num_kv_heads + h) * kPgRec);
  for (int i = tid; i < kPgRec / 16; i += kPcThreads) reinterpret_cast<uint4*>(rec)[i] = __ldg(src + i);
  __syncthreads();
  // keys: channels 8 ch .. + 7 are pair slot ch of the four lanes tig
  float s8[8], z8[8];
#pragma unroll
  for (int tig = 0; tig < 4; ++tig) {
    const int o = (ch >> 2) * 64 + tig * 16 + (ch & 3) * 4;
    const float2 sv = __half22float2(*reinterpret_cast<const __half2*>(rec + o));
    const float2 zv = __half22float2(*reinterpret_cast<const __half2*>(rec + 256 + o));
    s8[2 * tig] = sv.x;
    s8[2 * tig + 1] = sv.y;
    z8[2 * tig] = zv.x;
    z8[2 * tig + 1] = zv.y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = (tid >> 4) + 16 * i, gid = t & 7, r = (t >> 3) & 1;
    if (t < lo || t >= hi) continue;
    {
      const int sh = 4 * (ch >> 3) + 8 * r;
      uint32_t o[4];
#pragma unroll
      for (int tig = 0; tig < 4; ++tig) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + off_kc() + i * 1024 + (gid * 4 + tig) * 32 +
                                                              4 * (ch & 7)) >> sh;
        o[tig] = pack_bf2(fmaf((float)(w & 15u), s8[2 * tig], z8[2 * tig]),
                          fmaf((float)((w >> 16) & 15u), s8[2 * tig + 1], z8[2 * tig + 1]));
      }
      *reinterpret_cast<uint4*>(ko + t * pitch) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    {
      const int mt = ch >> 1, hi8 = (t >> 3) & 1, tig = (t & 7) >> 1, e = t & 1, w8 = 2 * (mt & 3) + hi8;
      const int sh = 4 * (mt >> 2) + 8 * (ch & 1) + 16 * e;
      const int so = off_vs(4) + vs_scale_off(t, ch >> 2);
      const float s = __half2float(*reinterpret_cast<const __half*>(rec + so));
      const float z = __half2float(*reinterpret_cast<const __half*>(rec + so + 512));
      const uint8_t* wp = rec + off_vc(4) + (2 * i + (w8 >> 2)) * 512 + tig * 16 + 4 * (w8 & 3);
      uint32_t o[4];
#pragma unroll
      for (int gp = 0; gp < 4; ++gp) {
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wp + (2 * gp) * 64) >> sh;
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wp + (2 * gp + 1) * 64) >> sh;
        o[gp] = pack_bf2(fmaf((float)(w0 & 15u), s, z), fmaf((float)(w1 & 15u), s, z));
      }
      *reinterpret_cast<uint4*>(vo + t * pitch) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

int launch_paged_gather(const jfa_paged& c, const int32_t* cu, const int32_t* start, int n_total,
                        uint16_t* k_out, uint16_t* v_out, uint8_t* ws, cudaStream_t st) {
  PagedGatherParams p;
  p.c = c;
  p.cu = cu;
  p.start = start;
  p.k_out = k_out;
  p.v_out = v_out;
  p.flag = reinterpret_cast<uint32_t*>(ws + paged_ws(c.batch, c.num_kv_heads).off_flag);
  p.n_total = n_total;
  // a range of n > 0 tokens touches at most n / 64 + 2 groups (n groups when n < 2)
  const long long rows = c.batch < n_total ? c.batch : n_total;
  const unsigned grid = (unsigned)(n_total / kKG + 2 * rows);
  return launch_pdl(paged_gather_kernel, dim3(grid, c.num_kv_heads), dim3(kPcThreads), 0, st, p) == cudaSuccess
             ? JFA_OK
             : JFA_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// fork: a child takes its parent's tail, table row and length
// ---------------------------------------------------------------------------
struct PagedForkParams {
  jfa_paged c;
  const int32_t* pairs;
  uint32_t* flag;
  int n;
};

__global__ void __launch_bounds__(kPcThreads) paged_fork_kernel(const __grid_constant__ PagedForkParams p) {
  const int tid = threadIdx.x, h = blockIdx.y;
  pdl_wait();
  const int src = p.pairs[2 * blockIdx.x], dst = p.pairs[2 * blockIdx.x + 1];
  bool bad = src < 0 || src >= p.c.batch || dst < 0 || dst >= p.c.batch || src == dst;
  // no row may be written twice, or written and read (n <= JFA_MAX_BATCH = threads)
  if (tid < p.n && tid != (int)blockIdx.x) {
    const int d = p.pairs[2 * tid + 1];
    bad |= d == src || d == dst || p.pairs[2 * tid] == dst;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
    return;
  }
  const int n = checked_len(p.c.seq_lens[src], p.c.max_pages, p.flag);
  const int count = n - split_point(n);
  const size_t hkv = p.c.num_kv_heads;
  const size_t so = ((size_t)src * hkv + h) * kPgTailBytes, d0 = ((size_t)dst * hkv + h) * kPgTailBytes;
  uint8_t* tk = reinterpret_cast<uint8_t*>(p.c.tail_k);
  uint8_t* tv = reinterpret_cast<uint8_t*>(p.c.tail_v);
  // the swizzle depends on the slot alone: slots copy as they are.  All loads
  // first: a thread has at most four chunks of each
  uint4 wk[4], wv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = tid + i * kPcThreads;
    if (x < count * 16) {
      wk[i] = *reinterpret_cast<const uint4*>(tk + so + 16 * x);
      wv[i] = *reinterpret_cast<const uint4*>(tv + so + 16 * x);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = tid + i * kPcThreads;
    if (x < count * 16) {
      *reinterpret_cast<uint4*>(tk + d0 + 16 * x) = wk[i];
      *reinterpret_cast<uint4*>(tv + d0 + 16 * x) = wv[i];
    }
  }
  if (h == 0) {
    for (int i = tid; i < p.c.max_pages; i += kPcThreads)
      p.c.table[(size_t)dst * p.c.max_pages + i] = p.c.table[(size_t)src * p.c.max_pages + i];
    if (tid == 0) p.c.seq_lens[dst] = n;
  }
}

int launch_paged_fork(const jfa_paged& c, const int32_t* pairs, int n, uint8_t* ws, cudaStream_t st) {
  PagedForkParams p;
  p.c = c;
  p.pairs = pairs;
  p.flag = reinterpret_cast<uint32_t*>(ws + paged_ws(c.batch, c.num_kv_heads).off_flag);
  p.n = n;
  return launch_pdl(paged_fork_kernel, dim3(n, c.num_kv_heads), dim3(kPcThreads), 0, st, p) == cudaSuccess
             ? JFA_OK
             : JFA_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// move: pages to other places of the pool, and the table's entries after them
// ---------------------------------------------------------------------------
struct PagedMoveParams {
  jfa_paged c;
  const int32_t* moves;
  const int32_t* remap;
  uint32_t* flag;
  int n;
};

constexpr int kMvThreads = 160;  // 152 threads x 4 chunks of 16 bytes are one record
static_assert(kPgRec == 152 * 4 * 16, "record in four chunks a thread");

// CTAs [0, n * H_kv): one record each, all its loads before its stores (no
// page is both source and destination).  CTAs after them: a table row each.
// HBM-bound: 2 * 9728 B per page and KV head.
__global__ void __launch_bounds__(kMvThreads) paged_move_kernel(const __grid_constant__ PagedMoveParams p) {
  const int tid = threadIdx.x, hkv = p.c.num_kv_heads;
  pdl_wait();
  const long long x = blockIdx.x, copies = (long long)p.n * hkv;
  if (x >= copies) {
    const int row = (int)(x - copies);
    const int n = checked_len(p.c.seq_lens[row], p.c.max_pages, p.flag);
    for (int i = tid; i < split_point(n) / kKG; i += kMvThreads) {
      int32_t* e = p.c.table + (size_t)row * p.c.max_pages + i;
      const int page = *e;
      const int to = page >= 0 && page < p.c.n_pages ? p.remap[page] : -1;
      if (to < 0 || to >= p.c.n_pages) set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
      else *e = to;
    }
    return;
  }
  const int m = (int)(x / hkv), h = (int)(x % hkv);
  const int src = p.moves[2 * m], dst = p.moves[2 * m + 1];
  bool bad = src < 0 || src >= p.c.n_pages || dst < 0 || dst >= p.c.n_pages || src == dst;
  // with a remap, the moves are its pages that do not stay, onto pages that do
  if (!bad && p.remap) bad = p.remap[src] != dst || p.remap[dst] != dst;
  if (bad) {
    if (tid == 0) set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
    return;
  }
  if (tid >= 152) return;
  uint8_t* pages = static_cast<uint8_t*>(p.c.pages);
  const uint4* s = reinterpret_cast<const uint4*>(pages + ((size_t)src * hkv + h) * kPgRec) + tid;
  uint4* d = reinterpret_cast<uint4*>(pages + ((size_t)dst * hkv + h) * kPgRec) + tid;
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __ldcs(s + i * 152);
#pragma unroll
  for (int i = 0; i < 4; ++i) __stcs(d + i * 152, w[i]);
}

int launch_paged_move(const jfa_paged& c, const int32_t* moves, int n, const int32_t* remap,
                      uint8_t* ws, cudaStream_t st) {
  PagedMoveParams p;
  p.c = c;
  p.moves = moves;
  p.remap = remap;
  p.flag = reinterpret_cast<uint32_t*>(ws + paged_ws(c.batch, c.num_kv_heads).off_flag);
  p.n = n;
  const long long grid = (long long)n * c.num_kv_heads + (remap ? c.batch : 0);
  if (grid == 0) return JFA_OK;
  if (grid > 0x7FFFFFFFll) return JFA_ERR_UNSUPPORTED;
  return launch_pdl(paged_move_kernel, dim3((unsigned)grid), dim3(kMvThreads), 0, st, p) == cudaSuccess
             ? JFA_OK
             : JFA_ERR_CUDA;
}

}  // namespace jfa
