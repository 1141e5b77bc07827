// paged_cache.cu — the paged 4-bit cache apart from its attention: append
// (quantize complete groups into pages, keep the rest in the bf16 tails),
// read-back as bf16 rows, fork and page moves.
#include "jfa_paged.cuh"
#include "jfa_quant.cuh"

namespace jfa {

constexpr int kPcThreads = 256;

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

// Scale and zero point of a group from its fp32 minimum and maximum (bf16
// values), by the rule of jfa_quant.cuh.  The fp32 quotient is 2^-22 off at
// most; where that leaves the scale's directed rounding open (a range that is
// 15 times an fp16 number: every fifteenth), the smaller candidate is right if
// 15 times it, exact in fp32, reaches the range; fp64 decides where the range
// is not exact in fp32.
__device__ __noinline__ uint16_t scale_fp64(float mn, float mx) {
  uint16_t sb, zb;
  double z, s;
  quant_params((double)mn, (double)mx, 4, zb, sb, z, s);
  return sb;
}
struct GroupParams {
  float z, inv;  // zero point, 1 / scale (0 for scale 0: every code 0)
  uint16_t sb, zb;
};
__device__ __forceinline__ GroupParams group_params(float mn, float mx) {
  GroupParams g;
  const __half zh = __float2half_rd(mn);
  g.zb = __half_as_ushort(zh);
  g.z = __half2float(zh);
  const float d = mx - g.z, q = d * (1.f / 15.f);
  const __half lo = __float2half_ru(q * (1.f - 0x1p-21f)), hi = __float2half_ru(q * (1.f + 0x1p-21f));
  g.sb = __half_as_ushort(lo);
  if (g.sb != __half_as_ushort(hi)) {
    if (!(d + g.z == mx && mx - d == g.z)) g.sb = scale_fp64(mn, mx);
    else if (15.f * __half2float(lo) < d) g.sb = __half_as_ushort(hi);
  }
  const float s = __half2float(__ushort_as_half(g.sb));
  g.inv = s > 0.f ? 1.f / s : 0.f;
  return g;
}

// Eight codes of a word: x[a][e][b] at bit 4 a + 16 e + 8 b, of the group [a][e].
// t = 1.5 * 2^23 + round((x - z) / s): the sum of the shifted bit patterns less
// that of 1.5 * 2^23's is the word.  The fp32 quotient's error is below 3e-6 at
// 15; a word with one that near a border (or not a number) is formed again, by
// exact remainders.  bf16 numbers over an fp16 scale lie on a border exactly
// about once in 900, that is in every fourth warp's word.
struct WordIn {
  float x[2][2][2], z[2][2], inv[2][2];
};
__device__ __noinline__ uint32_t code_fp64(float x, float z, float s, uint32_t* flag) {
  if (x != x) {  // the ranges pass over it: code 0, as in jfa_pack_kv, but not unseen
    set_flag(flag, JFA_DEVERR_NONFINITE_QUANT);
    return 0u;
  }
  return quant_code((double)x, (double)z, (double)s, 4);
}
// The remainder d - (c + 1/2) s at the border next to the quotient is exact,
// and so is its sign, where d = x - z is (both ways of undoing it agree); else
// the fp64 quotient decides.
__device__ __noinline__ uint32_t word_exact(WordIn in, uint32_t* flag) {
  uint32_t word = 0u;
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // the scale is the fp16 number nearest to 1 / inv
      const float z = in.z[a][e], inv = in.inv[a][e], s = inv > 0.f ? __half2float(__float2half_rn(1.f / inv)) : 0.f;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float x = in.x[a][e][b], d = x - z, down = floorf(d * inv), rest = fmaf(-(down + 0.5f), s, d);
        uint32_t c = (uint32_t)(int)down;
        c += rest > 0.f || (rest == 0.f && (c & 1u)) ? 1u : 0u;
        if (!(d + z == x && x - d == z && s > 0.f)) c = code_fp64(x, z, s, flag);
        word |= (c & 15u) << (4 * a + 16 * e + 8 * b);
      }
    }
  return word;
}
__device__ __forceinline__ uint32_t quant_word(const WordIn& in, uint32_t* flag) {
  constexpr float kRound = 12582912.f;
  constexpr uint32_t kBits = 0x4B400000u;
  uint32_t word = 0u;
  bool near = false;
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float d = in.x[a][e][b] - in.z[a][e], t = fmaf(d, in.inv[a][e], kRound);
        near |= !(fabsf(fmaf(d, in.inv[a][e], kRound - t)) <= 0.49999f);
        word += __float_as_uint(t) << (4 * a + 16 * e + 8 * b);
      }
  return near ? word_exact(in, flag) : word - kBits * 0x11111111u;
}
__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t part(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

constexpr int kApThreads = 128;

// A CTA per (unit, KV head, keys or values); a unit is one page of a sequence
// to be packed.  The first unit of a sequence that gets tokens (there is one
// even when no page is complete) also rewrites the tail, after it has read
// what it packs of the old one; the later pages hold new tokens only.
//
// The rows go from memory to registers to the record: a thread loads the
// 16-byte chunks whose codes share words of the record (keys: chunks w and
// w + 8 of tokens t and t + 8, twice; values: chunks 2 m, 2 m + 1, + 8, + 9 of
// a token pair), so that shared memory carries only the key channels' ranges.
// Memory traffic is the bound for prompts (512 B of rows in and 152 B of
// record out per token and KV head), the issue rate and the chain lengths ->
// table -> rows what holds it at 19 us for 7600 rows of 8 KV heads (floor 6.6
// us): 1600 instructions a warp, 590 of them for codes on borders.  Keys and
// values in one block of 256 threads with the rows staged in shared memory
// take a quarter longer (cold 31 us against 25).  A decode step's append (one
// row a sequence) is bound by its launch and two dependent loads.
__global__ void __launch_bounds__(kApThreads, 6) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  __shared__ int wsum[kApThreads / 32];
  __shared__ int mine[5];  // row, unit of it, first new row, their number, length
  __shared__ uint32_t rng[2][kApThreads / 32][kD / 2];  // key minima, maxima (channel pairs) by warp
  // key zero point, 1 / scale; ten to a chunk of 8 channels against bank conflicts
  __shared__ __align__(16) float2 zi[kD / 8 * 10];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
  const bool keys = blockIdx.z == 0;
  pdl_wait();
  {
    static_assert(kMaxBatch == 2 * kApThreads, "two sequences a thread");
    int units[2] = {0, 0}, a[2] = {0, 0}, n_new[2] = {0, 0}, len[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // all loads first
      const int row = 2 * tid + i;
      if (row >= p.c.batch) continue;
      len[i] = p.c.seq_lens[row];
      a[i] = p.cu ? p.cu[row] : row * p.n_each;
      n_new[i] = (p.cu ? p.cu[row + 1] : a[i] + p.n_each);  // (the range's end)
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (a[i] < 0 || n_new[i] < a[i] || n_new[i] > p.n_total) {
        set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
        continue;
      }
      len[i] = checked_len(len[i], p.c.max_pages, p.flag);
      n_new[i] -= a[i];
      if (n_new[i] > len[i]) {  // a range longer than its sequence is padded in front
        a[i] += n_new[i] - len[i];
        n_new[i] = len[i];
      }
      if (n_new[i] > 0) units[i] = max(1, (split_point(len[i]) - split_point(len[i] - n_new[i])) / kKG);
    }
    // which sequence has this CTA's unit: prefix sums over the sequences
    int s = units[0] + units[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) wsum[warp] = s;
    if (tid == 0) mine[0] = -1;
    __syncthreads();
    int at = s - units[0] - units[1];
    for (int w = 0; w < warp; ++w) at += wsum[w];
    const int x = blockIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (x >= at && x < at + units[i]) {
        mine[0] = 2 * tid + i;
        mine[1] = x - at;
        mine[2] = a[i];
        mine[3] = n_new[i];
        mine[4] = len[i];
      }
      at += units[i];
    }
    __syncthreads();
  }
  const int row = mine[0], j = mine[1], n_new = mine[3], n1 = mine[4];
  if (row < 0) return;
  const int n0 = n1 - n_new, nq0 = split_point(n0), nq1 = split_point(n1);
  const size_t seg = (size_t)row * p.c.num_kv_heads + h;
  uint8_t* tail = reinterpret_cast<uint8_t*>(keys ? p.c.tail_k : p.c.tail_v) + seg * kPgTailBytes;
  const int64_t tok = keys ? p.k_tok : p.v_tok;
  const uint16_t* fresh = (keys ? p.k_new + h * p.k_head : p.v_new + h * p.v_head) + (int64_t)mine[2] * tok;

  if (nq1 > nq0) {
    const int g = nq0 / kKG + j, t0 = g * kKG;
    const int page = p.c.table[(size_t)row * p.c.max_pages + g];
    const bool page_ok = page >= 0 && page < p.c.n_pages;
    if (!page_ok && tid == 0) set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
    uint8_t* rec = static_cast<uint8_t*>(p.c.pages) +
                   ((size_t)(page_ok ? page : 0) * p.c.num_kv_heads + h) * kPgRec;
    // chunk ch of the group's token t: from the old tail below n0, else new
    auto load = [&](int t, int ch) {
      const int tau = t0 + t;
      const void* at = tau < n0 ? static_cast<const void*>(tail + tail_chunk(tau - nq0, ch))
                                : static_cast<const void*>(fresh + (int64_t)(tau - n0) * tok + 8 * ch);
      return *static_cast<const uint4*>(at);
    };
    bool bad = false;
    if (keys) {
      // lane (g4, w), pass k: tokens t = 16 mt + gid and t + 8 with 8 mt + gid = 16 k + 4 warp + g4
      const int w = lane & 7, q0 = 4 * warp + (lane >> 3);
      uint4 x[2][2][2];  // [pass][r][chunk w, w + 8]
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int q = q0 + 16 * k, t = (q >> 3) * 16 + (q & 7);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < 2; ++c) x[k][r][c] = load(t + 8 * r, w + 8 * c);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t lo = part(x[0][0][c], i), hi = lo;
#pragma unroll
          for (int k = 1; k < 4; ++k) {
            lo = bmin2(lo, part(x[k >> 1][k & 1][c], i));
            hi = bmax2(hi, part(x[k >> 1][k & 1][c], i));
          }
#pragma unroll
          for (int o = 8; o < 32; o <<= 1) {
            lo = bmin2(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
            hi = bmax2(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
          }
          if (lane < 8) {
            rng[0][warp][4 * (w + 8 * c) + i] = lo;
            rng[1][warp][4 * (w + 8 * c) + i] = hi;
          }
        }
      __syncthreads();
      {
        uint32_t lo = rng[0][0][tid >> 1], hi = rng[1][0][tid >> 1];
#pragma unroll
        for (int i = 1; i < kApThreads / 32; ++i) {
          lo = bmin2(lo, rng[0][i][tid >> 1]);
          hi = bmax2(hi, rng[1][i][tid >> 1]);
        }
        const GroupParams gp = group_params(tid & 1 ? bf_hi(lo) : bf_lo(lo), tid & 1 ? bf_hi(hi) : bf_lo(hi));
        bad |= !finite_h(gp.sb) || !finite_h(gp.zb);
        zi[(tid >> 3) * 10 + (tid & 7)] = make_float2(gp.z, gp.inv);
        if (page_ok) {
          *reinterpret_cast<uint16_t*>(rec + off_ks() + ks_scale_off(tid)) = gp.sb;
          *reinterpret_cast<uint16_t*>(rec + off_ks() + ks_zero_off(tid)) = gp.zb;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // channels 2 i, 2 i + 1 of the chunks: word w of lane 4 gid + i
        float4 par[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) par[c] = *reinterpret_cast<const float4*>(&zi[(w + 8 * c) * 10 + 2 * i]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          WordIn in;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            in.z[c][0] = par[c].x, in.inv[c][0] = par[c].y, in.z[c][1] = par[c].z, in.inv[c][1] = par[c].w;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t v = part(x[k][r][c], i);
              in.x[c][0][r] = bf_lo(v);
              in.x[c][1][r] = bf_hi(v);
            }
          }
          const uint32_t word = quant_word(in, p.flag);
          const int q = q0 + 16 * k;
          if (page_ok)
            *reinterpret_cast<uint32_t*>(rec + off_kc() + (q >> 3) * 1024 + ((q & 7) * 4 + i) * 32 + 4 * w) = word;
        }
      }
    } else {
      // lane (hi8, m, tig): tokens t, t + 1 with t = 16 warp + 8 hi8 + 2 tig
      const int tig = lane & 3, m = (lane >> 2) & 3, hi8 = lane >> 4, t = 16 * warp + 8 * hi8 + 2 * tig;
      uint4 x[2][2][2];  // [token][32-channel group (m >> 1) + 2 hs][chunk 2 m + 8 hs, next]
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int hs = 0; hs < 2; ++hs)
#pragma unroll
          for (int c = 0; c < 2; ++c) x[e][hs][c] = load(t + e, 2 * m + 8 * hs + c);
      // ranges of the thread's 16 channels; the group's other 16 are lane ^ 4's
      float mn[2][2], mx[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int hs = 0; hs < 2; ++hs) {
          uint32_t lo = x[e][hs][0].x, hi = lo;
#pragma unroll
          for (int i = 1; i < 8; ++i) {
            lo = bmin2(lo, part(x[e][hs][i >> 2], i & 3));
            hi = bmax2(hi, part(x[e][hs][i >> 2], i & 3));
          }
          lo = bmin2(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, 4));
          hi = bmax2(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, 4));
          mn[e][hs] = fminf(bf_lo(lo), bf_hi(lo));
          mx[e][hs] = fmaxf(bf_lo(hi), bf_hi(hi));
        }
      // even m: the first token's two groups, odd m: the second's
      const bool odd = m & 1;
      float z[2][2], inv[2][2];
#pragma unroll
      for (int hs = 0; hs < 2; ++hs) {
        const GroupParams gp = group_params(odd ? mn[1][hs] : mn[0][hs], odd ? mx[1][hs] : mx[0][hs]);
        bad |= !finite_h(gp.sb) || !finite_h(gp.zb);
        if (page_ok) {
          uint8_t* at = rec + off_vs(4) + vs_scale_off(t + odd, (m >> 1) + 2 * hs);
          *reinterpret_cast<uint16_t*>(at) = gp.sb;
          *reinterpret_cast<uint16_t*>(at + 512) = gp.zb;
        }
        const float oz = __shfl_xor_sync(0xFFFFFFFFu, gp.z, 4), oi = __shfl_xor_sync(0xFFFFFFFFu, gp.inv, 4);
        z[0][hs] = odd ? oz : gp.z;
        z[1][hs] = odd ? gp.z : oz;
        inv[0][hs] = odd ? oi : gp.inv;
        inv[1][hs] = odd ? gp.inv : oi;
      }
      const int w8 = 2 * m + hi8;
      uint8_t* at = rec + off_vc(4) + (2 * warp + (w8 >> 2)) * 512 + tig * 16 + 4 * (w8 & 3);
#pragma unroll
      for (int gid = 0; gid < 8; ++gid) {  // channel gid of the chunks
        WordIn in;
#pragma unroll
        for (int hs = 0; hs < 2; ++hs)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            in.z[hs][e] = z[e][hs];
            in.inv[hs][e] = inv[e][hs];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t v = part(x[e][hs][c], gid >> 1);
              in.x[hs][e][c] = gid & 1 ? bf_hi(v) : bf_lo(v);
            }
          }
        const uint32_t word = quant_word(in, p.flag);
        if (page_ok) *reinterpret_cast<uint32_t*>(at + gid * 64) = word;
      }
    }
    if (bad) set_flag(p.flag, JFA_DEVERR_NONFINITE_QUANT);
  }
  // the new tail: after a packed page it restarts at nq1, all of it new
  // (slots past it keep what they held)
  if (j == 0) {
    if (nq1 > nq0) __syncthreads();  // the old tail has been read
    const int from = nq1 > nq0 ? nq1 : n0;
    for (int i = tid; i < (n1 - from) * 16; i += kApThreads) {
      const int ch = i & 15, tau = from + (i >> 4);
      *reinterpret_cast<uint4*>(tail + tail_chunk(tau - nq1, ch)) =
          *reinterpret_cast<const uint4*>(fresh + (int64_t)(tau - n0) * tok + 8 * ch);
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
  return launch_pdl(paged_append_kernel, dim3(rows + n_total / kKG, c.num_kv_heads, 2), dim3(kApThreads), 0, st, p) ==
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

// Eight codes of a word, shifted so that a byte of it holds the codes of two
// scales: bits 0-3 with scale s, 4-7 with 16 s (given as s / 16, exact).
__device__ __forceinline__ float code_value(uint32_t byte, int hs, float s, float z) {
  const float f = __uint_as_float((byte & (15u << (4 * hs))) | 0x4B000000u) - 8388608.f;  // 2^23 + code 2^(4 hs)
  return fmaf(f, s, z);
}
// 32 consecutive bytes of a row
__device__ __forceinline__ void store32(uint16_t* o, const uint32_t* w) {
  if ((reinterpret_cast<uintptr_t>(o) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(o), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

constexpr int kGtThreads = 128;

// A CTA per (64-token group of a sequence's range, KV head, keys or values).
// The record's words go from memory to registers to whole rows, by the same
// shares as in the append: a thread's words hold the codes of whole 16-byte
// chunks (keys: chunks w and w + 8 of tokens t and t + 8, twice; values: a
// token pair's chunks 2 m, 2 m + 1, + 8, + 9), so nothing passes through shared
// memory and all loads are under way together.  HBM-bound: 152 B in and 512 B
// out per token and KV head; 9267 tokens of 8 KV heads take 10.0 us, 4.9 TB/s
// (cold 13.5 us; 18 with the record staged in shared memory).
__global__ void __launch_bounds__(kGtThreads) paged_gather_kernel(const __grid_constant__ PagedGatherParams p) {
  __shared__ int wsum[kGtThreads / 32];
  __shared__ int mine[6];  // row, group of its range, first output row, their number, first token, length
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
  const bool keys = blockIdx.z == 0;
  pdl_wait();
  {
    static_assert(kMaxBatch == 2 * kGtThreads, "two sequences a thread");
    int units[2] = {0, 0}, a[2], cnt[2], from[2], len[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 2 * tid + i;
      if (row >= p.c.batch) continue;
      a[i] = p.cu[row];
      cnt[i] = p.cu[row + 1] - a[i];
      from[i] = p.start ? p.start[row] : 0;
      if (cnt[i] == 0) continue;
      len[i] = checked_len(p.c.seq_lens[row], p.c.max_pages, p.flag);
      if (a[i] < 0 || cnt[i] < 0 || a[i] > p.n_total - cnt[i] || from[i] < 0 || from[i] > len[i] - cnt[i])
        set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
      else
        units[i] = (from[i] + cnt[i] - 1) / kKG - from[i] / kKG + 1;
    }
    // which sequence has this CTA's unit: prefix sums over the sequences
    int s = units[0] + units[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) wsum[warp] = s;
    if (tid == 0) mine[0] = -1;
    __syncthreads();
    int at = s - units[0] - units[1];
    for (int w = 0; w < warp; ++w) at += wsum[w];
    const int x = blockIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (x >= at && x < at + units[i]) {
        mine[0] = 2 * tid + i;
        mine[1] = x - at;
        mine[2] = a[i];
        mine[3] = cnt[i];
        mine[4] = from[i];
        mine[5] = len[i];
      }
      at += units[i];
    }
    __syncthreads();
  }
  const int row = mine[0], a = mine[2], cnt = mine[3], s = mine[4], nq = split_point(mine[5]);
  if (row < 0) return;
  const int g = s / kKG + mine[1], t0 = g * kKG;
  const int lo = max(s, t0) - t0, hi = min(s + cnt, t0 + kKG) - t0;  // tokens of the group to write
  const int64_t pitch = (int64_t)p.c.num_kv_heads * kD;
  // of token t0 (may lie before the rows)
  uint16_t* out = (keys ? p.k_out : p.v_out) + ((int64_t)a + t0 - s) * pitch + (int64_t)h * kD;
  if (t0 >= nq) {
    const uint8_t* tail = reinterpret_cast<const uint8_t*>(keys ? p.c.tail_k : p.c.tail_v) +
                          ((size_t)row * p.c.num_kv_heads + h) * kPgTailBytes;
    for (int i = lo * 16 + tid; i < hi * 16; i += kGtThreads)
      *reinterpret_cast<uint4*>(out + (i >> 4) * pitch + 8 * (i & 15)) =
          *reinterpret_cast<const uint4*>(tail + tail_chunk(i >> 4, i & 15));
    return;
  }
  const int page = p.c.table[(size_t)row * p.c.max_pages + g];
  if (page < 0 || page >= p.c.n_pages) {
    if (tid == 0) set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
    return;
  }
  const uint8_t* rec = static_cast<const uint8_t*>(p.c.pages) + ((size_t)page * p.c.num_kv_heads + h) * kPgRec;
  auto word = [&](int at) { return __ldg(reinterpret_cast<const uint32_t*>(rec + at)); };
  auto half2f = [](uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); };
  if (keys) {
    const int w = lane & 7, q0 = 4 * warp + (lane >> 3);
    uint32_t code[2][4], sc[2][4], zp[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) code[k][i] = word(off_kc() + ((q0 + 16 * k) >> 3) * 1024 + ((q0 & 7) * 4 + i) * 32 + 4 * w);
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // chunk w + 8 c: pair slot w + 8 c of lane i
        const int at = ((w >> 2) + 2 * c) * 64 + i * 16 + (w & 3) * 4;
        sc[c][i] = word(at);
        zp[c][i] = word(256 + at);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float2 s2[4], z2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s2[i] = half2f(sc[c][i]);
        z2[i] = half2f(zp[c][i]);
        if (c) s2[i] = make_float2(s2[i].x * 0.0625f, s2[i].y * 0.0625f);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int q = q0 + 16 * k, t = (q >> 3) * 16 + (q & 7) + 8 * r;
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = pack_bf2(code_value(code[k][i] >> (8 * r), c, s2[i].x, z2[i].x),
                            code_value(code[k][i] >> (8 * r + 16), c, s2[i].y, z2[i].y));
          if (t >= lo && t < hi)
            *reinterpret_cast<uint4*>(out + t * pitch + 8 * (w + 8 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
  } else {
    const int tig = lane & 3, m = (lane >> 2) & 3, hi8 = lane >> 4, t = 16 * warp + 8 * hi8 + 2 * tig, w8 = 2 * m + hi8;
    uint32_t code[8], sc[2], zp[2];
#pragma unroll
    for (int hs = 0; hs < 2; ++hs) {
      const int at = off_vs(4) + vs_scale_off(t, (m >> 1) + 2 * hs);  // of both tokens
      sc[hs] = word(at);
      zp[hs] = word(at + 512);
    }
#pragma unroll
    for (int gid = 0; gid < 8; ++gid)
      code[gid] = word(off_vc(4) + (2 * warp + (w8 >> 2)) * 512 + (gid * 4 + tig) * 16 + 4 * (w8 & 3));
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int hs = 0; hs < 2; ++hs) {
        const float2 s2 = half2f(sc[hs]), z2 = half2f(zp[hs]);
        const float sv = (e ? s2.y : s2.x) * (hs ? 0.0625f : 1.f), zv = e ? z2.y : z2.x;
        uint32_t o[8];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[4 * c + i] = pack_bf2(code_value(code[2 * i] >> (8 * c + 16 * e), hs, sv, zv),
                                    code_value(code[2 * i + 1] >> (8 * c + 16 * e), hs, sv, zv));
        if (t + e >= lo && t + e < hi) store32(out + (t + e) * pitch + 16 * m + 64 * hs, o);
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
  return launch_pdl(paged_gather_kernel, dim3(grid, c.num_kv_heads, 2), dim3(kGtThreads), 0, st, p) == cudaSuccess
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
  const int n = p.c.seq_lens[src];
  if (checked_len(n, p.c.max_pages, p.flag) != n) return;  // the child stays as it is
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
// HBM-bound: 2 * 9728 B per page and KV head; 1000 pages of 8 KV heads with
// the fork before them take 27.3 us, 94 % of the copy rate.
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
