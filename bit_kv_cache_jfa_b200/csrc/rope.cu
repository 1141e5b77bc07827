// rope.cu — jfa_qk_norm_rope: the RMS norm of every query and key head and its
// rotation by position, in one pass in front of the cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * w        (w = null: y = x)
//   (a, b) -> m (a cos p f_i - b sin p f_i,  a sin p f_i + b cos p f_i)
// for the pairs (a, b) of channels (i, i + r/2) or (2i, 2i + 1), i < r/2; the
// channels from r on pass through.  fp32 throughout, one rounding at the end.
//
// Angles: f_i comes as a 64-bit fraction of a turn, F = f_i / 2 pi * 2^64, so
// p F mod 2^64 is the angle's fraction of a turn without a range reduction,
// its error p times F's (2^-53 f_i from the host's 64-bit arithmetic: 1e-9 at
// a position of ten million); its upper 32 bits go to sincospif, as the nearest
// fp32 number of half turns: 2^-25 of one, 1e-7 of a channel, where bf16 outputs
// keep 2^-9.
#include "jfa_paged.cuh"

namespace jfa {

constexpr int kRpWarps = 4;
constexpr int kRpRows = 8;  // heads of a unit

enum : int { kRpHalf = 0, kRpInter = 1, kRpHalfOdd = 2 };

struct RopeParams {
  jfa_rope r;
  uint32_t units, slices;  // units = tokens * slices, slices of kRpRows heads
};

__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf_lo(u[i]);
    x[2 * i + 1] = bf_hi(u[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
}

// A warp per unit: eight heads of one token, four at a time, 8 lanes a head.
// All its rows are requested first, the sines and cosines (two pairs a lane)
// are formed meanwhile and shared through 512 bytes of shared memory.  A lane
// holds two 16-byte chunks of its head:
//   kRpHalf (r a multiple of 16): the chunks of channels i and i + r/2, so
//     the pairs are its own, and 8 pairs' cos and sin serve 16 channels;
//   kRpInter: chunks l and l + 8, pairs within them;
//   kRpHalfOdd: chunks l and l + 8; the partners come through shared memory
//     (fp32, a 9-float pitch a chunk against bank conflicts).
// HBM-bound when there are many tokens: 512 B a head; 8192 tokens of 32 and 8
// heads take 30.0 us, 5.6 TB/s, 64 tokens 2.6 us.  A token's sines are formed
// again by each of its warps (446 instructions a warp in all): a block per
// token, which forms them once and waits for them, took 95.8 us.
template <int MODE>
__global__ void __launch_bounds__(32 * kRpWarps) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs_s[kRpWarps][kD / 2];
  __shared__ float ex_s[MODE == kRpHalfOdd ? kRpWarps : 1][MODE == kRpHalfOdd ? 4 * 145 : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane >> 3, l = lane & 7;
  const uint32_t u = blockIdx.x * kRpWarps + warp;
  pdl_wait();
  if (u >= p.units) return;
  const uint32_t tok = u / p.slices;
  const int64_t t = tok;
  const int r = p.r.rotary_dim, h2 = r >> 1, nq = p.r.num_heads, rows = nq + p.r.num_kv_heads;
  const int row0 = (int)(u - tok * p.slices) * kRpRows + sub;
  const int hc = h2 >> 3;  // kRpHalf: chunks of half the rotary channels
  const int ca = MODE != kRpHalf || l < hc ? l : 2 * l;  // past them: 2 hc + 2 (l - hc)
  const int cb = MODE != kRpHalf ? l + 8 : (l < hc ? l + hc : 2 * l + 1);
  uint4 raw[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = row0 + 4 * i;
    if (row < rows) {
      const uint16_t* x = row < nq ? p.r.q + t * p.r.q_tok + row * p.r.q_head
                                   : p.r.k + t * p.r.k_tok + (row - nq) * p.r.k_head;
      raw[i][0] = *reinterpret_cast<const uint4*>(x + 8 * ca);
      raw[i][1] = *reinterpret_cast<const uint4*>(x + 8 * cb);
    } else {
      raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    }
  }
  {
    const int64_t pos = p.r.positions64 ? static_cast<const int64_t*>(p.r.positions)[t]
                                        : (int64_t) static_cast<const int32_t*>(p.r.positions)[t];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = lane + 32 * i;
      if (k < h2) {
        const uint64_t turn = (uint64_t)pos * p.r.freq[k];
        float sn, cs;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
        cs_s[warp][k] = make_float2(cs * p.r.amplitude, sn * p.r.amplitude);
      }
    }
    __syncwarp();
  }
  constexpr int NC = MODE == kRpHalfOdd ? 16 : 8;
  float cs[NC], sn[NC];  // of the lane's pairs; kRpHalfOdd: of its channels, sn with the partner's sign
  int pc[MODE == kRpHalfOdd ? 16 : 1];  // kRpHalfOdd: the partner's place, -1 where a channel passes through
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    float2 v = make_float2(1.f, 0.f);
    if (MODE == kRpHalf) {
      if (l < hc) v = cs_s[warp][8 * l + j];
    } else if (MODE == kRpInter) {
      const int k = (j < 4 ? 4 * l : 4 * l + 28) + j;
      if (k < h2) v = cs_s[warp][k];
    } else {
      const int c = 8 * l + (j < 8 ? j : j + 56), q = c < h2 ? c + h2 : c - h2;
      if (c < r) {
        v = cs_s[warp][min(c, q)];
        if (c < h2) v.y = -v.y;
      }
      pc[MODE == kRpHalfOdd ? j : 0] = c < r ? (q >> 3) * 9 + (q & 7) : -1;
    }
    cs[j] = v.x;
    sn[j] = v.y;
  }
  uint4 wr[2];
  const uint16_t* held = nullptr;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = row0 + 4 * i;
    const bool is_q = row < nq;
    const uint16_t* w = is_q ? p.r.q_weight : p.r.k_weight;
    float x[16], y[16];
    unpack8(raw[i][0], x);
    unpack8(raw[i][1], x + 8);
    if (p.r.q_weight || p.r.k_weight) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      if (w) {
        const float rs = rsqrtf(ss * (1.f / kD) + p.r.eps);
        if (w != held) {  // the weights stay over the query heads, then over the key heads
          held = w;
          wr[0] = *reinterpret_cast<const uint4*>(w + 8 * ca);
          wr[1] = *reinterpret_cast<const uint4*>(w + 8 * cb);
        }
        float wf[16];
        unpack8(wr[0], wf);
        unpack8(wr[1], wf + 8);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= rs * wf[j];
      }
    }
    // a channel that passes through is taken as it is, infinite ones too
    if (MODE == kRpHalf) {
      const bool on = l < hc;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = on ? fmaf(x[j], cs[j], -x[8 + j] * sn[j]) : x[j];
        y[8 + j] = on ? fmaf(x[8 + j], cs[j], x[j] * sn[j]) : x[8 + j];
      }
    } else if (MODE == kRpInter) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool on = (j < 4 ? 4 * l : 4 * l + 28) + j < h2;
        y[2 * j] = on ? fmaf(x[2 * j], cs[j], -x[2 * j + 1] * sn[j]) : x[2 * j];
        y[2 * j + 1] = on ? fmaf(x[2 * j + 1], cs[j], x[2 * j] * sn[j]) : x[2 * j + 1];
      }
    } else {
      float* e = ex_s[MODE == kRpHalfOdd ? warp : 0] + sub * 145;
#pragma unroll
      for (int j = 0; j < 16; ++j) e[9 * (j < 8 ? l : l + 8) + (j & 7)] = x[j];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int q = pc[MODE == kRpHalfOdd ? j : 0];
        y[j] = q >= 0 ? fmaf(x[j], cs[j & (NC - 1)], e[max(q, 0)] * sn[j & (NC - 1)]) : x[j];
      }
      __syncwarp();
    }
    if (row < rows) {
      uint16_t* o = is_q ? p.r.q_out + t * p.r.qo_tok + row * p.r.qo_head
                         : p.r.k_out + t * p.r.ko_tok + (row - nq) * p.r.ko_head;
      *reinterpret_cast<uint4*>(o + 8 * ca) = pack8(y);
      *reinterpret_cast<uint4*>(o + 8 * cb) = pack8(y + 8);
    }
  }
}

int launch_qk_norm_rope(const jfa_rope& r, cudaStream_t st) {
  RopeParams p;
  p.r = r;
  const long long slices = ((long long)r.num_heads + r.num_kv_heads + kRpRows - 1) / kRpRows;
  const long long units = slices * r.n_tokens;
  if (units > 0x7FFFFFFFll) return JFA_ERR_UNSUPPORTED;
  p.slices = (uint32_t)slices;
  p.units = (uint32_t)units;
  const dim3 grid((unsigned)((units + kRpWarps - 1) / kRpWarps)), block(32 * kRpWarps);
  cudaError_t e;
  if (r.interleaved) e = launch_pdl(qk_norm_rope_kernel<kRpInter>, grid, block, 0, st, p);
  else if (r.rotary_dim % 16 == 0) e = launch_pdl(qk_norm_rope_kernel<kRpHalf>, grid, block, 0, st, p);
  else e = launch_pdl(qk_norm_rope_kernel<kRpHalfOdd>, grid, block, 0, st, p);
  return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

}  // namespace jfa
