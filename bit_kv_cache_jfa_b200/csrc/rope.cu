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
// a position of ten million); its upper 32 bits go to sincospif.
#include "jfa_paged.cuh"

namespace jfa {

constexpr int kRpThreads = 256;
constexpr int kRpRows = kRpThreads / 16;  // heads of one pass: 16 lanes x 8 channels each

struct RopeParams {
  jfa_rope r;
  int half_shfl;  // the partner channels are a whole chunk of another lane
};

__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// One CTA per token.  Each half warp takes a head: a lane holds 8 consecutive
// channels (16-byte loads and stores), its cos and sin, computed once per
// token by the first r/2 threads, stay in registers over the heads.  The
// partner of a channel in the half layout is r/2 away: 8-channel chunks come
// by shuffles when r/2 is a multiple of 8, else element by element from the
// row itself (in the first cache level by then), before any lane stores.
// HBM-bound from a few hundred tokens on: 512 B per head and token.
template <bool INTER>
__global__ void __launch_bounds__(kRpThreads) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs_s[kD / 2];
  const int tid = threadIdx.x, l = tid & 15, hw = tid >> 4;
  const int64_t t = blockIdx.x;
  const int r = p.r.rotary_dim, h2 = r >> 1;
  pdl_wait();
  if (tid < h2) {
    const int64_t pos = p.r.positions64 ? static_cast<const int64_t*>(p.r.positions)[t]
                                : (int64_t)static_cast<const int32_t*>(p.r.positions)[t];
    const uint64_t turn = (uint64_t)pos * p.r.freq[tid];
    float sn, cs;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
    cs_s[tid] = make_float2(cs * p.r.amplitude, sn * p.r.amplitude);
  }
  const int rows = p.r.num_heads + p.r.num_kv_heads;
  const int c0 = 8 * l;
  const bool turned = c0 < r;  // some of the lane's channels rotate
  __syncthreads();
  // this lane's cos and signed sin (the partner's weight) per channel
  float cs[8], sn[8];
  int pc[8];  // partner channel
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = c0 + i;
    const bool on = c < r;
    const bool first = INTER ? (i & 1) == 0 : c < h2;
    const int k = INTER ? c >> 1 : (first ? c : c - h2);
    const float2 v = on ? cs_s[k] : make_float2(1.f, 0.f);
    cs[i] = v.x;
    sn[i] = first ? -v.y : v.y;
    pc[i] = on ? (INTER ? c ^ 1 : (first ? c + h2 : c - h2)) : c;
  }
  const int psrc = (tid & 16) + (pc[0] >> 3);  // the lane that holds the partner chunk
  const uint16_t* held = nullptr;
  float wa[8], wb[8];
  for (int row = hw; row < rows; row += kRpRows) {
    const bool is_q = row < p.r.num_heads;
    const int head = is_q ? row : row - p.r.num_heads;
    const uint16_t* x = is_q ? p.r.q + t * p.r.q_tok + head * p.r.q_head : p.r.k + t * p.r.k_tok + head * p.r.k_head;
    uint16_t* y = is_q ? p.r.q_out + t * p.r.qo_tok + head * p.r.qo_head
                       : p.r.k_out + t * p.r.ko_tok + head * p.r.ko_head;
    const uint16_t* w = is_q ? p.r.q_weight : p.r.k_weight;
    const unsigned mask = 0xFFFFu << (tid & 16);
    const uint4 raw = *reinterpret_cast<const uint4*>(x + c0);
    float a[8], b[8];
    unpack8(raw, a);
    // raw partner channels
    if (INTER) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = a[i ^ 1];
    } else if (p.half_shfl) {
      uint4 pw;
      pw.x = __shfl_sync(mask, raw.x, psrc);
      pw.y = __shfl_sync(mask, raw.y, psrc);
      pw.z = __shfl_sync(mask, raw.z, psrc);
      pw.w = __shfl_sync(mask, raw.w, psrc);
      unpack8(pw, b);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = turned ? __uint_as_float((uint32_t)x[pc[i]] << 16) : 0.f;
      __syncwarp(mask);  // every lane has read before any stores in place
    }
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], ss);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float rs = rsqrtf(ss * (1.f / kD) + p.r.eps);
      if (w != held) {  // the weights stay over the query heads, then over the key heads
        held = w;
        unpack8(*reinterpret_cast<const uint4*>(w + c0), wa);
#pragma unroll
        for (int i = 0; i < 8; ++i) wb[i] = __uint_as_float((uint32_t)w[pc[i]] << 16);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= rs * wa[i];
        b[i] *= rs * wb[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i >= r) b[i] = 0.f;  // a channel that passes through, infinite ones too
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y0 = fmaf(a[2 * i], cs[2 * i], b[2 * i] * sn[2 * i]);
      const float y1 = fmaf(a[2 * i + 1], cs[2 * i + 1], b[2 * i + 1] * sn[2 * i + 1]);
      __nv_bfloat162 v = __floats2bfloat162_rn(y0, y1);
      o[i] = *reinterpret_cast<uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(y + c0) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

int launch_qk_norm_rope(const jfa_rope& r, cudaStream_t st) {
  RopeParams p;
  p.r = r;
  p.half_shfl = r.rotary_dim % 16 == 0;
  const dim3 grid((unsigned)r.n_tokens), block(kRpThreads);
  const cudaError_t e = r.interleaved ? launch_pdl(qk_norm_rope_kernel<true>, grid, block, 0, st, p)
                                      : launch_pdl(qk_norm_rope_kernel<false>, grid, block, 0, st, p);
  return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

}  // namespace jfa
