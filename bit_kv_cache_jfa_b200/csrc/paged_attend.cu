// paged_attend.cu — jfa_paged_attend: attention of one query token per
// sequence over the paged 4-bit cache and its bf16 tails, whole or through a
// sliding window with the first tokens kept.
//
//   out[b][h] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - max),
// over the visible tokens t < n (all, or t >= n - window and t < sinks), the
// packed ones dequantised: k = s_c k' + m_c (per channel, 64 tokens),
// v = s_j v' + m_j (per token and 32 channels).
//
// What bounds it: the cache is read once, 152 B per packed token and KV head,
// for 4 * 128 * G flop, far under the tensor rate: HBM, if the SM keeps up
// with unpacking 4-bit codes (1021 instructions a record, 503 of them on the
// half-rate logic pipe, 108 MMAs).  By the growth of a call with its length
// (32768 to 65536 tokens of 16 sequences, 4 KV heads of 8 query heads; 131072
// to 262144 of one, 8 KV heads of 4) it streams 5.8 and 6.4 TB/s, 88 and 98 %
// of the copy rate; 16 to 18 us a call do not grow: launch, the chain to the
// first keys (5 us), warps that end apart (8 us), merges (4 to 7 us).  16
// sequences of 30001 to 32768 tokens take 66.6 us (floor 46.7), one of 131072
// 40.8 us (24.3).  So the codes never leave the registers of the
// warp that loads them: they are stored in the order of the mma.sync
// fragments, one AND turns a 32-bit word into a ready fp16 operand (subnormal
// code * 2^(pos - 24), exact), and the scales go to the other operand:
//   logits  A = key codes (16 tokens x 16 channels),
//           B = q_c s_c of the KV head's <= 8 query heads, hi = fp16(q_c s_c)
//           and lo = q_c s_c - hi, one product each;
//   values  A = value codes (16 channels x 16 tokens), B = fp16(p_t s_tj).
//
// q_c s_c has 19 bits (8 of bf16, 11 of fp16), so hi + lo is it exactly (but
// for what falls under fp16's smallest step, 2^-25 of 8 max |q|): a logit is
// as exact as its 32-bit sums, whatever the range of the keys.  With hi alone
// its error grows with that range (0.07 where a channel is a hundred times
// the others' size and the query four times), for 7 % of the time less (60.0
// against 64.2 us, 16 sequences of 32768 tokens, 4 KV heads of 8 query heads).
// The weights are fp16, and so is a weight times its value's scale: 2^-11 at
// most each of a token's share, whatever keys and values are (3e-4 of an output
// at unit-normal data, against the 1.6e-3 of its bf16); the mass is summed from
// the rounded weights.  Further halves would double the value MMAs.
// The query is scaled by a power of two to [1/8, 1/4) first, so that q s,
// times the 16 of the codes' position, stays in fp16's range at every scale a
// record can hold (131008 / 15).  The weights are taken against a reference
// r, p_t = 2^(u - r), that rises only when one would pass 2^15, and then to
// leave it at 2^10: sums are rarely scaled again, and the largest weight lies
// between 2^10 and 2^15.  So a weight keeps its 11 bits down to 2^-24 of the
// largest at least, and loses less than 2^-35 of it below: the mass and the
// zero points' sums hold however many tokens share the mass.  The codes' sums
// are scaled by a power of two 2^x, by which the largest value scale of a group
// comes into [2^-3, 2): where x > 0 it goes to the scales (exactly), else to
// the weights of that group (past fp16 otherwise), so that small values lose
// no more, and large ones cost the groups beside them nothing.
#include <float.h>

#include "jfa_approx.cuh"
#include "jfa_paged.cuh"

namespace jfa {

constexpr int kPaThreads = 32 * kPgWarps;
constexpr int kPaK = 512 + 4096;   // key scales, zero points and codes
constexpr int kPaV = 1024 + 4096;  // the same of the values
// Per warp two key buffers and one value buffer: while the values of a group
// are used the next keys have arrived, and while keys are used the values
// arrive.  A third key buffer made it 3 % slower: a warp does not wait for
// copies once the first have come (130 of its 4500 cycles a group, before the
// keys had a second product).
constexpr int kPaWarpBytes = 2 * kPaK + kPaV;
constexpr int kPaSmem = kPgWarps * kPaWarpBytes;
constexpr int kPaTailTok = 16;                      // tokens of a tail item
constexpr int kPaTailBytes = kPaTailTok * kPgRow;   // of K or V
// Items per CTA, at least: few CTAs leave warps alone on their scheduler, many
// leave more partials to merge over CTAs (2.5 us where there is one).  4 against
// 8: one sequence of 1000 / 4000 tokens, 8 KV heads, 9.9 / 10.6 and 11.4 / 10.8
// us; 32 of 200, 9.3 both; 17 of 171..1203 under a window of 270, 9.4 and 11.2;
// 8 of 2000, 4 KV heads, where shares of 8 meet the segments' ends, 11.9 and
// 11.0.  With 2, one of 1000 takes 10.4, the others as much.
constexpr int kPaMinItems = 4;
// Where a CTA's share is below this many items, its ends move to the ends of
// segments of at most kPgWarps items (one a warp): 96 sequences of 57..312
// tokens, 8 KV heads, 19.8 -> 16.3 us, 3 of 273..502 11.4 -> 9.2, one of 300, 2
// KV heads, 10.3 -> 8.0.  Larger shares would not feel the merge.  Segments of
// up to 18 were mixed (faster for 96 under a window, slower for one of 1000).
constexpr int kPaSnap = 64;
static_assert(kPaTailBytes <= kPaK && kPaTailBytes <= kPaV, "a tail item fits the buffers");
static_assert(kPgPart * 4 <= kPaWarpBytes, "a warp's partial fits its buffers");
static_assert(kPaSmem + 4096 <= 227 * 1024, "shared memory");
// The largest weight is 2^kPaTop at most (fp16 ends at 2^16); the room that a
// raised reference leaves under that: a maximum that grows by less than 2^5
// raises nothing, so that after a warp's first group the sums are rarely
// scaled again.
constexpr float kPaTop = 15.f;
constexpr float kPaRoom = 5.f;
// Bits by which a group's value scales may be smaller than those that the
// codes' sums are scaled for before that changes.
constexpr int kPaSlack = 3;
constexpr float kPaLn2 = 0.6931471805599453f;
// Where a reference starts: finite, so that a masked logit (-inf) minus it is
// -inf and its weight 0, and below every logit.
constexpr float kPaMin = -FLT_MAX;

struct PagedAttendParams {
  jfa_paged c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  float* part_cta;   // [grid][2][8][132]
  float* part_warp;  // [grid][kPgWarps][8][132]
  uint32_t* ticket;  // [batch][H_kv]
  uint32_t* flag;
  int64_t q_row;
  int G, window, sinks;
  float kappa;  // scale * log2(e)
};

// What a sequence of n tokens shows and how it is cut into items: the groups
// with kept first tokens, the groups from the window on, then the tail, 16
// tokens an item.
struct RowView {
  int n, nq, win_lo, sink_end;  // visible: t < sink_end or win_lo <= t < n
  int gs, gw, ng, tq0, items;   // groups [0, gs) and [gw, ng), tail items from tq0 on
};
__device__ __forceinline__ RowView row_view(int n, int window, int sinks) {
  RowView v;
  v.n = n;
  v.nq = split_point(n);
  v.win_lo = window > 0 ? max(n - window, 0) : 0;
  v.sink_end = min(sinks, v.win_lo);
  v.ng = v.nq / kKG;
  v.gw = min(v.win_lo / kKG, v.ng);
  v.gs = min((v.sink_end + kKG - 1) / kKG, v.gw);
  v.tq0 = v.sink_end > v.nq ? 0 : max(v.win_lo - v.nq, 0) / kPaTailTok;
  v.items = v.gs + (v.ng - v.gw) + (n - v.nq + kPaTailTok - 1) / kPaTailTok - v.tq0;
  return v;
}

// x / d and x % d for a quotient below 2^20 (here: KV heads), from an fp32
// quotient that is off by one at most.
__device__ __forceinline__ int div_small(int x, int d, int& rem) {
  int q = (int)__fdividef((float)x, (float)d);
  rem = x - q * d;
  if (rem < 0) {
    --q;
    rem += d;
  } else if (rem >= d) {
    ++q;
    rem -= d;
  }
  return q;
}

// A range of n cut into parts whose sizes differ by one at most, the longer first.
struct Cut {
  int q, r;
  __device__ __forceinline__ Cut(int n, int parts) : q(n / parts), r(n % parts) {}
  __device__ __forceinline__ int begin(int i) const { return i * q + min(i, r); }
  __device__ __forceinline__ int part_of(int x) const {
    const int longer = r * (q + 1);
    return x < longer ? x / (q + 1) : r + (x - longer) / q;
  }
};

// The segment at one end of a CTA's range, where other CTAs share it.
struct RangeEnd {
  int seg, sa, items, ca, cb;  // its first item and their number, its CTAs ca .. cb
  bool shared, last;           // last: this CTA's items were the last to come
};

enum : int { kItTail = 1, kItMask = 2, kItSkip = 4, kItFirst = 8, kItLast = 16 };

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void ldmatrix4(uint32_t a[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t a[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 2^x, the hardware's: 2^-22 relative; what is below 2^-126 becomes 0
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// a b - c
__device__ __forceinline__ uint32_t h2_rest(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b),
                            __hneg2(*reinterpret_cast<__half2*>(&c)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// 16-bit halves kept for the visible ones of two tokens.
__device__ __forceinline__ uint32_t half_mask(bool lo, bool hi) {
  return (lo ? 0xFFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
}

// Persistent: the items of all (sequence, KV head) segments, in a row, are cut
// into equal ranges, one per CTA and in it one per warp.  A warp carries the
// reference, mass and weighted values of its current segment; what it
// finishes alone it writes out, the rest is merged in fixed order (so results
// do not depend on timing): over the CTA's warps in shared memory, over CTAs
// by the last one to add its items to the segment's ticket.
__global__ void __launch_bounds__(kPaThreads, 1) paged_attend_kernel(const __grid_constant__ PagedAttendParams p) {
  extern __shared__ __align__(128) uint8_t pa_smem[];
  __shared__ int pre[kMaxBatch + 1];
  __shared__ int wsum[kMaxBatch / 32];
  __shared__ int lens[kMaxBatch];
  __shared__ __align__(16) int has_short[kPgWarps];  // a segment of at most kPgWarps items, by warp
  __shared__ uint64_t bars[kPgWarps][2 + 1];
  __shared__ int tail_seg[kPgWarps + 1], head_seg[kPgWarps + 1];
  __shared__ RangeEnd ends[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int hkv = p.c.num_kv_heads, G = p.G, H = p.c.num_heads;
  uint8_t* ring = pa_smem + warp * kPaWarpBytes;
  uint64_t* bar_k = bars[warp];
  uint64_t* bar_v = &bars[warp][2];
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i <= 2; ++i) mbar_init(&bars[warp][i], 1);
    fence_mbar_init();
  }
  pdl_wait();
  {
    int items = 0;
    if (tid < p.c.batch) {
      const int n = checked_len(p.c.seq_lens[tid], p.c.max_pages, p.flag);
      items = row_view(n, p.window, p.sinks).items * hkv;
      lens[tid] = n;
    }
    const bool any = __any_sync(0xFFFFFFFFu, items > 0 && items <= kPgWarps * hkv);
    if (lane == 0) has_short[warp] = any;
    batch_prefix(items, pre, wsum);
  }
  auto row_of = [&](int row) { return row_view(lens[row], p.window, p.sinks); };
  const int T = pre[kMaxBatch];
  // sequences that show nothing: zeros, spread over the CTAs
  for (int row = blockIdx.x; row < p.c.batch; row += gridDim.x) {
    if (pre[row + 1] != pre[row]) continue;
    for (int i = tid; i < H * (kD / 8); i += kPaThreads)
      *reinterpret_cast<uint4*>(p.out + (size_t)row * H * kD + 8 * i) = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = tid; i < H; i += kPaThreads) p.lse[(size_t)row * H + i] = -INFINITY;
  }
  const int C = min((int)gridDim.x, (T + kPaMinItems - 1) / kPaMinItems);
  if ((int)blockIdx.x >= C) return;
  const Cut ctas(T, C);
  int r0 = ctas.begin(blockIdx.x), r1 = ctas.begin(blockIdx.x + 1);
  static_assert(kPgWarps == 12 && kMaxBatch <= 8 * 32, "has_short in two loads");
  const int4 h0 = *reinterpret_cast<const int4*>(has_short), h1 = *reinterpret_cast<const int4*>(has_short + 4);
  if (T < kPaSnap * C && (h0.x | h0.y | h0.z | h0.w | h1.x | h1.y | h1.z | h1.w)) {
    // A cut inside a short segment moves to the segment's nearer end: nothing
    // to merge over CTAs there.  Lane 0 looks up r0, lane 1 r1.
    const int x = lane == 0 ? r0 : r1;
    int to = x;
    if (lane < 2 && x < T) {
      const int row = batch_find(pre, x), items = row_of(row).items;
      int rel;
      div_small(x - pre[row], items, rel);
      if (items <= kPgWarps) to = x - rel + (2 * rel >= items ? items : 0);
    }
    r0 = __shfl_sync(0xFFFFFFFFu, to, 0);
    r1 = __shfl_sync(0xFFFFFFFFu, to, 1);
    if (r0 == r1) return;
  }
  const int nw = min(kPgWarps, r1 - r0);  // the first nw warps have items
  const Cut warps(r1 - r0, nw);
  const int i0 = warp < nw ? r0 + warps.begin(warp) : r1, i1 = warp < nw ? r0 + warps.begin(warp + 1) : r1;

  // ---- item descriptors: lane l holds those of item base + l
  int base = i0;
  size_t d_off = 0;  // byte offset in the pages (or in the tails)
  int d_seg = 0, d_t0 = 0, d_kind = 0;
  auto describe = [&]() {
    const int x = base + lane;
    if (x < i1) {
      const int row = batch_find(pre, x);
      const RowView v = row_of(row);
      int j;
      const int head = div_small(x - pre[row], v.items, j);
      d_seg = row * hkv + head;
      d_kind = (j == 0 ? kItFirst : 0) | (j == v.items - 1 ? kItLast : 0);
      const int npk = v.gs + v.ng - v.gw;
      if (j < npk) {
        const int g = j < v.gs ? j : v.gw + j - v.gs;
        d_t0 = g * kKG;
        if (d_t0 < v.win_lo && d_t0 + kKG > v.sink_end) d_kind |= kItMask;
        int page = p.c.table[(size_t)row * p.c.max_pages + g];
        if (page < 0 || page >= p.c.n_pages) {
          set_flag(p.flag, JFA_DEVERR_BAD_INDEX);
          page = 0;
          d_kind |= kItSkip | kItMask;
        }
        d_off = ((size_t)page * hkv + head) * kPgRec;
      } else {
        const int tq = v.tq0 + j - npk;
        d_t0 = v.nq + tq * kPaTailTok;
        d_kind |= kItTail;
        if (d_t0 + kPaTailTok > v.n || (d_t0 < v.win_lo && d_t0 + kPaTailTok > v.sink_end)) d_kind |= kItMask;
        d_off = (size_t)d_seg * kPgTailBytes + tq * kPaTailBytes;
      }
    }
  };
  // the lane that holds an item's descriptor requests its copies
  // Out of L2 first, shared pages too: 64 sequences that share 20000 tokens take
  // 271.6 us with and without the hint, pages of their own 2 to 4 % less with it.
  const uint64_t pol = policy_evict_first();
  auto issue_k = [&](int x, int st) {
    if (lane == x - base) {
      const bool tl = (d_kind & kItTail) != 0;
      const uint8_t* src = (tl ? reinterpret_cast<const uint8_t*>(p.c.tail_k) : static_cast<const uint8_t*>(p.c.pages)) + d_off;
      const uint32_t bytes = tl ? kPaTailBytes : kPaK;
      mbar_expect_tx(&bar_k[st], bytes);
      bulk_g2s(ring + st * kPaK, src, bytes, &bar_k[st], pol);
    }
  };
  auto issue_v = [&](int x) {
    if (lane == x - base) {
      const bool tl = (d_kind & kItTail) != 0;
      const uint8_t* src = (tl ? reinterpret_cast<const uint8_t*>(p.c.tail_v)
                               : static_cast<const uint8_t*>(p.c.pages) + kPaK) + d_off;
      const uint32_t bytes = tl ? kPaTailBytes : kPaV;
      mbar_expect_tx(bar_v, bytes);
      bulk_g2s(ring + 2 * kPaK, src, bytes, bar_v, pol);
    }
  };

  // ---- state of the current segment; lane (gid, tig): heads 2 tig, 2 tig + 1
  float acc[8][4];   // codes' part, channels 16 mt + gid (+ 8), times 2^(pos - 24) and 2^vx
  float dz[4];       // rows 0-3: zero-point sums per channel group, row 4: mass
  float m_run[2], kap[2] = {0.f, 0.f};  // reference, kappa * 2^x of the query's scaling
  int vx = 0;              // the values' codes are summed times 2^vx
  // B fragment of the scaled query, head gid, times the codes' position factor;
  // of each four pairs the second and third change places
  uint32_t qf[16] = {};
  int seg = 0;
  bool own_start = false;  // the segment's first item was this warp's
  RowView rv = {};
  int my_head_seg = -1, my_tail_seg = -1;

  auto reset = [&](int s) {
    seg = s;
    int head;
    const int row = div_small(s, hkv, head);
    rv = row_of(row);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    dz[0] = dz[1] = dz[2] = dz[3] = 0.f;
    m_run[0] = m_run[1] = kPaMin;
    vx = 0;
    const bool ok = gid < G;
    const uint16_t* qr = p.q + (int64_t)row * p.q_row + (size_t)(head * G + (ok ? gid : 0)) * kD;
    uint32_t w[16];
    uint32_t mx = 0u;  // largest magnitude, as bits
#pragma unroll
    for (int pp = 0; pp < 16; ++pp) {
      w[pp] = ok ? *reinterpret_cast<const uint32_t*>(qr + 16 * (pp >> 1) + 2 * tig + 8 * (pp & 1)) : 0u;
      mx = max(mx, max(w[pp] << 16, w[pp]) & 0x7FFF0000u);
      mx = max(mx, max((w[pp] << 16) & 0x7FFF0000u, w[pp] & 0x7FFF0000u));
    }
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    // 2^(x - 3) <= max|q| < 2^(x - 2); a zero, subnormal or overflowing query is left as it is
    const int ex = (int)(mx >> 23);
    const int x = ex == 0 || ex >= 250 ? 0 : ex - 127 + 3;
    const float down = __uint_as_float((uint32_t)(127 - x) << 23), up = __uint_as_float((uint32_t)(127 + x) << 23);
#pragma unroll
    for (int pp = 0; pp < 16; ++pp) {
      const float f = pp < 8 ? 16.f * down : down;  // KeyPos<4>::factor
      qf[(pp & 12) | (pp & 1) << 1 | (pp >> 1 & 1)] = pack_h2(bf_lo(w[pp]) * f, bf_hi(w[pp]) * f);
    }
    kap[0] = p.kappa * __shfl_sync(0xFFFFFFFFu, up, 8 * tig);
    kap[1] = p.kappa * __shfl_sync(0xFFFFFFFFu, up, 8 * tig + 4);
  };

  auto pow2 = [](int e) { return __uint_as_float((uint32_t)(127 + e) << 23); };

  // the segment's sums out of the registers: dst[h * stride + ...] = m, l, acc
  auto store_partial = [&](float* dst) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float l = __shfl_sync(0xFFFFFFFFu, dz[e], 16 + tig);
      float zj[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) zj[j] = __shfl_sync(0xFFFFFFFFu, dz[e], j * 4 + tig);
      const int h = 2 * tig + e;
      if (h < G) {
        float* row = dst + h * kPartStride;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          const float us = pow2(((mt >> 2) ? 20 : 24) - vx);
          row[4 + 16 * mt + gid] = fmaf(acc[mt][e], us, zj[mt >> 1]);
          row[4 + 16 * mt + gid + 8] = fmaf(acc[mt][2 + e], us, zj[mt >> 1]);
        }
        if (gid == 0) {
          row[0] = m_run[e];
          row[1] = l;
        }
      }
    }
  };
  auto store_out = [&]() {
    int head;
    const int row = div_small(seg, hkv, head);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float l = __shfl_sync(0xFFFFFFFFu, dz[e], 16 + tig);
      float zj[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) zj[j] = __shfl_sync(0xFFFFFFFFu, dz[e], j * 4 + tig);
      const int h = 2 * tig + e;
      if (h < G) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // only skipped pages: zeros
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.out) + ((size_t)row * H + head * G + h) * kD;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          const float us = pow2(((mt >> 2) ? 20 : 24) - vx);
          o[16 * mt + gid] = __float2bfloat16_rn(fmaf(acc[mt][e], us, zj[mt >> 1]) * inv);
          o[16 * mt + gid + 8] = __float2bfloat16_rn(fmaf(acc[mt][2 + e], us, zj[mt >> 1]) * inv);
        }
        if (gid == 0 && p.lse) p.lse[(size_t)row * H + head * G + h] = l == 0.f ? -INFINITY : (m_run[e] + log2f(l)) * kPaLn2;
      }
    }
  };
  // everything summed so far, to the references n0, n1 (at or above m_run)
  auto rescale = [&](float n0, float n1) {
    const float a0 = approx_weight(m_run[0], n0), a1 = approx_weight(m_run[1], n1);
    m_run[0] = n0;
    m_run[1] = n1;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      acc[mt][0] *= a0;
      acc[mt][1] *= a1;
      acc[mt][2] *= a0;
      acc[mt][3] *= a1;
    }
    dz[0] *= a0;
    dz[1] *= a1;
    dz[2] *= a0;
    dz[3] *= a1;
  };
  // the lane's largest logits of heads 2 tig + e: where one is more than kPaTop
  // over its reference, the references go to kPaRoom below kPaTop over the largest
  auto raise_max = [&](float mx0, float mx1) {
    if (__any_sync(0xFFFFFFFFu, mx0 > m_run[0] + kPaTop || mx1 > m_run[1] + kPaTop)) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, o));
      }
      rescale(mx0 > m_run[0] + kPaTop ? mx0 - (kPaTop - kPaRoom) : m_run[0],
              mx1 > m_run[1] + kPaTop ? mx1 - (kPaTop - kPaRoom) : m_run[1]);
    }
  };

  // every warp's first keys are requested before any other copy, so that the
  // first products start when a third of the buffers has been filled
  if (i0 < i1) {
    describe();
    __syncwarp();
    issue_k(i0, 0);
  }
  __syncthreads();
  if (i0 < i1) {
    issue_v(i0);
    if (i0 + 1 < i1) issue_k(i0 + 1, 1);
  }
  if (warp < 2) {  // while the first copies are on their way
    const int x = warp == 0 ? r0 : r1 - 1, row = batch_find(pre, x), items = row_of(row).items;
    int rel;
    const int head = div_small(x - pre[row], items, rel), sa = x - rel;
    // finished here, or one segment fills the range
    const bool alone = (sa >= r0 && sa + items <= r1) || (warp == 1 && sa <= r0);
    const RangeEnd e = {row * hkv + head, sa, items, ctas.part_of(sa), ctas.part_of(sa + items - 1), !alone, false};
    if (lane == 0) ends[warp] = e;
  }
  int st = 0;
  uint32_t par_k = 0u, par_v = 0u;  // bit s: parity of key buffer s
  // rows of the mass and zero-point product: lanes gid < 4 the zero points, 4 ones
  const uint32_t z_mask = gid < 4 ? 0xFFFFFFFFu : 0u, z_one = gid == 4 ? kOneH2 : 0u;
  bool failed = false, ready = false;  // ready: the next keys were seen to have come
  for (int i = i0; i < i1; ++i) {
    if (i + 2 - base >= 32 && i + 2 < i1) {  // the next keys' descriptor is needed below
      base = i;
      describe();
      __syncwarp();
    }
    const int kind = __shfl_sync(0xFFFFFFFFu, d_kind, i - base);
    const int t0 = __shfl_sync(0xFFFFFFFFu, d_t0, i - base);
    {
      const int s = __shfl_sync(0xFFFFFFFFu, d_seg, i - base);
      if (i == i0 || (kind & kItFirst)) {
        reset(s);
        own_start = (kind & kItFirst) != 0;
      }
    }
    auto visible = [&](int t) {
      return !(kind & kItSkip) && t < rv.n && (t >= rv.win_lo || t < rv.sink_end);
    };
    failed = !__all_sync(0xFFFFFFFFu, ready || mbar_wait_bounded(&bar_k[st], (par_k >> st) & 1u));
    if (failed) break;
    par_k ^= 1u << st;
    const uint8_t* rk = ring + st * kPaK;
    const uint8_t* rvb = ring + 2 * kPaK;
    if (!(kind & kItTail)) {
      // ---- logits (log2 units) u[mt][2 r + e]: token 16 mt + gid + 8 r, head
      // 2 tig + e.  Half of the code words at a time (slots 4 h .. 4 h + 3 in
      // their low, 8 more in their high nibbles): the B operands of these slots,
      // hi = fp16(q s F) and lo = q s F - hi, the zero points' share, and four
      // chains of MMAs, one an m-tile.
      float u[4][4] = {};
      // [0]: slots 0-7, with the factor 16.  A lane's zero points of four pairs,
      // as they lie, are an A operand of two k-steps at once: rows gid have the
      // first and third pair, rows gid + 8 the second and fourth, so the upper
      // rows of one product (bz) and the lower of the other (by) count.
      float bz[2][4] = {}, by[2][4] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t hi[2][4], lo[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {  // slots 4 h + 8 n ..
          const int i4 = h + 2 * n;
          const uint4 sv = *reinterpret_cast<const uint4*>(rk + i4 * 64 + tig * 16);
          const uint4 zv = *reinterpret_cast<const uint4*>(rk + (4 + i4) * 64 + tig * 16);
          const uint32_t sk[4] = {sv.x, sv.y, sv.z, sv.w};
          const uint32_t* q1 = qf + 4 * i4;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int y = (x & 1) << 1 | x >> 1;
            hi[n][x] = h2_mul(q1[y], sk[x]);
            lo[n][x] = h2_rest(q1[y], sk[x], hi[n][x]);
          }
          mma16816(bz[n], zv.x, zv.y, zv.z, zv.w, q1[0], q1[1]);
          mma16816(by[n], zv.x, zv.y, zv.z, zv.w, q1[2], q1[3]);
        }
        uint32_t w[4][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          const uint4 c = *reinterpret_cast<const uint4*>(rk + 512 + mt * 1024 + lane * 32 + 16 * h);
          w[mt][0] = c.x, w[mt][1] = c.y, w[mt][2] = c.z, w[mt][3] = c.w;
        }
#pragma unroll
        for (int x = 0; x < 4; x += 2)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t mask = 0x000F000Fu << (4 * n);
            uint32_t a[4][4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              a[mt][0] = w[mt][x] & mask, a[mt][1] = (w[mt][x] >> 8) & mask;
              a[mt][2] = w[mt][x + 1] & mask, a[mt][3] = (w[mt][x + 1] >> 8) & mask;
              mma16816(u[mt], a[mt][0], a[mt][1], a[mt][2], a[mt][3], hi[n][x], hi[n][x + 1]);
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
              mma16816(u[mt], a[mt][0], a[mt][1], a[mt][2], a[mt][3], lo[n][x], lo[n][x + 1]);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float bk = (bz[1][e] + by[1][2 + e] + (bz[0][e] + by[0][2 + e]) * 0.0625f) * kap[e];
        const float ku = kap[e] * KeyPos<4>::unscale;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          u[mt][e] = fmaf(u[mt][e], ku, bk);
          u[mt][2 + e] = fmaf(u[mt][2 + e], ku, bk);
        }
      }
      __syncwarp();
      if (i + 2 < i1) issue_k(i + 2, st);
      const bool there = mbar_try_wait(bar_v, par_v);  // asked early, used below
      if (kind & kItMask) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (!visible(t0 + 16 * mt + gid + 8 * (x >> 1))) u[mt][x] = -INFINITY;
      }
      float mx0 = u[0][0], mx1 = u[0][1];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        mx0 = fmaxf(mx0, fmaxf(u[mt][0], u[mt][2]));
        mx1 = fmaxf(mx1, fmaxf(u[mt][1], u[mt][3]));
      }
      raise_max(mx0, mx1);
      // ---- weights, fp16, as the values' B operand (tokens down, head gid)
      uint32_t pa[4], pb[4];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        pa[mt] = movmatrix_trans(pack_h2(approx_weight(u[mt][0], m_run[0]), approx_weight(u[mt][1], m_run[1])));
        pb[mt] = movmatrix_trans(pack_h2(approx_weight(u[mt][2], m_run[0]), approx_weight(u[mt][3], m_run[1])));
      }
      failed = !__all_sync(0xFFFFFFFFu, there || mbar_wait_bounded(bar_v, par_v));
      if (failed) break;
      par_v ^= 1u;
      ready = i + 1 < i1 && mbar_try_wait(&bar_k[st ^ 1], (par_k >> (st ^ 1)) & 1u);
      if (kind & kItMask) {
        // What a masked token holds does not matter, infinities too: its scales
        // and zero points become 0 where they lie (lane l: tokens 2 l, 2 l + 1),
        // so that the products below need no branch.
        const uint32_t m = half_mask(visible(t0 + 2 * lane), visible(t0 + 2 * lane + 1));
        uint32_t* at = reinterpret_cast<uint32_t*>(ring + 2 * kPaK + vs_scale_off(2 * lane, 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          at[2 * j] &= m;
          at[128 + 2 * j] &= m;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy into the buffer
        __syncwarp();
      }
      {  // the group's largest value scale, times 2^fit, is in [1, 2)
        const uint4 sw = *reinterpret_cast<const uint4*>(rvb + lane * 16);
        const uint32_t s2 = __vmaxu2(__vmaxu2(sw.x, sw.y), __vmaxu2(sw.z, sw.w));
        const uint32_t smax = __reduce_max_sync(0xFFFFFFFFu, max(s2 & 0xFFFFu, s2 >> 16));
        const int fit = max(15 - (int)(smax >> 10), -14);  // (at -14 the scale is infinite or NaN)
        if (vx > fit || (vx < fit - kPaSlack && smax != 0u)) {
          const float f = pow2(fit - vx);
          vx = fit;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[mt][x] *= f;
        }
      }
      // 2^vx as fp16x2, to the scales or to the weights.  Branches around the 40
      // multiplications save 1 % at unit-normal values and cost as much at others.
      const uint32_t s_up = (uint32_t)(15 + max(vx, 0)) * 0x04000400u, p_down = (uint32_t)(15 + min(vx, 0)) * 0x04000400u;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint4 s0 = *reinterpret_cast<const uint4*>(rvb + kk * 128 + tig * 32);
        const uint4 s1 = *reinterpret_cast<const uint4*>(rvb + kk * 128 + tig * 32 + 16);
        const uint32_t sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
        const uint2 zz = *reinterpret_cast<const uint2*>(rvb + 512 + kk * 128 + tig * 32 + (gid & 3) * 8);
        const uint32_t za0 = (zz.x & z_mask) | z_one, za2 = (zz.y & z_mask) | z_one;
        const uint32_t va = h2_mul(pa[kk], p_down), vb = h2_mul(pb[kk], p_down);
        uint32_t bh[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bh[j][0] = h2_mul(va, h2_mul(sv[2 * j], s_up));
          bh[j][1] = h2_mul(vb, h2_mul(sv[2 * j + 1], s_up));
        }
        mma16816(dz, za0, 0u, za2, 0u, pa[kk], pb[kk]);
        const uint4 v0 = *reinterpret_cast<const uint4*>(rvb + 1024 + (2 * kk) * 512 + lane * 16);
        const uint4 v1 = *reinterpret_cast<const uint4*>(rvb + 1024 + (2 * kk + 1) * 512 + lane * 16);
        const uint32_t vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t vs[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) vs[x] = vw[x] >> 8;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          const int w = mt & 3;
          const uint32_t mask = 0x000F000Fu << (4 * (mt >> 2));
          mma16816(acc[mt], vw[2 * w] & mask, vs[2 * w] & mask, vw[2 * w + 1] & mask, vs[2 * w + 1] & mask,
                   bh[mt >> 1][0], bh[mt >> 1][1]);
        }
      }
    } else {
      // ---- 16 tail tokens, exact bf16 rows: keys are A rows as they lie
      uint32_t qw[16];
      {
        const bool ok = gid < G;
        int head;
        const int row = div_small(seg, hkv, head);
        const uint16_t* qr = p.q + (int64_t)row * p.q_row + (size_t)(head * G + (ok ? gid : 0)) * kD;
#pragma unroll
        for (int pp = 0; pp < 16; ++pp)
          qw[pp] = ok ? *reinterpret_cast<const uint32_t*>(qr + 16 * (pp >> 1) + 2 * tig + 8 * (pp & 1)) : 0u;
      }
      const int mi = lane >> 3, r = lane & 7;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        uint32_t a[4];
        ldmatrix4(a, smem_u32(rk) + tail_chunk(r + 8 * (mi & 1), 2 * ks + (mi >> 1)));
        mma_bf16(d, a[0], a[1], a[2], a[3], qw[2 * ks], qw[2 * ks + 1]);
      }
      __syncwarp();
      if (i + 2 < i1) issue_k(i + 2, st);
      const bool there = mbar_try_wait(bar_v, par_v);  // asked early, used below
      float u[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) u[x] = visible(t0 + gid + 8 * (x >> 1)) ? d[x] * p.kappa : -INFINITY;
      raise_max(fmaxf(u[0], u[2]), fmaxf(u[1], u[3]));
      // weights as a bf16 high part and its remainder: values are bf16 (fp16 would
      // not hold them), so the weights are too; 2^-17 of one at most is left out
      uint32_t ph[2], pl[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float w0 = approx_weight(u[2 * x], m_run[0]), w1 = approx_weight(u[2 * x + 1], m_run[1]);
        const uint32_t hi = pack_bf2(w0, w1);
        ph[x] = movmatrix_trans(hi);
        pl[x] = movmatrix_trans(pack_bf2(w0 - bf_lo(hi), w1 - bf_hi(hi)));
      }
      failed = !__all_sync(0xFFFFFFFFu, there || mbar_wait_bounded(bar_v, par_v));
      if (failed) break;
      par_v ^= 1u;
      ready = i + 1 < i1 && mbar_try_wait(&bar_k[st ^ 1], (par_k >> (st ^ 1)) & 1u);
      const uint32_t one = gid == 4 ? 0x3F803F80u : 0u;
      mma_bf16(dz, one, 0u, one, 0u, ph[0], ph[1]);
      mma_bf16(dz, one, 0u, one, 0u, pl[0], pl[1]);
      const uint32_t ma = half_mask(visible(t0 + 2 * tig), visible(t0 + 2 * tig + 1));
      const uint32_t mb = half_mask(visible(t0 + 2 * tig + 8), visible(t0 + 2 * tig + 9));
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        uint32_t a[4];
        ldmatrix4_trans(a, smem_u32(rvb) + tail_chunk(r + 8 * (mi >> 1), 2 * mt + (mi & 1)));
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        mma_bf16(o, a[0] & ma, a[1] & ma, a[2] & mb, a[3] & mb, ph[0], ph[1]);
        mma_bf16(o, a[0] & ma, a[1] & ma, a[2] & mb, a[3] & mb, pl[0], pl[1]);
        const float ps = pow2(vx - ((mt >> 2) ? 20 : 24));  // to the accumulator's scale
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[mt][x] = fmaf(o[x], ps, acc[mt][x]);
      }
    }
    __syncwarp();
    st ^= 1;
    if (i + 1 < i1) issue_v(i + 1);
    if (kind & kItLast) {
      if (own_start) {
        store_out();
      } else {
        store_partial(p.part_warp + ((size_t)blockIdx.x * kPgWarps + warp) * kPgPart);
        my_head_seg = seg;
      }
    } else if (i == i1 - 1) {
      my_tail_seg = seg;
      __syncwarp();
      store_partial(reinterpret_cast<float*>(ring));  // every copy has been used
    }
  }
  if (failed) {  // give up: the copies that may be in flight, once more (bounded)
    set_flag(p.flag, JFA_DEVERR_TIMEOUT);
    mbar_wait_bounded(&bar_k[0], par_k & 1u);
    mbar_wait_bounded(&bar_k[1], par_k >> 1);
    mbar_wait_bounded(bar_v, par_v);
  }
  if (lane == 0) {
    tail_seg[warp] = my_tail_seg;
    head_seg[warp] = my_head_seg;
    if (warp == 0) tail_seg[kPgWarps] = head_seg[kPgWarps] = -1;
  }
  __syncthreads();

  // ---- merge over the CTA's warps.  Runs: a segment's warps w .. e - 1 that
  // hold it last, and warp e if it ended there; the first warp may also have
  // ended a segment of the CTA before.  A warp takes a (run, head) at a time,
  // a lane 4 channels.
  auto seg_range = [&](int s, int& sa, int& sb) {
    int head;
    const int row = div_small(s, hkv, head), items = row_of(row).items;
    sa = pre[row] + head * items;
    sb = sa + items;
  };
  auto smem_part = [&](int w) { return reinterpret_cast<const float*>(pa_smem + w * kPaWarpBytes); };
  auto gmem_part = [&](int w) { return p.part_warp + ((size_t)blockIdx.x * kPgWarps + w) * kPgPart; };
  auto finish = [&](int s, int h, float M, float L, float4 O) {
    int head;
    const int row = div_small(s, hkv, head);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t at = (size_t)row * H + head * G + h;
    *reinterpret_cast<uint2*>(p.out + at * kD + 4 * lane) =
        make_uint2(pack_bf2(O.x * inv, O.y * inv), pack_bf2(O.z * inv, O.w * inv));
    if (lane == 0 && p.lse) p.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPaLn2;
  };
  {
    const int ts = lane < kPgWarps ? tail_seg[lane] : -1;
    const int before = __shfl_up_sync(0xFFFFFFFFu, ts, 1);
    const uint32_t starts = __ballot_sync(0xFFFFFFFFu, ts >= 0 && (lane == 0 || before != ts));
    const int head0 = head_seg[0], nruns = __popc(starts) + (head0 >= 0);
    for (int c = warp; c < nruns * G; c += kPgWarps) {
      const int run = c / G, h = c % G;
      // shared partials of the warps in mask and, if wh >= 0, warp wh's in the workspace
      int sg, wh;
      uint32_t mask = 0u;
      if (run == __popc(starts)) {
        sg = head0;
        wh = 0;
      } else {
        const int w0 = __fns(starts, 0, run + 1);
        sg = __shfl_sync(0xFFFFFFFFu, ts, w0);
        mask = __ballot_sync(0xFFFFFFFFu, ts == sg);
        const int w1 = w0 + __popc(mask);
        wh = head_seg[w1] == sg ? w1 : -1;
      }
      // a lane takes one partial's maximum and mass, then every lane 4 channels
      const bool mine = (mask >> lane) & 1u;
      const float* pl = smem_part(min(lane, kPgWarps - 1)) + h * kPartStride;
      const float* pg = gmem_part(wh < 0 ? 0 : wh) + h * kPartStride;
      float4 og = make_float4(0.f, 0.f, 0.f, 0.f);
      float mg = kPaMin, lg = 0.f;
      if (wh >= 0) {
        mg = pg[0];
        lg = pg[1];
        og = *reinterpret_cast<const float4*>(pg + 4 + 4 * lane);
      }
      const float ml = mine ? pl[0] : kPaMin;
      float M = ml;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
      M = fmaxf(__shfl_sync(0xFFFFFFFFu, M, 0), mg);
      const float fl = mine ? exp2_ftz(ml - M) : 0.f, fg = wh >= 0 ? exp2_ftz(mg - M) : 0.f;
      float L = mine ? fl * pl[1] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
      L = fmaf(lg, fg, __shfl_sync(0xFFFFFFFFu, L, 0));
      float4 O = make_float4(og.x * fg, og.y * fg, og.z * fg, og.w * fg);
#pragma unroll 4
      for (uint32_t m = mask; m;) {
        const int w = __ffs(m) - 1;
        m &= m - 1;
        const float f = __shfl_sync(0xFFFFFFFFu, fl, w);
        const float4 v = *reinterpret_cast<const float4*>(smem_part(w) + h * kPartStride + 4 + 4 * lane);
        O.x = fmaf(v.x, f, O.x);
        O.y = fmaf(v.y, f, O.y);
        O.z = fmaf(v.z, f, O.z);
        O.w = fmaf(v.w, f, O.w);
      }
      int sa, sb;
      seg_range(sg, sa, sb);
      if (sa >= r0 && sb <= r1) {
        finish(sg, h, M, L, O);
      } else {
        float* dst = p.part_cta + ((size_t)blockIdx.x * 2 + (sa < r0 ? 0 : 1)) * kPgPart + h * kPartStride;
        if (lane == 0) *reinterpret_cast<float2*>(dst) = make_float2(M, L);
        *reinterpret_cast<float4*>(dst + 4 + 4 * lane) = O;
      }
    }
  }

  // ---- the segments at the range's ends that other CTAs share
  __syncthreads();
  if (warp < 2 && lane == 0 && ends[warp].shared) {
    const RangeEnd e = ends[warp];
    const uint32_t mine = (uint32_t)(min(e.sa + e.items, r1) - max(e.sa, r0));
    __threadfence();  // the block's partials (before the barrier) come before its ticket
    if (atomicAdd(&p.ticket[e.seg], mine) + mine == (uint32_t)e.items) {
      __threadfence();  // the others' partials are read after it
      p.ticket[e.seg] = 0u;
      ends[warp].last = true;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int end = 0; end < 2; ++end) {
    if (!ends[end].last) continue;
    const int s = ends[end].seg, sa = ends[end].sa, ca = ends[end].ca, cb = ends[end].cb;
    // G heads, 12 / G warps each on every so-manieth CTA's partial
    const int per = kPgWarps / G, h = warp % G, sub = warp / G;
    auto part = [&](int c) {
      return p.part_cta + ((size_t)c * 2 + (sa < ctas.begin(c) ? 0 : 1)) * kPgPart + h * kPartStride;
    };
    float* buf = reinterpret_cast<float*>(pa_smem) + warp * kPartStride;
    if (sub < per) {
      float M = kPaMin, L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kAt = 8;  // partials whose loads are under way together
      for (int c0 = ca + sub; c0 <= cb; c0 += kAt * per) {
        float2 ml[kAt];
        float4 v[kAt];
#pragma unroll
        for (int i = 0; i < kAt; ++i) {
          const bool on = c0 + i * per <= cb;
          const float* src = part(on ? c0 + i * per : c0);
          ml[i] = on ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(kPaMin, 0.f);
          v[i] = on ? __ldcg(reinterpret_cast<const float4*>(src + 4 + 4 * lane)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float n = M;
#pragma unroll
        for (int i = 0; i < kAt; ++i) n = fmaxf(n, ml[i].x);
        const float fo = exp2_ftz(M - n);
        M = n;
        L *= fo;
        O.x *= fo;
        O.y *= fo;
        O.z *= fo;
        O.w *= fo;
#pragma unroll
        for (int i = 0; i < kAt; ++i) {
          const float f = exp2_ftz(ml[i].x - M);
          L = fmaf(ml[i].y, f, L);
          O.x = fmaf(v[i].x, f, O.x);
          O.y = fmaf(v[i].y, f, O.y);
          O.z = fmaf(v[i].z, f, O.z);
          O.w = fmaf(v[i].w, f, O.w);
        }
      }
      if (lane == 0) {
        buf[0] = M;
        buf[1] = L;
      }
      *reinterpret_cast<float4*>(buf + 4 + 4 * lane) = O;
    }
    __syncthreads();
    if (warp < G) {
      float M = kPaMin;
      for (int i = 0; i < per; ++i) M = fmaxf(M, reinterpret_cast<const float*>(pa_smem)[(h + i * G) * kPartStride]);
      float L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < per; ++i) {
        const float* src = reinterpret_cast<const float*>(pa_smem) + (h + i * G) * kPartStride;
        const float f = exp2_ftz(src[0] - M);
        const float4 v = *reinterpret_cast<const float4*>(src + 4 + 4 * lane);
        L = fmaf(src[1], f, L);
        O.x = fmaf(v.x, f, O.x);
        O.y = fmaf(v.y, f, O.y);
        O.z = fmaf(v.z, f, O.z);
        O.w = fmaf(v.w, f, O.w);
      }
      finish(s, h, M, L, O);
    }
    __syncthreads();
  }
}

int launch_paged_attend(const jfa_paged& c, const uint16_t* q, int64_t q_row, float scale, int window,
                        int sinks, uint8_t* ws, uint16_t* out, float* lse, cudaStream_t st) {
  const PagedWs w = paged_ws(c.batch, c.num_kv_heads);
  PagedAttendParams p;
  p.c = c;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.part_cta = reinterpret_cast<float*>(ws + w.off_cta);
  p.part_warp = reinterpret_cast<float*>(ws + w.off_warp);
  p.ticket = reinterpret_cast<uint32_t*>(ws + w.off_ticket);
  p.flag = reinterpret_cast<uint32_t*>(ws + w.off_flag);
  p.q_row = q_row;
  p.G = c.num_heads / c.num_kv_heads;
  p.window = window;
  p.sinks = sinks;
  p.kappa = scale * 1.4426950408889634f;
  static bool configured[64] = {false};  // per device: the attribute is set on each
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return JFA_ERR_CUDA;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    if (cudaFuncSetAttribute(paged_attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPaSmem) != cudaSuccess)
      return JFA_ERR_CUDA;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  const int sms = num_sms_current();
  return launch_pdl(paged_attend_kernel, dim3(sms < kPgMaxCtas ? sms : kPgMaxCtas), dim3(kPaThreads), (size_t)kPaSmem,
                    st, p) == cudaSuccess
             ? JFA_OK
             : JFA_ERR_CUDA;
}

}  // namespace jfa
