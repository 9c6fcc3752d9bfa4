// kvq_fp4_decode.cuh -- decode attention over the microscaled 4-bit cache.
//
//   O = softmax(q K^^T / sqrt(dh)) V^,  K^ = code * block scale * sK
//
// sK goes into the logits' scale and sV to the normalised output; the inner
// loop works on code * block scale, which is exact in f16.
//
// A unit of work is one KV head's page: 16 tokens of K and of V, 2304 (1152)
// bytes.  The units of all (sequence, KV head) segments, in order, are cut
// into one contiguous run per CTA, of equal cost (kvq_decode.cuh: CostSplit,
// a segment costing kPc pages beside its own); a segment cut over CTAs leaves
// partial states (m, l, o) in the workspace, and the CTA that completes it
// merges them.  Where the host can tell that every segment is short and each
// has an SM to itself, a CTA takes one whole segment, with no plan to build
// and nothing to merge (SEG).
//
// A CTA's run is cut once more into one contiguous run per warp, and each warp
// goes through its own: its lanes copy the warp's next pages (codes and scales
// of K, then of V: one bulk copy each) into the warp's own ring of shared
// memory, and it works through them two at a time, with no barrier between
// warps before the end.  A segment that lies whole in a warp's run is written
// by that warp; the others' states (a warp has at most two: of the segment
// that its run begins in and of the one that it ends in) are merged after one
// barrier.
// Per page, 16 tokens against the group's G <= 8 query heads:
//   S = K^ Q^T  m16n8k16 f16 matrix steps: lane (g, t) converts the codes of
//               token rows g and g + 8, dims t dh/4 .. (t + 1) dh/4, and
//               multiplies them by their block scales (exact)
//   P = 2^(x - m + 7) in binary32, rounded once to f16 (the 2^7 keeps small
//               weights out of f16's subnormals; it cancels in the division)
//   O^T += V^T P^T  lane (g, t) holds dims g dh/8 .. (g + 1) dh/8 of tokens
//               t, t + 8, t + 4, t + 12: two tokens' codes are interleaved
//               four bits by four with two shifts and two selects per eight
//               values, so that one conversion gives the token pair that the
//               matrix step wants
#pragma once

#include "kvq_decode.cuh"
#include "kvq_fp4.cuh"

namespace kvq {
namespace fp4 {

#ifndef KVQ_FP4_WARPS
#define KVQ_FP4_WARPS 16
#endif
#ifndef KVQ_FP4_CTAS
#define KVQ_FP4_CTAS 1
#endif
#ifndef KVQ_FP4_NP
#define KVQ_FP4_NP 2
#endif
#ifndef KVQ_FP4_PC
#define KVQ_FP4_PC 16
#endif
constexpr int kDecWarps = KVQ_FP4_WARPS;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecCtas = KVQ_FP4_CTAS;  // CTAs per SM
constexpr int kPc = KVQ_FP4_PC;         // fixed cost of a piece, in pages
constexpr int kMaxStages = 8;
constexpr float kPBias = 7.f;           // log2 of the factor that the weights carry

struct DecParams {
  const uint16_t* q;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  int max_blocks, B, Hq, Hkv, G;
  int64_t num_blocks;
  int window, sinks;
  const float* ks;
  const float* vs;
  int per_head;
  float logit_scale;  // log2(e) / sqrt(dh)
  int P;              // CTAs that share the units
  int S;              // ring stages of a warp
  uint32_t* ws_cnt;   // [B * Hkv] arrivals (zero between calls)
  float2* ws_ml;      // [slots][G]
  float* ws_o;        // [slots][G][DH]
  uint16_t* out;
  uint32_t* status;
};

// Workspace: kvq_decode_attn's table of arrival counters, then per partial
// slot the (m, l) and o of a group's heads.  The piece of segment sigma =
// b Hkv + g that CTA c holds has slot c + sigma (CTA ranges are ordered).
struct DecWs {
  size_t ml, o, total;
};
inline DecWs dec_ws(int B, int G, int Hkv, int DH, int P) {
  const size_t slots = static_cast<size_t>(P) + static_cast<size_t>(B) * Hkv;
  DecWs w;
  w.ml = KVQ_WS_COUNTER_BYTES;
  w.o = w.ml + round256(slots * G * sizeof(float2));
  w.total = w.o + round256(slots * G * DH * sizeof(float));
  return w;
}

// Dynamic shared memory (byte offsets).
struct DecSmem {
  int bars, bad, ml, o, plan, total;
};
template <int DH>
__host__ __device__ inline DecSmem dec_smem(int S, int G, int B, bool seg) {
  DecSmem s;
  s.bars = kDecWarps * S * 2 * Page<DH>::kBytes;  // the rings are at 0
  s.bad = s.bars + kDecWarps * S * 8;
  s.ml = (s.bad + kDecWarps * S * 4 + 15) & ~15;  // [warps][2][G] (m, l) of a warp's first and last piece
  s.o = s.ml + kDecWarps * 2 * G * 8;             // [warps][G][DH] o of the first; the last's is in the ring
  s.plan = s.o + kDecWarps * G * DH * 4;
  s.total = s.plan + (seg ? 0 : (3 * B + 2) * 4);
  return s;
}

// The pages' and costs' exclusive prefix sums over the sequences, in units of
// (sequence, all KV heads): off[0 .. B], voff[0 .. B], and the checked lengths.
KVQ_DEVI void dec_plan(const DecParams& p, int32_t* off, int32_t* len, int32_t* voff,
                       uint64_t* warp_tot) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kDecThreads - 1) / kDecThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  uint64_t local = 0;  // pages (low), segments that have any (high)
  for (int b = b0; b < b1; ++b) {
    int L = __ldg(p.seq_lens + b);
    if (L < 0 || L > p.max_blocks * kTok) {
      if (blockIdx.x == 0) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
      L = 0;
    }
    const int n = visible(p.window, p.sinks, L).count;
    len[b] = L;
    off[b] = n;
    local += (static_cast<uint64_t>(n > 0) << 32) + static_cast<uint32_t>(n);
  }
  uint64_t incl = local;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t o = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  uint64_t base = 0;
  for (int w = 0; w < warp; ++w) base += warp_tot[w];
  uint64_t at = base + incl - local;
  for (int b = b0; b < b1; ++b) {
    const int n = off[b];
    const int pages = static_cast<int>(at & 0xFFFFFFFFu) * p.Hkv;
    off[b] = pages;
    voff[b] = pages + static_cast<int>(at >> 32) * p.Hkv * kPc;
    at += (static_cast<uint64_t>(n > 0) << 32) + static_cast<uint32_t>(n);
  }
  if (tid == kDecThreads - 1) {
    const int pages = static_cast<int>(at & 0xFFFFFFFFu) * p.Hkv;
    off[p.B] = pages;
    voff[p.B] = pages + static_cast<int>(at >> 32) * p.Hkv * kPc;
  }
  __syncthreads();
}

// Bits of a where m is set, of b elsewhere.
KVQ_DEVI uint32_t select_bits(uint32_t a, uint32_t b, uint32_t m) { return (a & m) | (b & ~m); }

// What a warp needs to know of the piece that it works on.
struct PieceView {
  int lo, sinks, L;  // tokens [lo, L) and [0, sinks) are visible
  float ls[2];       // logit scale (log2 units) of heads 2t, 2t + 1
};

// Running maximum (of the raw dot products), the exponent's offset
// 7 - max * ls, and the lane's share of the denominator, of heads 2t, 2t + 1.
struct Running {
  float m[2], c[2], l[2];
};

// NP staged pages of one warp: dot products, online softmax, weighted sum.
//   page[i]: K page, V page behind it; tok0[i]: first token; skip[i]: masked out
template <int DH, int NP>
KVQ_DEVI void dec_pages(const uint8_t* const (&page)[NP], const int (&tok0)[NP], const bool (&skip)[NP],
                        const PieceView& pv, int g, int t, const uint32_t (&qb)[DH / 16][2],
                        float (&o)[DH / 16][4], Running& st) {
  using P = Page<DH>;
  constexpr int KW = DH / 32;  // code words of a K row that a lane converts
  constexpr int VW = DH / 64;  // of a V row
  // ---- S = K^ Q^T: x of (token g, head 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1)
  float x[NP][4];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint8_t* kp = page[i];
    uint32_t k0[KW], k1[KW], sc0[2], sc1[2];  // codes, block scales (in both halves) of rows g, g + 8
    if (DH == 128) {
      const uint4 a = *reinterpret_cast<const uint4*>(kp + g * P::kRow + t * 16);
      const uint4 b = *reinterpret_cast<const uint4*>(kp + (g + 8) * P::kRow + t * 16);
      k0[0] = a.x; k0[1] = a.y; k0[KW - 2] = a.z; k0[KW - 1] = a.w;
      k1[0] = b.x; k1[1] = b.y; k1[KW - 2] = b.z; k1[KW - 1] = b.w;
      const uint32_t s0 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(
          *reinterpret_cast<const uint16_t*>(kp + P::kScaleOff + g * 8 + 2 * t));
      const uint32_t s1 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(
          *reinterpret_cast<const uint16_t*>(kp + P::kScaleOff + (g + 8) * 8 + 2 * t));
      sc0[0] = prmt(s0, s0, 0x1010u);
      sc0[1] = prmt(s0, s0, 0x3232u);
      sc1[0] = prmt(s1, s1, 0x1010u);
      sc1[1] = prmt(s1, s1, 0x3232u);
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(kp + g * P::kRow + t * 8);
      const uint2 b = *reinterpret_cast<const uint2*>(kp + (g + 8) * P::kRow + t * 8);
      k0[0] = a.x; k0[1] = a.y;
      k1[0] = b.x; k1[1] = b.y;
      const uint32_t r0 = kp[P::kScaleOff + g * 4 + t], r1 = kp[P::kScaleOff + (g + 8) * 4 + t];
      const uint32_t s0 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(r0 | (r1 << 8)));
      sc0[0] = sc0[1] = prmt(s0, s0, 0x1010u);
      sc1[0] = sc1[1] = prmt(s0, s0, 0x3232u);
    }
    x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      uint32_t a[4], b[4];
      e2m1x8_to_f16x2x4(k0[w], a);
      e2m1x8_to_f16x2x4(k1[w], b);
      const uint32_t f0 = sc0[w * 2 / KW], f1 = sc1[w * 2 / KW];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t f[4] = {hmul2(a[2 * e], f0), hmul2(b[2 * e], f1), hmul2(a[2 * e + 1], f0),
                               hmul2(b[2 * e + 1], f1)};
        mma_f16(x[i], f, qb[2 * w + e][0], qb[2 * w + e][1]);
      }
    }
  }
  // ---- V's codes and scales of tokens t, t + 8, t + 4, t + 12
  uint32_t v[NP][4][VW], vs[NP][2];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint8_t* vp = page[i] + P::kBytes;
    uint32_t s4[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int row = t + 8 * (y & 1) + 4 * (y >> 1);
      if (DH == 128) {
        const uint2 w = *reinterpret_cast<const uint2*>(vp + row * P::kRow + g * 8);
        v[i][y][0] = w.x;
        v[i][y][VW - 1] = w.y;
        s4[y] = vp[P::kScaleOff + row * 8 + g];
      } else {
        v[i][y][0] = *reinterpret_cast<const uint32_t*>(vp + row * P::kRow + g * 4);
        s4[y] = vp[P::kScaleOff + row * 4 + (g >> 1)];
      }
    }
    vs[i][0] = s4[0] | (s4[1] << 8);
    vs[i][1] = s4[2] | (s4[3] << 8);
    // the edges of what is visible: masked keys get -inf, and masked values, which may hold
    // anything, a scale of 0 (their weight of 0 would not clear a NaN)
    if (skip[i] || tok0[i] + kTok > pv.L || (tok0[i] < pv.lo && tok0[i] + kTok > pv.sinks)) {
      auto seen = [&](int r) {
        const int tok = tok0[i] + r;
        return !skip[i] && tok < pv.L && (tok >= pv.lo || tok < pv.sinks);
      };
      if (!seen(g)) x[i][0] = x[i][1] = -INFINITY;
      if (!seen(g + 8)) x[i][2] = x[i][3] = -INFINITY;
      vs[i][0] &= (seen(t) ? 0xFFu : 0u) | (seen(t + 8) ? 0xFF00u : 0u);
      vs[i][1] &= (seen(t + 4) ? 0xFFu : 0u) | (seen(t + 12) ? 0xFF00u : 0u);
    }
  }
  // ---- online softmax; the maximum is raised only when it grows by over 8 (in log2 units)
  float mx0 = fmaxf(x[0][0], x[0][2]), mx1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
  for (int i = 1; i < NP; ++i) {
    mx0 = fmaxf(mx0, fmaxf(x[i][0], x[i][2]));
    mx1 = fmaxf(mx1, fmaxf(x[i][1], x[i][3]));
  }
  if (__any_sync(kFull, (mx0 - st.m[0]) * pv.ls[0] > kRescaleThreshold ||
                            (mx1 - st.m[1]) * pv.ls[1] > kRescaleThreshold)) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, d));
      mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, d));
    }
    const float n0 = fmaxf(st.m[0], mx0), n1 = fmaxf(st.m[1], mx1);
    // (-inf to -inf: nothing seen yet, nothing to scale)
    const float a0 = n0 == -INFINITY ? 1.f : fast_exp2((st.m[0] - n0) * pv.ls[0]);
    const float a1 = n1 == -INFINITY ? 1.f : fast_exp2((st.m[1] - n1) * pv.ls[1]);
    st.l[0] *= a0;
    st.l[1] *= a1;
#pragma unroll
    for (int mt = 0; mt < DH / 16; ++mt) {
      o[mt][0] *= a0;
      o[mt][2] *= a0;
      o[mt][1] *= a1;
      o[mt][3] *= a1;
    }
    st.m[0] = n0;
    st.m[1] = n1;
    // with nothing seen any finite offset keeps 2^-inf = 0 (and a NaN a NaN)
    st.c[0] = n0 == -INFINITY ? 0.f : fmaf(-n0, pv.ls[0], kPBias);
    st.c[1] = n1 == -INFINITY ? 0.f : fmaf(-n1, pv.ls[1], kPBias);
  }
  // ---- P^T as the B operand: head g of tokens (t, t + 8) and (t + 4, t + 12)
  uint32_t pb[NP][2];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float p0 = fast_exp2(fmaf(x[i][0], pv.ls[0], st.c[0])), p1 = fast_exp2(fmaf(x[i][1], pv.ls[1], st.c[1]));
    const float p2 = fast_exp2(fmaf(x[i][2], pv.ls[0], st.c[0])), p3 = fast_exp2(fmaf(x[i][3], pv.ls[1], st.c[1]));
    st.l[0] += p0 + p2;
    st.l[1] += p1 + p3;
    const uint32_t h0 = f32x2_to_f16x2(p0, p2), h1 = f32x2_to_f16x2(p1, p3);
    const int src = 4 * t + (g >> 1);
    const uint32_t pa0 = __shfl_sync(kFull, h0, src), pa1 = __shfl_sync(kFull, h1, src);
    const uint32_t pc0 = __shfl_sync(kFull, h0, src + 16), pc1 = __shfl_sync(kFull, h1, src + 16);
    pb[i][0] = (g & 1) ? pa1 : pa0;
    pb[i][1] = (g & 1) ? pc1 : pc0;
  }
  // ---- O^T += V^T P^T
  constexpr uint32_t kLow = 0x0F0F0F0Fu;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint32_t sp0 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(vs[i][0]));
    const uint32_t sp1 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(vs[i][1]));
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      // even dims and odd dims of the eight, the two tokens side by side
      uint32_t e0[4], d0[4], e1[4], d1[4];
      e2m1x8_to_f16x2x4(select_bits(v[i][0][w], v[i][1][w] << 4, kLow), e0);
      e2m1x8_to_f16x2x4(select_bits(v[i][0][w] >> 4, v[i][1][w], kLow), d0);
      e2m1x8_to_f16x2x4(select_bits(v[i][2][w], v[i][3][w] << 4, kLow), e1);
      e2m1x8_to_f16x2x4(select_bits(v[i][2][w] >> 4, v[i][3][w], kLow), d1);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t f[4] = {hmul2(e0[y], sp0), hmul2(d0[y], sp0), hmul2(e1[y], sp1), hmul2(d1[y], sp1)};
        mma_f16(o[4 * w + y], f, pb[i][0], pb[i][1]);
      }
    }
  }
}

// A segment that warps share, or CTAs: units [a, z) of it in this CTA.
struct Shared {
  int b, gkv, first, pages;  // first unit of the whole segment, its pages
  int wa, wz;                // first and last warp that hold some of it
  int np, c_lo;              // pieces over CTAs (1: all of it is here), the first one's CTA
};

template <int DH, bool SEG>
__global__ void __launch_bounds__(kDecThreads, kDecCtas) decode_kernel(const __grid_constant__ DecParams p) {
  using PG = Page<DH>;
  constexpr int MT = DH / 16;
  constexpr int kSlot = 2 * PG::kBytes;
  constexpr int kNP = KVQ_FP4_NP;  // pages of a step
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t warp_tot[kDecWarps];
  __shared__ int32_t bounds[2];
  __shared__ Shared list[kDecWarps + 1];
  __shared__ int list_n;
  __shared__ int32_t wstart[kDecWarps + 1];  // first unit of each warp's run
  __shared__ uint32_t merge_s[kDecWarps + 1];
  const DecSmem sm = dec_smem<DH>(p.S, p.G, p.B, SEG);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * p.S * kSlot;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + sm.bars) + warp * p.S;
  uint32_t* bad_s = reinterpret_cast<uint32_t*>(smem + sm.bad) + warp * p.S;
  float2* cml = reinterpret_cast<float2*>(smem + sm.ml);
  float* co = reinterpret_cast<float*>(smem + sm.o);
  int32_t* off = reinterpret_cast<int32_t*>(smem + sm.plan);  // [B + 1]
  int32_t* len = off + p.B + 1;                               // [B]
  int32_t* voff = len + p.B;                                  // [B + 1]

  if (lane < p.S) mbar_init(&full[lane], 1);
  if (tid == 0) list_n = 0;
  fence_mbar_init();
  __syncwarp();
  pdl_wait();
  pdl_allow_next();

  const int c = blockIdx.x;
  int u0 = 0, u1 = 0, seg_b = 0, seg_g = 0, seg_len = 0;
  int V = 0, Pe = 1;
  if (SEG) {
    seg_b = c / p.Hkv;
    seg_g = c - seg_b * p.Hkv;
    seg_len = __ldg(p.seq_lens + seg_b);
    if (seg_len < 0 || seg_len > p.max_blocks * kTok) {
      if (seg_g == 0 && tid == 0) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
      seg_len = 0;
    }
    u1 = visible(p.window, p.sinks, seg_len).count;
    if (u1 == 0) {  // nothing to attend to
      uint16_t* o = p.out + (static_cast<int64_t>(seg_b) * p.Hq + seg_g * p.G) * DH;
      for (int i = tid; i < p.G * DH; i += kDecThreads) o[i] = 0;
      return;
    }
  } else {
    dec_plan(p, off, len, voff, warp_tot);
    for (int b = c; b < p.B; b += gridDim.x) {  // sequences with nothing to attend to
      if (off[b + 1] != off[b]) continue;
      uint16_t* o = p.out + static_cast<int64_t>(b) * p.Hq * DH;
      for (int i = tid; i < p.Hq * DH; i += kDecThreads) o[i] = 0;
    }
    const int W = off[p.B];
    V = voff[p.B];
    // a CTA has a step for every warp at least
    Pe = min(p.P, (W + kDecWarps - 1) / kDecWarps);
    const CostSplit split(V, Pe);
    if ((tid == 0 || tid == 32) && c < Pe)
      bounds[tid >> 5] = pages_before(off, voff, p.B, p.Hkv, split(c + (tid >> 5)), kPc);
    __syncthreads();
    if (c < Pe) {
      u0 = bounds[0];
      u1 = bounds[1];
    }
  }

  // ---- this warp's run of pages [w0, w1)
  const int total = u1 - u0;
  auto run_start = [&](int w) { return u0 + static_cast<int>(static_cast<int64_t>(total) * w / kDecWarps); };
  auto warp_of = [&](int u) {  // the warp whose run holds unit u
    return static_cast<int>((static_cast<int64_t>(u - u0 + 1) * kDecWarps - 1) / total);
  };
  const int w0 = run_start(warp), w1 = run_start(warp + 1);
  const int mine = w1 - w0;
  if (lane < 2) wstart[warp + lane] = lane ? w1 : w0;  // (neighbours write the same)
  // the (sequence, KV head) segment of unit u
  auto segment = [&](int u, int& b, int& gkv, int& pages, int& p0, int& L) {
    if (SEG) {
      b = seg_b;
      gkv = seg_g;
      pages = total;
      p0 = u;
      L = seg_len;
    } else {
      b = find_seq(off, p.B, u);
      pages = (off[b + 1] - off[b]) / p.Hkv;
      gkv = (u - off[b]) / pages;
      p0 = u - off[b] - gkv * pages;
      L = len[b];
    }
  };
  // lane j holds the block id (and KV head) of the warp's page 32 i + j, fetched 32 pages ahead
  int blk_now = -1, head_now = 0, blk_next = -1, head_next = 0;
  auto fetch = [&](int k, int& blk, int& head) {
    blk = -1;
    head = 0;
    if (k >= mine) return;
    int b, pages, p0, L;
    segment(w0 + k, b, head, pages, p0, L);
    const Visible vis = visible(p.window, p.sinks, L);
    const int col = p0 < vis.sink ? p0 : vis.first + p0 - vis.sink;
    if (col >= 0 && col < p.max_blocks)
      blk = __ldg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks + col);
  };
  // The warp's next n pages into stages s, s + 1, ...: lanes 2i and 2i + 1 copy
  // K and V of page i.
  fetch(lane, blk_now, head_now);
  fetch(32 + lane, blk_next, head_next);
  int issued = 0;
  auto issue = [&](int s, int n) {
    const int k = issued + (lane >> 1);
    const int ba = __shfl_sync(kFull, blk_now, k & 31), ha = __shfl_sync(kFull, head_now, k & 31);
    int blk = ba, head = ha;
    if (((issued + n - 1) ^ issued) & 32) {  // the last of them are of the next 32
      const int bb = __shfl_sync(kFull, blk_next, k & 31), hb = __shfl_sync(kFull, head_next, k & 31);
      if ((k ^ issued) & 32) {
        blk = bb;
        head = hb;
      }
    }
    if (((issued + n) ^ issued) & 32) {
      blk_now = blk_next;
      head_now = head_next;
      fetch(((issued + n) | 31) + 1 + lane, blk_next, head_next);
    }
    if (lane < 2 * n) {
      int st = s + (lane >> 1);
      if (st >= p.S) st -= p.S;
      const bool bad = blk < 0 || blk >= p.num_blocks;
      if (!(lane & 1)) {
        bad_s[st] = bad;
        if (bad) {
          flag_status(p.status, KVQ_DEV_BAD_BLOCK);
          mbar_arrive(&full[st]);
        } else {
          mbar_arrive_expect_tx(&full[st], kSlot);
        }
      }
      __syncwarp((1u << (2 * n)) - 1u);  // (n <= 8)
      if (!bad)
        bulk_load(ring + st * kSlot + (lane & 1) * PG::kBytes,
                  ((lane & 1) ? p.vc : p.kc) + (static_cast<int64_t>(blk) * p.Hkv + head) * PG::kBytes,
                  PG::kBytes, &full[st]);
    }
    issued += n;
  };
  if (mine > 0) issue(0, min(p.S, mine));

  int done = 0, stage = 0;
  uint32_t parity = 0;
  bool dead = false;
  for (int u = w0; u < w1;) {
    // ---- a piece: the part of one segment inside the warp's run
    int b, gkv, pages, p0;
    PieceView pv;
    segment(u, b, gkv, pages, p0, pv.L);
    const Visible vis = visible(p.window, p.sinks, pv.L);
    pv.lo = vis.lo;
    pv.sinks = p.sinks;
    const int n = min(w1 - u, pages - p0);
    // the group's queries: head g, dims t dh/4 .. (t + 1) dh/4, scaled by a power of two to f16
    uint32_t qb[MT][2];
    {
      uint32_t raw[DH / 8];
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<int64_t>(b) * p.Hq + gkv * p.G + (g < p.G ? g : 0)) * DH + t * (DH / 4));
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        const uint4 w = g < p.G ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        raw[4 * i] = w.x; raw[4 * i + 1] = w.y; raw[4 * i + 2] = w.z; raw[4 * i + 3] = w.w;
      }
      const float ls = __ldg(p.ks + (p.per_head ? gkv : 0)) * p.logit_scale;
      const int qa = q_fragments<KVQ_FMT_E4M3, DH>(raw, qb);
      // (kept above 0 where it would underflow, so that it times -inf stays -inf)
      pv.ls[0] = fmaxf(ls * __int_as_float((127 - __shfl_sync(kFull, qa, 8 * t)) << 23), 0x1p-120f);
      pv.ls[1] = fmaxf(ls * __int_as_float((127 - __shfl_sync(kFull, qa, 8 * t + 4)) << 23), 0x1p-120f);
    }
    Running st;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = st.c[0] = st.c[1] = 0.f;
    float o[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

    for (int j = 0; j < n; j += kNP) {
      const uint8_t* page[kNP];
      int tok0[kNP];
      bool skip[kNP];
      const int first = stage, have = min(kNP, n - j);
#pragma unroll
      for (int i = 0; i < kNP; ++i) {
        const int pg = p0 + j + i;
        tok0[i] = (pg < vis.sink ? pg : vis.first + pg - vis.sink) * kTok;
        page[i] = ring + stage * kSlot;
        skip[i] = true;
        if (i < have) {
          if (!dead && !__all_sync(kFull, mbar_wait(&full[stage], parity))) {
            dead = true;  // the wait ran out: no more copies, the rest is skipped
            if (lane == 0) flag_status(p.status, KVQ_DEV_WAIT_TIMEOUT);
          }
          skip[i] = bad_s[stage] != 0;
          if (++stage == p.S) {
            stage = 0;
            parity ^= 1u;
          }
        }
      }
      if (!dead) {
        dec_pages<DH, kNP>(page, tok0, skip, pv, g, t, qb, o, st);
        __syncwarp();
        const int more = min(have, mine - issued);
        if (more > 0) issue(first, more);
      }
      if (!dead) done += have;
    }

#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      st.l[0] += __shfl_xor_sync(kFull, st.l[0], d);
      st.l[1] += __shfl_xor_sync(kFull, st.l[1], d);
    }
    if (n == pages) {  // the whole segment: its output
      const float sv = __ldg(p.vs + (p.per_head ? gkv : 0));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * t + e;
        if (h >= p.G) continue;
        const float f = st.l[e] > 0.f ? sv / st.l[e] : 0.f;
        uint4* dst = reinterpret_cast<uint4*>(
            p.out + (static_cast<int64_t>(b) * p.Hq + gkv * p.G + h) * DH + g * (DH / 8));
#pragma unroll
        for (int mt = 0; mt < MT; mt += 4)
          dst[mt / 4] = make_uint4(f32x2_to_bf16x2(o[mt][e] * f, o[mt][2 + e] * f),
                                   f32x2_to_bf16x2(o[mt + 1][e] * f, o[mt + 1][2 + e] * f),
                                   f32x2_to_bf16x2(o[mt + 2][e] * f, o[mt + 2][2 + e] * f),
                                   f32x2_to_bf16x2(o[mt + 3][e] * f, o[mt + 3][2 + e] * f));
      }
    } else {
      // its state: the warp's first piece, or its last (all of the ring's pages are used by then)
      const int k = u == w0 ? 0 : 1;
      float* dst0 = k == 0 ? co + warp * p.G * DH : reinterpret_cast<float*>(ring);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * t + e;
        if (h >= p.G) continue;
        // m in log2 units
        if (g == 0)
          cml[(warp * 2 + k) * p.G + h] = make_float2(st.m[e] == -INFINITY ? -INFINITY : st.m[e] * pv.ls[e], st.l[e]);
        float* dst = dst0 + h * DH + g * (DH / 8);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          *reinterpret_cast<float2*>(dst + 2 * mt) = make_float2(o[mt][e], o[mt][2 + e]);
      }
      const int a = u - p0;  // the segment's first unit
      if (lane == 0 && u == max(a, u0)) {  // the first of its pieces in the CTA announces it
        Shared s;
        s.b = b;
        s.gkv = gkv;
        s.first = a;
        s.pages = pages;
        s.wa = warp;
        s.wz = warp_of(min(a + pages, u1) - 1);
        s.np = 1;
        s.c_lo = 0;
        if (!SEG && (a < u0 || a + pages > u1)) {
          const CostSplit split(V, Pe);
          const int v_first = voff[b] + gkv * (pages + kPc) + kPc;
          s.c_lo = split.cta_of(v_first);
          s.np = split.cta_of(v_first + pages - 1) - s.c_lo + 1;
        }
        list[atomicAdd(&list_n, 1)] = s;
      }
    }
    u += n;
  }
  __syncthreads();

  // ---- the shared segments: a float4 of one head's output a thread
  const int n4 = p.G * DH / 4, shared = list_n;
  bool split_any = false;
  for (int i = tid; i < shared * n4; i += kDecThreads) {
    const int k = i / n4, e = i - k * n4, h = 4 * e / DH;
    const Shared s = list[k];
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w0_ = s.wa; w0_ <= s.wz; w0_ += 4) {  // four warps at a time, their loads together
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int w = w0_ + y;
        ml[y] = make_float2(-INFINITY, 0.f);
        v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w <= s.wz && wstart[w] < wstart[w + 1]) {
          const bool head = wstart[w] >= s.first;
          ml[y] = cml[(w * 2 + (head ? 0 : 1)) * p.G + h];
          v[y] = *reinterpret_cast<const float4*>(
              (head ? co + w * p.G * DH : reinterpret_cast<const float*>(smem + w * p.S * kSlot)) + 4 * e);
        }
      }
      const float nm = fmaxf(fmaxf(M, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
      const float r = M == -INFINITY ? 1.f : fast_exp2(M - nm);
      l *= r;
      acc.x *= r;
      acc.y *= r;
      acc.z *= r;
      acc.w *= r;
      M = nm;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float a = ml[y].x == -INFINITY ? 1.f : fast_exp2(ml[y].x - M);  // (-inf: l and o are 0, or NaN)
        l += ml[y].y * a;
        acc.x += v[y].x * a;
        acc.y += v[y].y * a;
        acc.z += v[y].z * a;
        acc.w += v[y].w * a;
      }
    }
    if (s.np == 1) {
      const float f = l > 0.f ? __ldg(p.vs + (p.per_head ? s.gkv : 0)) / l : 0.f;
      *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(s.b) * p.Hq + s.gkv * p.G) * DH + 4 * e) =
          make_uint2(f32x2_to_bf16x2(acc.x * f, acc.y * f), f32x2_to_bf16x2(acc.z * f, acc.w * f));
    } else {
      const int64_t slot = c + static_cast<int64_t>(s.b) * p.Hkv + s.gkv;
      *reinterpret_cast<float4*>(p.ws_o + slot * p.G * DH + 4 * e) = acc;
      if (4 * e % DH == 0) p.ws_ml[slot * p.G + h] = make_float2(M, l);
    }
  }
  if (!SEG) {
    for (int k = 0; k < shared; ++k) split_any |= list[k].np > 1;
    if (split_any) {  // the same for every thread
      // Publish the pieces: the barrier orders every thread's stores before the
      // acquire-release arrivals, and an arrival that completes a count makes all
      // pieces of that segment visible to this CTA.
      __syncthreads();
      if (tid < shared) {
        const Shared s = list[tid];
        merge_s[tid] = s.np > 1 && atom_add_acq_rel_gpu(p.ws_cnt + static_cast<int64_t>(s.b) * p.Hkv + s.gkv, 1u) + 1 ==
                                       static_cast<uint32_t>(s.np);
      }
      __syncthreads();
      const int K = max(1, min(kDecThreads / n4, kDecWarps));  // [K][n4] fits co
      float4* part = reinterpret_cast<float4*>(co);
      for (int k = 0; k < shared; ++k) {
        if (!merge_s[k]) continue;
        const Shared s = list[k];
        // thread (y, e): the pieces y, y + K, ... of output float4 e
        const int64_t sigma = static_cast<int64_t>(s.b) * p.Hkv + s.gkv;
        const float2* ml = p.ws_ml + (s.c_lo + sigma) * p.G;
        const float4* ob = reinterpret_cast<const float4*>(p.ws_o + (s.c_lo + sigma) * p.G * DH);
        for (int i = tid; i < K * n4; i += kDecThreads) {
          const int y0 = i / n4, e = i - y0 * n4, h = 4 * e / DH;
          float M = -INFINITY, l = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int j = y0; j < s.np; j += 8 * K) {  // eight pieces at a time, their loads together
            float2 m8[8];
            float4 v8[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const int x = j + y * K;
              m8[y] = x < s.np ? __ldcg(ml + static_cast<int64_t>(x) * p.G + h) : make_float2(-INFINITY, 0.f);
              v8[y] = x < s.np ? __ldcg(ob + static_cast<int64_t>(x) * n4 + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float nm = M;
#pragma unroll
            for (int y = 0; y < 8; ++y) nm = fmaxf(nm, m8[y].x);
            const float a = M == -INFINITY ? 1.f : fast_exp2(M - nm);
            l *= a;
            acc.x *= a;
            acc.y *= a;
            acc.z *= a;
            acc.w *= a;
            M = nm;
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const float w = m8[y].x == -INFINITY ? 1.f : fast_exp2(m8[y].x - M);
              l += m8[y].y * w;
              acc.x += v8[y].x * w;
              acc.y += v8[y].y * w;
              acc.z += v8[y].z * w;
              acc.w += v8[y].w * w;
            }
          }
          part[i] = acc;
          if (4 * e % DH == 0) cml[y0 * p.G + h] = make_float2(M, l);
        }
        __syncthreads();
        for (int e = tid; e < n4; e += kDecThreads) {
          const int h = 4 * e / DH;
          float M = -INFINITY, l = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int y = 0; y < K; ++y) M = fmaxf(M, cml[y * p.G + h].x);
          for (int y = 0; y < K; ++y) {
            const float2 x = cml[y * p.G + h];
            const float4 v = part[y * n4 + e];
            const float w = x.x == -INFINITY ? 1.f : fast_exp2(x.x - M);
            l += x.y * w;
            acc.x += v.x * w;
            acc.y += v.y * w;
            acc.z += v.z * w;
            acc.w += v.w * w;
          }
          const float f = l > 0.f ? __ldg(p.vs + (p.per_head ? s.gkv : 0)) / l : 0.f;
          *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(s.b) * p.Hq + s.gkv * p.G) * DH + 4 * e) =
              make_uint2(f32x2_to_bf16x2(acc.x * f, acc.y * f), f32x2_to_bf16x2(acc.z * f, acc.w * f));
        }
        if (tid == 0) p.ws_cnt[sigma] = 0u;
        __syncthreads();
      }
    }
  }
  // after a timeout: the copies still in flight land (or the wait runs out) before the CTA leaves
  for (; dead && done < issued; ++done)
    mbar_wait(&full[done % p.S], static_cast<uint32_t>((done / p.S) & 1));
}

}  // namespace fp4
}  // namespace kvq
