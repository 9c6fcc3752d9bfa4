// kvq_fp4_decode.cuh -- decode attention over the microscaled 4-bit cache.
//
//   O = softmax(q K^^T / sqrt(dh)) V^,  K^ = code * block scale * sK
//
// sK goes into the logits' scale and sV to the normalised output; the inner
// loop works on code * block scale, which is exact in f16.
//
// A unit of work is the page of HG neighbouring KV heads: 16 tokens of K and of
// V, HG * 1152 (576) contiguous bytes each.  The units of all (sequence, HG
// heads) segments, in order, are cut into one contiguous run per CTA, of equal
// cost (kvq_decode.cuh: CostSplit, a segment costing kPc units beside its own);
// a segment cut over CTAs leaves partial states (m, l, o) in the workspace, and
// the CTA that completes it merges them.  Where every segment is as long as the
// others (one sequence) or short, the host gives each a number of CTAs of its
// own and there is no plan to build (FIX).
//
// Consumer warp w of a CTA's 8 works on head w % HG of every (8 / HG)th unit from
// w / HG on, four units a step.  The HG warps of a unit share a ring of shared
// memory, which a producer warp fills (one bulk copy for the heads' K, one for
// their V) as they let go of its slots; there is no other barrier before a segment
// ends.  Then the 8 / HG warps of a head merge their states.  HG trades the two
// ends: eight heads a unit make few, long copies and no states to merge in a CTA; one
// head makes the fewest pieces per segment where few sequences are cut over many CTAs.
// The producer has a warpgroup of its own and leaves its registers to the
// consumers (setmaxnreg: 384 threads launch with 168 each; a step of four pages
// takes over 200).
//
// What bounds it: the conversions.  A page takes a warp about 270 instructions, half
// of them at half rate (64 conversions of two values, 64 products by scales, 16 matrix
// steps); the loop alone needs 296 cycles a page and SM quarter with two warps there
// (411 with one page a step), and about 450 in place, among copies and waits.  32 sequences
// of 2049 tokens, 8 KV heads: 31.1 us (11.2 us at the measured bandwidth); of them
// 2.5 the plan and the block ids, 2.3 the first pages, 16 the loop, 5 the states of
// cut segments.  128 sequences of 17 to 16384 tokens under a window: 63.4 us (31.5).
// One of 32768: 19.0 us (5.6).
//
// Per page, 16 tokens against the group's G <= 8 query heads:
//   S = K^ Q^T  m16n8k16 f16 matrix steps: lane (g, t) converts the codes of
//               token rows g and g + 8, dims t dh/4 .. (t + 1) dh/4, and
//               multiplies them by their block scales (exact)
//   P = 2^(x - m + 7) in binary32, rounded once to f16 (the 2^7 keeps small
//               weights out of f16's subnormals; it cancels in the division).  One f16
//               a weight: within 2^-11, which bf16's 2^-8 in the output covers (error
//               against 64 bits 0.0017 relative, with binary32 weights 0.0016 to 0.0017);
//               a second part would take half as many matrix steps again
//   O^T += V^T P^T  lane (g, t) holds dims g dh/8 .. (g + 1) dh/8 of tokens
//               t, t + 8, t + 4, t + 12: two tokens' codes are interleaved
//               four bits by four with two shifts and two selects per eight
//               values, so that one conversion gives the token pair that the
//               matrix step wants
#pragma once

#include <type_traits>

#include "kvq_decode.cuh"
#include "kvq_fp4.cuh"

namespace kvq {
namespace fp4 {

constexpr int kDecWarps = 8;                       // consumers: a step of four pages needs their registers
constexpr int kDecThreads = kDecWarps * 32 + 128;  // and the producer's warpgroup
constexpr int kConsumerRegs = 224, kProducerRegs = 40;  // 256 x 224 + 128 x 40 <= 384 x 168
// Units of a step, and the fixed cost of a piece in pages.  32 sequences of 2049 tokens / 128 of
// mixed lengths: one unit 33.0 / 69.8 us, two 31.7 / 65.9, four 30.7 / 62.9, five 31.2 / 64.9;
// a cost of 4 32.4 / 62.9, 8 30.7 / 62.9, 16 32.1 / 66.6.
constexpr int kStepUnits = 4;
constexpr int kPc = 8;
constexpr int kMaxHeads = 8;            // most KV heads of a unit
constexpr int kMaxDepth = 12;           // most slots of a ring
constexpr int kMinUnits = 32;           // least units of a CTA that shares a segment: a step a warp
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
  int HG, NG;         // KV heads of a unit, and units side by side (Hkv / HG)
  int P;              // CTAs that share the units
  int cps;            // FIX: CTAs of a segment
  int depth;          // slots of a ring
  uint32_t* ws_cnt;   // [B * Hkv] arrivals (zero between calls)
  float2* ws_ml;      // [slots][G]
  float* ws_o;        // [slots][G][DH]
  uint16_t* out;
  uint32_t* status;
  int withhold;       // test builds: unit of CTA 0's run that is never copied; -1
};

// Workspace: kvq_decode_attn's table of arrival counters, then per partial
// slot the (m, l) and o of one KV head's query heads.  CTA c's piece of segment
// s = b NG + (group of heads) has slots (c + s) HG .. + HG - 1, one a head: unique,
// as the CTAs' runs are ordered (FIX: c HG .. + HG - 1).
struct DecWs {
  size_t ml, o, total;
};
inline DecWs dec_ws(int B, int G, int Hkv, int DH, int P) {
  const size_t slots = static_cast<size_t>(P) * kMaxHeads + static_cast<size_t>(B) * Hkv;
  DecWs w;
  w.ml = KVQ_WS_COUNTER_BYTES;
  w.o = w.ml + round256(slots * G * sizeof(float2));
  w.total = w.o + round256(slots * G * DH * sizeof(float));
  return w;
}

// Dynamic shared memory (byte offsets); S: slots of all rings.
struct DecSmem {
  int bars, bad, ml, o, plan, total;
};
template <int DH>
__host__ __device__ inline DecSmem dec_smem(int S, int HG, int G, int B, bool fix) {
  DecSmem s;
  s.bars = S * 2 * HG * Page<DH>::kBytes;  // the ring is at 0; full[S], empty[S]
  s.bad = s.bars + 2 * S * 8;
  s.ml = (s.bad + 2 * S * 4 + 15) & ~15;   // (bad[S], last[S]); [warps][G] (m, l)
  s.o = s.ml + kDecWarps * G * 8;          // [warps][G][DH] o
  s.plan = s.o + kDecWarps * G * DH * 4;
  s.total = s.plan + (fix ? 0 : (3 * B + 2) * 4);
  return s;
}

// The pages' and costs' exclusive prefix sums over the sequences, in units of
// (sequence, all its segments): off[0 .. B], voff[0 .. B], and the checked lengths.
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
  uint64_t base = lane < warp ? warp_tot[lane] : 0;  // (at most 32 warps)
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) base += __shfl_xor_sync(kFull, base, d);
  uint64_t at = base + incl - local;
  for (int b = b0; b < b1; ++b) {
    const int n = off[b];
    const int pages = static_cast<int>(at & 0xFFFFFFFFu) * p.NG;
    off[b] = pages;
    voff[b] = pages + static_cast<int>(at >> 32) * p.NG * kPc;
    at += (static_cast<uint64_t>(n > 0) << 32) + static_cast<uint32_t>(n);
  }
  if (tid == kDecThreads - 1) {
    const int pages = static_cast<int>(at & 0xFFFFFFFFu) * p.NG;
    off[p.B] = pages;
    voff[p.B] = pages + static_cast<int>(at >> 32) * p.NG * kPc;
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

// Running maximum (of the raw dot products), what a dot product loses before its scale (the
// maximum, 0 while that is -inf), and the lane's share of the denominator, of heads 2t, 2t + 1.
struct Running {
  float m[2], c[2], l[2];
};

// NP staged pages of one warp: dot products, online softmax, weighted sum.
//   kpage[i], vpage[i]: the head's pages; tok0[i]: first token; skip[i]: masked out
template <int DH, int NP>
KVQ_DEVI void dec_pages(const uint8_t* const (&kpage)[NP], const uint8_t* const (&vpage)[NP], const int (&tok0)[NP], const bool (&skip)[NP],
                        const PieceView& pv, int g, int t, const uint32_t (&qb)[DH / 16][2],
                        float (&o)[DH / 16][4], Running& st) {
  using P = Page<DH>;
  constexpr int KW = DH / 32;  // code words of a K row that a lane converts
  constexpr int VW = DH / 64;  // of a V row
  // ---- S = K^ Q^T: x of (token g, head 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1)
  float x[NP][4];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint8_t* kp = kpage[i];
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
    const uint8_t* vp = vpage[i];
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
    st.c[0] = n0 == -INFINITY ? 0.f : n0;
    st.c[1] = n1 == -INFINITY ? 0.f : n1;
  }
  // ---- P^T as the B operand: head g of tokens (t, t + 8) and (t + 4, t + 12)
  uint32_t pb[NP][2];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    // The difference comes before the scale: the maximum's own exponent is then 7 however large the
    // logits are (7 - m ls, rounded, leaves it the rounding of m ls, which passes f16's range from
    // logits of 2^26 on).
    const float p0 = fast_exp2(fmaf(x[i][0] - st.c[0], pv.ls[0], kPBias)), p1 = fast_exp2(fmaf(x[i][1] - st.c[1], pv.ls[1], kPBias));
    const float p2 = fast_exp2(fmaf(x[i][2] - st.c[0], pv.ls[0], kPBias)), p3 = fast_exp2(fmaf(x[i][3] - st.c[1], pv.ls[1], kPBias));
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

// Sums of states j = 0 .. n - 1 (m, l, four dims of o) for E outputs, U states at a time
// with their loads together: l and o scaled by 2^(kMergeUnit (m - M)), M the largest m.  A
// state with m of -inf has l and o of 0, or NaN.
struct State {
  float m, l;
  float4 o;
};
template <int E, int U, typename Load>
KVQ_DEVI void merge_states(int n, State (&a)[E], const Load& load) {
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int j = 0; j < n; j += U) {
    State x[E][U];
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int y = 0; y < U; ++y) {
        x[e][y] = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        if (j + y < n) load(j + y, e, x[e][y]);
      }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float m = a[e].m;
#pragma unroll
      for (int y = 0; y < U; ++y) m = fmaxf(m, x[e][y].m);
      const float r = a[e].m == -INFINITY ? 1.f : fast_exp2((a[e].m - m) * kMergeUnit);
      a[e].l *= r;
      a[e].o.x *= r;
      a[e].o.y *= r;
      a[e].o.z *= r;
      a[e].o.w *= r;
      a[e].m = m;
#pragma unroll
      for (int y = 0; y < U; ++y) {
        const float w = x[e][y].m == -INFINITY ? 1.f : fast_exp2((x[e][y].m - m) * kMergeUnit);
        a[e].l += x[e][y].l * w;
        a[e].o.x += x[e][y].o.x * w;
        a[e].o.y += x[e][y].o.y * w;
        a[e].o.z += x[e][y].o.z * w;
        a[e].o.w += x[e][y].o.w * w;
      }
    }
  }
}

KVQ_DEVI void store_out(uint16_t* dst, const State& a, float sv) {
  const float inv = a.l > 0.f ? 1.f / a.l : 0.f;
  *reinterpret_cast<uint2*>(dst) = make_uint2(output2(a.o.x, a.o.y, inv, sv), output2(a.o.z, a.o.w, inv, sv));
}

KVQ_DEVI void head_barrier(int head, int threads) {
  if (threads == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(head + 1), "r"(threads) : "memory");
}

// The producer: copies the CTA's units into the rings.  Unit i of the run belongs to
// ring i % (8 / HG), as its unit k = i / (8 / HG), in slot k % depth.  Lane j takes
// units j, j + 32, ..., each as soon as its slot is free, the block ids looked up 32
// units ahead.  A lane looks at its slot's phase only once the unit that the slot held
// last has been copied (all units below the first pending one have): the phase before
// is then complete, and the parity cannot stand for one two back.
template <int DH, typename Segment>
KVQ_DEVI void decode_copies(const DecParams& p, uint8_t* smem, uint64_t* full, uint64_t* empty, volatile uint32_t* bad_s,
                            volatile int32_t* last_s, volatile uint32_t* abort_flag, int u0, int u1,
                            const Segment& segment) {
  const int lane = threadIdx.x & 31;
  const int rings = kDecWarps / p.HG, S = rings * p.depth;
  const int half = p.HG * Page<DH>::kBytes;
  const int total = u1 - u0;
  auto fetch = [&](int i, int& blk, int& gr) {
    blk = -1;
    gr = 0;
    if (i >= total) return;
    int b, pages, p0, L;
    segment(u0 + i, b, gr, pages, p0, L);
    const Visible vis = visible(p.window, p.sinks, L);
    const int col = p0 < vis.sink ? p0 : vis.first + p0 - vis.sink;
    if (col >= 0 && col < p.max_blocks)
      blk = __ldg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks + col);
  };
  int blk_next, gr_next;
  fetch(lane, blk_next, gr_next);
  uint32_t idle = 0;
  for (int base = 0; base < total; base += 32) {
    const int i = base + lane;
    const int ring = i % rings, k = i / rings, s = ring * p.depth + k % p.depth, round = k / p.depth;
    const int blk = blk_next, gr = gr_next;
    fetch(i + 32, blk_next, gr_next);
    bool pending = i < total;
    while (true) {
      const uint32_t left = __ballot_sync(kFull, pending);
      if (left == 0) break;
      bool moved = false;
      if (pending && i - S < base + __ffs(left) - 1 &&
          (round == 0 || mbar_test_wait(&empty[s], static_cast<uint32_t>((round - 1) & 1)))) {
        const bool bad = blk < 0 || blk >= p.num_blocks;
#ifdef KVQ_TEST_HOOKS
        const bool held = blockIdx.x == 0 && i == p.withhold;  // its full barrier never completes
#else
        constexpr bool held = false;
#endif
        if (!held) {
          bad_s[s] = bad;
          last_s[s] = k;  // (a bad page completes its phase too)
          if (bad) {
            flag_status(p.status, KVQ_DEV_BAD_BLOCK);
            mbar_arrive(&full[s]);
          } else {
            const int64_t at = (static_cast<int64_t>(blk) * p.Hkv + gr * p.HG) * Page<DH>::kBytes;
            uint8_t* dst = smem + s * 2 * half;
            mbar_arrive_expect_tx(&full[s], 2 * half);
            bulk_load(dst, p.kc + at, half, &full[s]);
            bulk_load(dst + half, p.vc + at, half, &full[s]);
          }
        }
        pending = false;
        moved = true;
      }
      if (__any_sync(kFull, moved)) {
        idle = 0;
      } else if (++idle > kMaxPolls || (((idle & 63u) == 0u) && __any_sync(kFull, *abort_flag != 0u))) {
        if (lane == 0 && !*abort_flag) {
          *abort_flag = 1u;
          flag_status(p.status, KVQ_DEV_WAIT_TIMEOUT);
        }
        return;
      } else {
        __nanosleep(40);
      }
    }
  }
}

// The CTA's run, unit by unit (see the head of the file).
template <int DH, bool FIX, typename Segment>
KVQ_DEVI void decode_run(const DecParams& p, uint8_t* smem, const DecSmem& sm, uint64_t* full, uint64_t* empty,
                         volatile uint32_t* bad_s, volatile uint32_t* abort_flag, uint32_t* merge_s,
                         const int32_t* voff, int u0, int u1, int V, int Pe, int fix_np, const Segment& segment) {
  using PG = Page<DH>;
  constexpr int MT = DH / 16;
  constexpr int kNP = kStepUnits;
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = p.HG * PG::kBytes, slot_bytes = 2 * half;
  const int g = lane >> 2, t = lane & 3;
  const int wph = kDecWarps / p.HG;          // warps of a head
  const int head = warp % p.HG, po = warp / p.HG;
  const int hthreads = wph * 32, htid = po * 32 + lane;  // the head's threads
  float2* cml = reinterpret_cast<float2*>(smem + sm.ml) + head * wph * p.G;      // [wph][G]
  float* co = reinterpret_cast<float*>(smem + sm.o) + head * wph * p.G * DH;     // [wph][G][DH]
  // the ring of this warp's group (the HG warps of unit w / HG)
  uint8_t* ring = smem + po * p.depth * slot_bytes;
  full += po * p.depth;
  empty += po * p.depth;
  bad_s += po * p.depth;
  bool dead = false;
  auto timed_out = [&] {  // no more copies, the rest is skipped
    dead = true;
    if (lane == 0 && !*abort_flag) {
      *abort_flag = 1u;
      flag_status(p.status, KVQ_DEV_WAIT_TIMEOUT);
    }
  };
  // The queries of the piece that begins at unit u: head g, dims t dh/4 .. (t + 1) dh/4.  They
  // are asked for before the piece before is merged, the first ones before the first pages
  // arrive (behind those 28 MB they took 3.8 us).
  uint32_t raw[DH / 8];
  auto load_q = [&](int u) {
    int b, gr, pages, p0, L;
    segment(u, b, gr, pages, p0, L);
    const uint4* src = reinterpret_cast<const uint4*>(
        p.q + (static_cast<int64_t>(b) * p.Hq + (gr * p.HG + head) * p.G + (g < p.G ? g : 0)) * DH + t * (DH / 4));
#pragma unroll
    for (int k = 0; k < DH / 32; ++k) {
      const uint4 w = g < p.G ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
      raw[4 * k] = w.x; raw[4 * k + 1] = w.y; raw[4 * k + 2] = w.z; raw[4 * k + 3] = w.w;
    }
  };
  if (u0 < u1) load_q(u0);
  // Merges a segment's np pieces (the first in partial slot `first`, the next HG slots on),
  // by this head's warps: thread (y, e) takes pieces y, y + K, ... of output float4 e.
  const int n4 = p.G * DH / 4;
  auto merge_pieces = [&](int np, int64_t first, int sigma, uint16_t* orow, float sv) {
    const int K = max(1, min(hthreads / n4, wph));  // [K][n4] fits co
    const float2* ml = p.ws_ml + first * p.G;
    const float4* ob = reinterpret_cast<const float4*>(p.ws_o) + first * n4;
    auto piece = [&](int j, int e, State& v) {
      const int64_t at = static_cast<int64_t>(j) * p.HG;
      const float2 z = __ldcg(ml + at * p.G + 4 * e / DH);
      v.m = z.x;
      v.l = z.y;
      v.o = __ldcg(ob + at * n4 + e);
    };
    if (K == 1) {  // four outputs of a thread together
      for (int e0 = htid; e0 < n4; e0 += 4 * hthreads) {
        State a[4];
        merge_states<4, 4>(np, a, [&](int j, int y, State& v) { if (e0 + y * hthreads < n4) piece(j, e0 + y * hthreads, v); });
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (e0 + y * hthreads < n4) store_out(orow + 4 * (e0 + y * hthreads), a[y], sv);
      }
      if (htid == 0) p.ws_cnt[sigma] = 0u;
      return;
    }
    float4* part = reinterpret_cast<float4*>(co);
    for (int x = htid; x < K * n4; x += hthreads) {
      const int y0 = x / n4, e = x - y0 * n4;
      State a[1];
      merge_states<1, 8>((np - y0 + K - 1) / K, a, [&](int j, int, State& v) { piece(y0 + j * K, e, v); });
      part[x] = a[0].o;
      if (4 * e % DH == 0) cml[y0 * p.G + 4 * e / DH] = make_float2(a[0].m, a[0].l);
    }
    if (htid == 0) p.ws_cnt[sigma] = 0u;
    head_barrier(head, hthreads);
    for (int e = htid; e < n4; e += hthreads) {
      State a[1];
      merge_states<1, 4>(K, a, [&](int y, int, State& v) {
        const float2 z = cml[y * p.G + 4 * e / DH];
        v.m = z.x;
        v.l = z.y;
        v.o = part[y * n4 + e];
      });
      store_out(orow + 4 * e, a[0], sv);
    }
    head_barrier(head, hthreads);
  };
  // The run's first piece where others go on with its segment and this run goes on too: its
  // arrival is looked at when the run ends (a CTA that ends with the segment mostly comes later).
  int held_np = 0, held_c = 0, held_b = 0, held_gr = 0;
  uint32_t held_count = 0;

  int i = po;    // this warp's next unit of the run, its slot
  int slot = 0;
  uint32_t parity = 0;
  for (int u = u0; u < u1;) {
    // ---- a piece: the part of one segment inside the run
    int b, gr, pages, p0;
    PieceView pv;
    segment(u, b, gr, pages, p0, pv.L);
    const Visible vis = visible(p.window, p.sinks, pv.L);
    pv.lo = vis.lo;
    pv.sinks = p.sinks;
    const int n = min(u1 - u, pages - p0);
    const int end = u - u0 + n;
    const int gkv = gr * p.HG + head;
    int np = FIX ? fix_np : 1, c_lo = FIX ? c / p.cps * p.cps : c;  // CTAs that hold the segment, the first
    if (!FIX && n < pages) {
      const CostSplit split(V, Pe);
      const int v_first = voff[b] + gr * (pages + kPc) + kPc;
      c_lo = split.cta_of(v_first);
      np = split.cta_of(v_first + pages - 1) - c_lo + 1;
    }
    // the group's queries, scaled by a power of two to f16
    const float sv = __ldg(p.vs + (p.per_head ? gkv : 0));
    uint32_t qb[MT][2];
    {
      const float sk = __ldg(p.ks + (p.per_head ? gkv : 0));
      const int qa = q_fragments<KVQ_FMT_E4M3, DH>(raw, qb);
      pv.ls[0] = bounded_scale(sk * __int_as_float((127 - __shfl_sync(kFull, qa, 8 * t)) << 23) * p.logit_scale);
      pv.ls[1] = bounded_scale(sk * __int_as_float((127 - __shfl_sync(kFull, qa, 8 * t + 4)) << 23) * p.logit_scale);
    }
    Running st;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = st.c[0] = st.c[1] = 0.f;
    float o[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

    auto step = [&](auto units) {
      constexpr int NP = decltype(units)::value;
      const uint8_t *kpage[NP], *vpage[NP];
      int tok0[NP], slots[NP];
      bool skip[NP];
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int pg = p0 + i + u0 - u;
        tok0[k] = (pg < vis.sink ? pg : vis.first + pg - vis.sink) * kTok;
        kpage[k] = ring + slot * slot_bytes + head * PG::kBytes;
        vpage[k] = kpage[k] + half;
        slots[k] = slot;
        if (!dead && !__all_sync(kFull, wait_or_abort(&full[slot], parity, abort_flag))) timed_out();
        skip[k] = bad_s[slot] != 0u;
        i += wph;
        if (++slot == p.depth) {
          slot = 0;
          parity ^= 1u;
        }
      }
      if (!dead) {
        dec_pages<DH, NP>(kpage, vpage, tok0, skip, pv, g, t, qb, o, st);
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < NP; ++k) mbar_arrive(&empty[slots[k]]);
        }
      }
    };
    while (i + (kNP - 1) * wph < end) step(std::integral_constant<int, kNP>());
    while (i < end) step(std::integral_constant<int, 1>());
    if (u + n < u1) load_q(u + n);

    // ---- the head's warps merge their states
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      st.l[0] += __shfl_xor_sync(kFull, st.l[0], d);
      st.l[1] += __shfl_xor_sync(kFull, st.l[1], d);
    }
    uint16_t* orow = p.out + (static_cast<int64_t>(b) * p.Hq + gkv * p.G) * DH;
    const int sigma = b * p.Hkv + gkv;
    const int64_t seg = FIX ? 0 : static_cast<int64_t>(b) * p.NG + gr;
    const int64_t mine = (c + seg) * p.HG + head;  // partial slot
    if (wph == 1) {  // a warp has the head to itself: its state is the piece's
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * t + e;
        if (h >= p.G) continue;
        if (np == 1) {
          const float inv = st.l[e] > 0.f ? 1.f / st.l[e] : 0.f;
          uint4* dst = reinterpret_cast<uint4*>(orow + h * DH + g * (DH / 8));
#pragma unroll
          for (int mt = 0; mt < MT; mt += 4)
            dst[mt / 4] = make_uint4(output2(o[mt][e], o[mt][2 + e], inv, sv),
                                     output2(o[mt + 1][e], o[mt + 1][2 + e], inv, sv),
                                     output2(o[mt + 2][e], o[mt + 2][2 + e], inv, sv),
                                     output2(o[mt + 3][e], o[mt + 3][2 + e], inv, sv));
        } else {
          if (g == 0) p.ws_ml[mine * p.G + h] = make_float2(merge_max(st.m[e], pv.ls[e]), st.l[e]);
          float4* dst = reinterpret_cast<float4*>(p.ws_o + (mine * p.G + h) * DH + g * (DH / 8));
#pragma unroll
          for (int mt = 0; mt < MT; mt += 2)
            dst[mt / 2] = make_float4(o[mt][e], o[mt][2 + e], o[mt + 1][e], o[mt + 1][2 + e]);
        }
      }
    } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = 2 * t + e;
      if (h >= p.G) continue;
      if (g == 0) cml[po * p.G + h] = make_float2(merge_max(st.m[e], pv.ls[e]), st.l[e]);
      float* dst = co + (po * p.G + h) * DH + g * (DH / 8);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        *reinterpret_cast<float2*>(dst + 2 * mt) = make_float2(o[mt][e], o[mt][2 + e]);
    }
    head_barrier(head, hthreads);
    for (int e = htid; e < n4; e += hthreads) {  // a float4 of one query head's output
      const int h = 4 * e / DH;
      State a[1];
      merge_states<1, 4>(wph, a, [&](int w, int, State& v) {
        const float2 z = cml[w * p.G + h];
        v.m = z.x;
        v.l = z.y;
        v.o = *reinterpret_cast<const float4*>(co + w * p.G * DH + 4 * e);
      });
      if (np == 1) {
        store_out(orow + 4 * e, a[0], sv);
      } else {
        reinterpret_cast<float4*>(p.ws_o)[mine * n4 + e] = a[0].o;
        if (4 * e % DH == 0) p.ws_ml[mine * p.G + h] = make_float2(a[0].m, a[0].l);
      }
    }
    }
    head_barrier(head, hthreads);
    if (np > 1) {
      // Publish the piece: the barrier above orders the threads' stores before the
      // acquire-release arrival, and an arrival that completes the count makes all
      // pieces visible to this head's warps.
      uint32_t count = 0;
      if (htid == 0) count = atom_add_acq_rel_gpu(p.ws_cnt + sigma, 1u) + 1;
      if (u + n < u1) {
        held_np = np;
        held_c = c_lo;
        held_b = b;
        held_gr = gr;
        held_count = count;
      } else {
        if (htid == 0) merge_s[head] = count == static_cast<uint32_t>(np);
        head_barrier(head, hthreads);
        if (merge_s[head]) merge_pieces(np, (c_lo + seg) * p.HG + head, sigma, orow, sv);
      }
    }
    u += n;
  }
  if (!FIX && held_np) {
    head_barrier(head, hthreads);
    if (htid == 0) merge_s[head] = held_count == static_cast<uint32_t>(held_np);
    head_barrier(head, hthreads);
    if (merge_s[head]) {
      const int gkv = held_gr * p.HG + head;
      merge_pieces(held_np, (held_c + static_cast<int64_t>(held_b) * p.NG + held_gr) * p.HG + head,
                   held_b * p.Hkv + gkv, p.out + (static_cast<int64_t>(held_b) * p.Hq + gkv * p.G) * DH,
                   __ldg(p.vs + (p.per_head ? gkv : 0)));
    }
  }
}

template <int DH, bool FIX>
__global__ void __launch_bounds__(kDecThreads, 1) decode_kernel(const __grid_constant__ DecParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t warp_tot[kDecThreads / 32];
  __shared__ int32_t bounds[2];
  __shared__ uint32_t merge_s[kDecWarps];
  __shared__ uint32_t abort_s;
  const int S = p.depth * (kDecWarps / p.HG);  // slots of all rings
  const DecSmem sm = dec_smem<DH>(S, p.HG, p.G, p.B, FIX);
  const int tid = threadIdx.x;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + sm.bars);  // [S] a unit landed
  uint64_t* empty = full + S;                                    // [S] its HG warps are done with it
  volatile uint32_t* bad_s = reinterpret_cast<volatile uint32_t*>(smem + sm.bad);
  volatile int32_t* last_s = reinterpret_cast<volatile int32_t*>(bad_s + S);  // [S] last unit put there
  volatile uint32_t* abort_flag = &abort_s;
  int32_t* off = reinterpret_cast<int32_t*>(smem + sm.plan);  // [B + 1]
  int32_t* len = off + p.B + 1;                               // [B]
  int32_t* voff = len + p.B;                                  // [B + 1]

  if (tid < S) {
    mbar_init(&full[tid], 1);
    mbar_init(&empty[tid], p.HG);
    last_s[tid] = -1;
    fence_mbar_init();
  }
  if (tid == 0) abort_s = 0u;
  pdl_wait();
  pdl_allow_next();

  const int c = blockIdx.x;
  int u0 = 0, u1 = 0, fix_b = 0, fix_g = 0, fix_len = 0, fix_pages = 0, fix_np = 1;
  int V = 0, Pe = 1;
  if (FIX) {
    const int seg = c / p.cps, part = c - seg * p.cps;
    fix_b = seg / p.NG;
    fix_g = seg - fix_b * p.NG;
    fix_len = __ldg(p.seq_lens + fix_b);
    if (fix_len < 0 || fix_len > p.max_blocks * kTok) {
      if (fix_g == 0 && part == 0 && tid == 0) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
      fix_len = 0;
    }
    fix_pages = visible(p.window, p.sinks, fix_len).count;
    fix_np = max(1, min(p.cps, fix_pages / kMinUnits));
    if (part >= fix_np) return;
    u0 = static_cast<int>(static_cast<int64_t>(fix_pages) * part / fix_np);
    u1 = static_cast<int>(static_cast<int64_t>(fix_pages) * (part + 1) / fix_np);
    if (fix_pages == 0) {  // nothing to attend to
      uint16_t* o = p.out + (static_cast<int64_t>(fix_b) * p.Hq + fix_g * p.HG * p.G) * DH;
      for (int i = tid; i < p.HG * p.G * DH; i += kDecThreads) o[i] = 0;
      return;
    }
    __syncthreads();
  } else {
    dec_plan(p, off, len, voff, warp_tot);
    for (int b = c; b < p.B; b += gridDim.x) {  // sequences with nothing to attend to
      if (off[b + 1] != off[b]) continue;
      uint16_t* o = p.out + static_cast<int64_t>(b) * p.Hq * DH;
      for (int i = tid; i < p.Hq * DH; i += kDecThreads) o[i] = 0;
    }
    const int W = off[p.B];
    V = voff[p.B];
    // a CTA has a unit for every warp of a head at least
    const int least = kDecWarps / p.HG;
    Pe = min(p.P, (W + least - 1) / least);
    const CostSplit split(V, Pe);
    if ((tid == 0 || tid == 32) && c < Pe)
      bounds[tid >> 5] = pages_before(off, voff, p.B, p.NG, split(c + (tid >> 5)), kPc);
    __syncthreads();
    if (c < Pe) {
      u0 = bounds[0];
      u1 = bounds[1];
    }
  }
  // the segment of unit u: sequence, group of heads, its units, u's place in it, tokens
  auto segment = [&](int u, int& b, int& gr, int& pages, int& p0, int& L) {
    if (FIX) {
      b = fix_b;
      gr = fix_g;
      pages = fix_pages;
      p0 = u;
      L = fix_len;
    } else {
      b = find_seq(off, p.B, u);
      pages = (off[b + 1] - off[b]) / p.NG;
      gr = (u - off[b]) / pages;
      p0 = u - off[b] - gr * pages;
      L = len[b];
    }
  };

  if (tid < kDecWarps * 32) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
    decode_run<DH, FIX>(p, smem, sm, full, empty, bad_s, abort_flag, merge_s, voff, u0, u1, V, Pe, fix_np, segment);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (tid < kDecWarps * 32 + 32)
      decode_copies<DH>(p, smem, full, empty, bad_s, last_s, abort_flag, u0, u1, segment);
  }
  __syncthreads();
  // after a timeout: the copies still in flight land (or the wait runs out) before the CTA leaves
  if (*abort_flag && tid == 0)
    for (int s = 0; s < S; ++s)
      if (last_s[s] >= 0) mbar_wait(&full[s], static_cast<uint32_t>((last_s[s] / p.depth) & 1));
}

}  // namespace fp4
}  // namespace kvq
