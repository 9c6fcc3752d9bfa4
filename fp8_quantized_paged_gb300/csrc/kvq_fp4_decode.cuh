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
// A CTA's 16 warps take its pages in turn, each on its own: a warp's lane 0
// copies the warp's next pages (codes and scales of K, then of V: one bulk
// copy each) into the warp's own ring of shared memory, and all of it works
// through them, with no barrier between warps before the segment's end.
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
  int ring, bars, bad, comb, plan, total;
};
template <int DH>
__host__ __device__ inline DecSmem dec_smem(int S, int G, int B, bool seg) {
  DecSmem s;
  s.ring = 0;
  s.bars = kDecWarps * S * 2 * Page<DH>::kBytes;
  s.bad = s.bars + kDecWarps * S * 8;
  s.comb = (s.bad + kDecWarps * S * 4 + 15) & ~15;
  // [warps][G] (m, l), [warps][G][DH] o
  s.plan = s.comb + kDecWarps * G * (DH + 2) * 4;
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

KVQ_DEVI uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
KVQ_DEVI uint32_t lds16(uint32_t addr) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr));
  return r;
}
KVQ_DEVI uint32_t lds8(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}

// Bits of a where m is set, of b elsewhere.
KVQ_DEVI uint32_t select_bits(uint32_t a, uint32_t b, uint32_t m) { return (a & m) | (b & ~m); }

// One staged page of one warp: logits, online softmax, weighted sum.
//   kp, vp: shared addresses; tok0: first token; [lo, L) and [0, sinks) visible
template <int DH>
KVQ_DEVI void dec_page(uint32_t kp, uint32_t vp, int tok0, int lo, int sinks, int L, bool bad, int g,
                       int t, const uint32_t (&qb)[DH / 16][2], float (&o)[DH / 16][4],
                       SoftmaxState& st, float ls0, float ls1) {
  using P = Page<DH>;
  constexpr int KW = DH / 32;  // code words of a K row that a lane converts
  constexpr int VW = DH / 64;  // of a V row
  // ---- S = K^ Q^T
  uint32_t k0[KW], k1[KW];
  uint32_t sc0[2], sc1[2];  // block scales of rows g, g + 8, in both halves
  if (DH == 128) {
    const uint4 a = lds128(kp + g * P::kRow + t * 16), b = lds128(kp + (g + 8) * P::kRow + t * 16);
    k0[0] = a.x; k0[1] = a.y; k0[KW - 2] = a.z; k0[KW - 1] = a.w;
    k1[0] = b.x; k1[1] = b.y; k1[KW - 2] = b.z; k1[KW - 1] = b.w;
    const uint32_t s0 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(lds16(kp + P::kScaleOff + g * 8 + 2 * t));
    const uint32_t s1 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(lds16(kp + P::kScaleOff + (g + 8) * 8 + 2 * t));
    sc0[0] = prmt(s0, s0, 0x1010u);
    sc0[1] = prmt(s0, s0, 0x3232u);
    sc1[0] = prmt(s1, s1, 0x1010u);
    sc1[1] = prmt(s1, s1, 0x3232u);
  } else {
    const uint2 a = lds64(kp + g * P::kRow + t * 8), b = lds64(kp + (g + 8) * P::kRow + t * 8);
    k0[0] = a.x; k0[1] = a.y;
    k1[0] = b.x; k1[1] = b.y;
    const uint32_t r0 = lds8(kp + P::kScaleOff + g * 4 + t), r1 = lds8(kp + P::kScaleOff + (g + 8) * 4 + t);
    const uint32_t s0 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(r0 | (r1 << 8)));
    sc0[0] = sc0[1] = prmt(s0, s0, 0x1010u);
    sc1[0] = sc1[1] = prmt(s0, s0, 0x3232u);
  }
  float s[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[0][i] = s[1][i] = 0.f;
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
      mma_f16(s[e], f, qb[2 * w + e][0], qb[2 * w + e][1]);
    }
  }
  // ---- V's codes and scales, in flight while the softmax runs
  const int row[4] = {t, t + 8, t + 4, t + 12};
  uint32_t v[4][VW], vs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (DH == 128) {
      const uint2 w = lds64(vp + row[i] * P::kRow + g * 8);
      v[i][0] = w.x;
      v[i][VW - 1] = w.y;
      vs[i] = lds8(vp + P::kScaleOff + row[i] * 8 + g);
    } else {
      v[i][0] = lds32(vp + row[i] * P::kRow + g * 4);
      vs[i] = lds8(vp + P::kScaleOff + row[i] * 4 + (g >> 1));
    }
  }
  // ---- softmax: x of (token g, head 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1)
  float x[4], pr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = (s[0][i] + s[1][i]) * ((i & 1) ? ls1 : ls0);
  const bool edge = bad || tok0 + kTok > L || (tok0 < lo && tok0 + kTok > sinks);
  auto seen = [&](int r) { return !bad && tok0 + r < L && (tok0 + r >= lo || tok0 + r < sinks); };
  if (edge) {
    if (!seen(g)) x[0] = x[1] = -INFINITY;
    if (!seen(g + 8)) x[2] = x[3] = -INFINITY;
    // a masked token may hold anything; its weight is 0, so its scale has to be finite
#pragma unroll
    for (int i = 0; i < 4; ++i) vs[i] = seen(row[i]) ? vs[i] : 0u;
  }
  const float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
  if (__any_sync(kFull, mx0 > st.m[0] + kRescaleThreshold || mx1 > st.m[1] + kRescaleThreshold)) {
    float n0 = mx0, n1 = mx1;
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      n0 = fmaxf(n0, __shfl_xor_sync(kFull, n0, d));
      n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, d));
    }
    n0 = fmaxf(st.m[0], n0);
    n1 = fmaxf(st.m[1], n1);
    const float a0 = n0 == -INFINITY ? 1.f : fast_exp2(st.m[0] - n0);
    const float a1 = n1 == -INFINITY ? 1.f : fast_exp2(st.m[1] - n1);
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
  }
  const float c0 = st.m[0] - kPBias, c1 = st.m[1] - kPBias;
#pragma unroll
  for (int i = 0; i < 4; ++i) pr[i] = x[i] == -INFINITY ? 0.f : fast_exp2(x[i] - ((i & 1) ? c1 : c0));
  st.l[0] += pr[0] + pr[2];
  st.l[1] += pr[1] + pr[3];
  // ---- P^T as the B operand: head g of tokens (t, t + 8) and (t + 4, t + 12)
  const uint32_t h0 = f32x2_to_f16x2(pr[0], pr[2]), h1 = f32x2_to_f16x2(pr[1], pr[3]);
  const int src = 4 * t + (g >> 1);
  const uint32_t pa0 = __shfl_sync(kFull, h0, src), pa1 = __shfl_sync(kFull, h1, src);
  const uint32_t pb0 = __shfl_sync(kFull, h0, src + 16), pb1 = __shfl_sync(kFull, h1, src + 16);
  const uint32_t b0 = (g & 1) ? pa1 : pa0, b1 = (g & 1) ? pb1 : pb0;
  // ---- O^T += V^T P^T
  const uint32_t sp0 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(vs[0] | (vs[1] << 8)));
  const uint32_t sp1 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(vs[2] | (vs[3] << 8)));
  constexpr uint32_t kLow = 0x0F0F0F0Fu;
#pragma unroll
  for (int w = 0; w < VW; ++w) {
    // even dims and odd dims of the eight, the two tokens side by side
    uint32_t e0[4], d0[4], e1[4], d1[4];
    e2m1x8_to_f16x2x4(select_bits(v[0][w], v[1][w] << 4, kLow), e0);
    e2m1x8_to_f16x2x4(select_bits(v[0][w] >> 4, v[1][w], kLow), d0);
    e2m1x8_to_f16x2x4(select_bits(v[2][w], v[3][w] << 4, kLow), e1);
    e2m1x8_to_f16x2x4(select_bits(v[2][w] >> 4, v[3][w], kLow), d1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t f[4] = {hmul2(e0[i], sp0), hmul2(d0[i], sp0), hmul2(e1[i], sp1), hmul2(d1[i], sp1)};
      mma_f16(o[4 * w + i], f, b0, b1);
    }
  }
}

template <int DH, bool SEG>
__global__ void __launch_bounds__(kDecThreads, kDecCtas) decode_kernel(const __grid_constant__ DecParams p) {
  using PG = Page<DH>;
  constexpr int MT = DH / 16;
  constexpr int kSlot = 2 * PG::kBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t warp_tot[kDecWarps];
  __shared__ int32_t bounds[2];
  __shared__ uint32_t merge_s;
  const DecSmem sm = dec_smem<DH>(p.S, p.G, p.B, SEG);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + sm.ring + warp * p.S * kSlot;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + sm.bars) + warp * p.S;
  uint32_t* bad_s = reinterpret_cast<uint32_t*>(smem + sm.bad) + warp * p.S;
  float2* cml = reinterpret_cast<float2*>(smem + sm.comb);        // [warps][G]
  float* co = reinterpret_cast<float*>(cml + kDecWarps * p.G);    // [warps][G][DH]
  int32_t* off = reinterpret_cast<int32_t*>(smem + sm.plan);      // [B + 1]
  int32_t* len = off + p.B + 1;                                   // [B]
  int32_t* voff = len + p.B;                                      // [B + 1]

  if (lane < p.S) mbar_init(&full[lane], 1);
  fence_mbar_init();
  __syncwarp();
  pdl_wait();
  pdl_allow_next();

  const int c = blockIdx.x;
  int u0 = 0, u1 = 0, seg_b = 0, seg_g = 0, seg_len = 0;
  Visible seg_vis = {};
  int V = 0, Pe = 1;
  if (SEG) {
    seg_b = c / p.Hkv;
    seg_g = c - seg_b * p.Hkv;
    seg_len = __ldg(p.seq_lens + seg_b);
    if (seg_len < 0 || seg_len > p.max_blocks * kTok) {
      if (seg_g == 0 && tid == 0) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
      seg_len = 0;
    }
    seg_vis = visible(p.window, p.sinks, seg_len);
    u1 = seg_vis.count;
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
    // a CTA has a page for every warp at least
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
  const CostSplit split(V, Pe);

  // ---- this warp's pages: units u0 + warp, u0 + warp + 16, ...
  const int total = u1 - u0;
  const int mine = total > warp ? (total - warp + kDecWarps - 1) / kDecWarps : 0;
  // lane j holds the block id (and KV head) of the warp's page 32 i + j, fetched 32 pages ahead
  int blk_now = -1, head_now = 0, blk_next = -1, head_next = 0;
  auto fetch = [&](int k, int& blk, int& head) {
    blk = -1;
    head = 0;
    if (k >= mine) return;
    const int u = u0 + warp + k * kDecWarps;
    int b, pg;
    Visible vis;
    if (SEG) {
      b = seg_b;
      head = seg_g;
      pg = u;
      vis = seg_vis;
    } else {
      b = find_seq(off, p.B, u);
      const int pages = (off[b + 1] - off[b]) / p.Hkv;
      head = (u - off[b]) / pages;
      pg = u - off[b] - head * pages;
      vis = visible(p.window, p.sinks, len[b]);
    }
    const int col = pg < vis.sink ? pg : vis.first + pg - vis.sink;
    if (col >= 0 && col < p.max_blocks) blk = __ldg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks + col);
  };
  int issued = 0;
  auto issue = [&](int s) {  // the warp's next page into stage s = issued % S (all lanes)
    if ((issued & 31) == 0) {
      if (issued == 0) fetch(lane, blk_now, head_now);
      else {
        blk_now = blk_next;
        head_now = head_next;
      }
      fetch(issued + 32 + lane, blk_next, head_next);
    }
    const int blk = __shfl_sync(kFull, blk_now, issued & 31), head = __shfl_sync(kFull, head_now, issued & 31);
    if (lane == 0) {
      const bool bad = blk < 0 || blk >= p.num_blocks;
      bad_s[s] = bad;
      if (bad) {
        flag_status(p.status, KVQ_DEV_BAD_BLOCK);
        mbar_arrive(&full[s]);
      } else {
        const int64_t at = (static_cast<int64_t>(blk) * p.Hkv + head) * PG::kBytes;
        mbar_arrive_expect_tx(&full[s], kSlot);
        bulk_load(ring + s * kSlot, p.kc + at, PG::kBytes, &full[s]);
        bulk_load(ring + s * kSlot + PG::kBytes, p.vc + at, PG::kBytes, &full[s]);
      }
    }
    ++issued;
  };
  while (issued < p.S && issued < mine) issue(issued);

  int done = 0, stage = 0;
  uint32_t parity = 0;
  bool dead = false;
  int pos = 0;  // units of the CTA's earlier pieces
  for (int u = u0; u < u1;) {
    // ---- a piece: the part of one (sequence, KV head) segment inside [u0, u1)
    int b, gkv, pages, p0, L;
    if (SEG) {
      b = seg_b;
      gkv = seg_g;
      pages = total;
      p0 = 0;
      L = seg_len;
    } else {
      b = find_seq(off, p.B, u);
      pages = (off[b + 1] - off[b]) / p.Hkv;
      gkv = (u - off[b]) / pages;
      p0 = u - off[b] - gkv * pages;
      L = len[b];
    }
    const Visible vis = visible(p.window, p.sinks, L);
    const int n = min(u1 - u, pages - p0);
    const bool single = SEG || n == pages;
    const float ls = __ldg(p.ks + (p.per_head ? gkv : 0)) * p.logit_scale;
    const float sv = __ldg(p.vs + (p.per_head ? gkv : 0));
    // the group's queries: head g, dims t dh/4 .. (t + 1) dh/4, scaled by a power of two to f16
    uint32_t raw[DH / 8], qb[MT][2];
    {
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<int64_t>(b) * p.Hq + gkv * p.G + (g < p.G ? g : 0)) * DH + t * (DH / 4));
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        const uint4 w = g < p.G ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        raw[4 * i] = w.x; raw[4 * i + 1] = w.y; raw[4 * i + 2] = w.z; raw[4 * i + 3] = w.w;
      }
    }
    const int qa = q_fragments<KVQ_FMT_E4M3, DH>(raw, qb);
    const float ls0 = ls * __int_as_float((127 - __shfl_sync(kFull, qa, 8 * t)) << 23);
    const float ls1 = ls * __int_as_float((127 - __shfl_sync(kFull, qa, 8 * t + 4)) << 23);
    SoftmaxState st;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;
    float o[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

    // this warp's next page is unit warp + 16 done of the CTA's run
    while (warp + kDecWarps * done < pos + n) {
      if (!dead && !__all_sync(kFull, mbar_wait(&full[stage], parity))) {
        dead = true;  // the wait ran out: no more copies, the rest is skipped
        if (lane == 0) flag_status(p.status, KVQ_DEV_WAIT_TIMEOUT);
      }
      if (!dead) {
        const int pg = p0 + warp + kDecWarps * done - pos;
        const int tok0 = (pg < vis.sink ? pg : vis.first + pg - vis.sink) * kTok;
        const uint32_t kp = smem_u32(ring + stage * kSlot);
        dec_page<DH>(kp, kp + PG::kBytes, tok0, vis.lo, p.sinks, L, bad_s[stage] != 0, g, t, qb, o, st, ls0, ls1);
        __syncwarp();
        if (issued < mine) issue(stage);
      }
      ++done;
      if (++stage == p.S) {
        stage = 0;
        parity ^= 1u;
      }
    }
    pos += n;

    // ---- merge the warps' states of the piece
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      st.l[0] += __shfl_xor_sync(kFull, st.l[0], d);
      st.l[1] += __shfl_xor_sync(kFull, st.l[1], d);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = 2 * t + e;
      if (h < p.G) {
        if (g == 0) cml[warp * p.G + h] = make_float2(st.m[e], st.l[e]);
        if (st.m[e] != -INFINITY || st.l[e] != 0.f) {
          float* dst = co + (warp * p.G + h) * DH + g * (DH / 8);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            *reinterpret_cast<float2*>(dst + 2 * mt) = make_float2(o[mt][e], o[mt][2 + e]);
        }
      }
    }
    __syncthreads();
    const int64_t sigma = static_cast<int64_t>(b) * p.Hkv + gkv;
    const int64_t slot = c + sigma;
    uint16_t* orow = p.out + (static_cast<int64_t>(b) * p.Hq + gkv * p.G) * DH;
    for (int i = tid; i < p.G * DH; i += kDecThreads) {
      const int h = i / DH, d = i - h * DH;
      float M = -INFINITY, l = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, cml[w * p.G + h].x);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float2 ml = cml[w * p.G + h];
        if (ml.x != -INFINITY || ml.y != 0.f) {  // (-inf, 0): no visible token; its o is not there
          const float a = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - M);
          l += ml.y * a;
          acc += co[(w * p.G + h) * DH + d] * a;
        }
      }
      if (single) {
        const float r = acc * (l > 0.f ? sv / l : 0.f);
        orow[i] = static_cast<uint16_t>(f32x2_to_bf16x2(r, 0.f) & 0xFFFFu);
      } else {
        p.ws_o[slot * p.G * DH + i] = acc;
        if (d == 0) p.ws_ml[slot * p.G + h] = make_float2(M, l);
      }
    }
    __syncthreads();
    if (!single) {
      // Publish the piece: the barrier above orders every thread's stores
      // before thread 0's acquire-release arrival, and the arrival that
      // completes the count makes all pieces visible to this CTA.
      const int v_first = voff[b] + gkv * (pages + kPc) + kPc;
      const int c_lo = split.cta_of(v_first);
      const int np = split.cta_of(v_first + pages - 1) - c_lo + 1;
      if (tid == 0)
        merge_s = atom_add_acq_rel_gpu(p.ws_cnt + sigma, 1u) + 1 == static_cast<uint32_t>(np);
      __syncthreads();
      if (merge_s) {
        // thread (k, i): the pieces k, k + K, ... of output float4 i
        const int n4 = p.G * DH / 4;
        const int K = max(1, min(kDecThreads / n4, kDecWarps));  // [K][n4] fits co
        const float2* ml = p.ws_ml + (c_lo + sigma) * p.G;
        const float4* ob = reinterpret_cast<const float4*>(p.ws_o + (c_lo + sigma) * p.G * DH);
        float4* part = reinterpret_cast<float4*>(co);  // [K][n4]
        float2* pml = cml;                              // [K][G]
        for (int i = tid; i < K * n4; i += kDecThreads) {
          const int k = i / n4, e = i - k * n4, h = 4 * e / DH;
          float M = -INFINITY, l = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int j = k; j < np; j += 8 * K) {  // eight pieces at a time, their loads together
            float2 m8[8];
            float4 v8[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const int x = j + y * K;
              m8[y] = x < np ? __ldcg(ml + static_cast<int64_t>(x) * p.G + h) : make_float2(-INFINITY, 0.f);
              v8[y] = x < np ? __ldcg(ob + static_cast<int64_t>(x) * n4 + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float nm = M;
#pragma unroll
            for (int y = 0; y < 8; ++y) nm = fmaxf(nm, m8[y].x);
            const float a = (M == -INFINITY) ? 1.f : fast_exp2(M - nm);
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
          if (4 * e % DH == 0) pml[k * p.G + h] = make_float2(M, l);
        }
        __syncthreads();
        for (int e = tid; e < n4; e += kDecThreads) {
          const int h = 4 * e / DH;
          float M = -INFINITY, l = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; k < K; ++k) M = fmaxf(M, pml[k * p.G + h].x);
          for (int k = 0; k < K; ++k) {
            const float2 x = pml[k * p.G + h];
            const float4 v = part[k * n4 + e];
            const float w = x.x == -INFINITY ? 1.f : fast_exp2(x.x - M);
            l += x.y * w;
            acc.x += v.x * w;
            acc.y += v.y * w;
            acc.z += v.z * w;
            acc.w += v.w * w;
          }
          const float f = l > 0.f ? sv / l : 0.f;
          uint2 r;
          r.x = f32x2_to_bf16x2(acc.x * f, acc.y * f);
          r.y = f32x2_to_bf16x2(acc.z * f, acc.w * f);
          *reinterpret_cast<uint2*>(orow + 4 * e) = r;
        }
        if (tid == 0) p.ws_cnt[sigma] = 0u;
        __syncthreads();
      }
    }
    u += n;
  }
  // after a timeout: the copies still in flight land (or the wait runs out) before the CTA leaves
  for (; dead && done < issued; ++done) {
    mbar_wait(&full[done % p.S], static_cast<uint32_t>((done / p.S) & 1));
  }
}

}  // namespace fp4
}  // namespace kvq
