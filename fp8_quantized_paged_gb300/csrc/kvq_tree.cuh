// kvq_tree.cuh -- attention of trees of drafted tokens over the paged cache, on the
// 5th-generation tensor cores straight on the cache's codes.
//
//   O_j = softmax(q_j K^^T / sqrt(dh)) V^ over the tokens before the tree (in the window)
//   and node j's ancestors and itself,  K^ = float(code) sK
//
// A row is a (node, query head of the group) pair, a tile 128 of them (128 / G nodes) of a
// sequence and KV head: the M of both products.  A segment is a tile's keys, in blocks of
// kKeys.  The segments are laid end to end and cut into equal stretches, one a CTA, two CTAs
// an SM, so that a batch of any lengths keeps all SMs busy to the end; a segment that is cut
// leaves its rows' states in the workspace, which a second, dependent launch merges.  (A last
// arriver would read a piece of 64 KB for each of, say, 38 CTAs alone.)
//
//   warp 8 (producer)  copies a block's K pages, then its V pages, by TMA into a ring of 64 KB
//   warp 9 (issuer)    one lane: S = Q K^T (M 128, N kKeys); when the softmax has made P of it,
//     O += P V with P from tensor memory, V as it lies (token-major: an MN-major operand)
//   warps 0-7 (softmax)  thread = row (TMEM lane) and half of the block's keys: mask, running
//     maximum (raised lazily, exchanged between a row's two threads), P over the S columns
//     that it came from
// The products run on the codes as they are: no conversion, no registers between memory and the
// tensor cores.  For that Q and P are split into parts that 8 bits hold:
//   q  2^a q = q1 + q2, E4M3 both, 2^a taking the row's largest to [2^7, 2^8): bf16's 8 bits are
//     4 + 4, so exact within 2^8 of the largest; the parts add in one accumulator
//   P  weights times 2^7 as f16, then p1 + p2 + p3, E5M2 each (f16's upper byte, so a part is
//     subtracted exactly in f16): 2^-9 of the weight, or 2^-24 of the row's largest.  Three
//     E5M2 parts and not two E4M3 ones, whose range of 2^17 would drop a long context's small
//     weights beside one large one
// Over bf16 caches the operands are bf16: q itself, P as two parts.
//
// NaN and infinities: a key that is masked gets -inf by selection.  V's rows that no row sees
// count as zeros; those that only some see are searched for NaN and infinities, which are taken
// out of the shared tile (a weight of 0 would not clear them) and put back at the end into the
// rows that see them.
//
// Every wait is bounded; a timeout sets KVQ_DEV_WAIT_TIMEOUT, the roles stop, and the CTA waits
// (bounded) for its copies and matrix steps in flight.
#pragma once

#include <climits>

#include "../../include/kvq_step.h"
#include "kvq_decode.cuh"
#include "kvq_fp4.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace tree {

constexpr int kRows = 128;  // rows of a tile (MMA M)
constexpr int kSoftWarps = 8, kProdWarp = 8, kMmaWarp = 9;
constexpr int kTreeThreads = 320;
constexpr int kTreeCtas = 2;                          // CTAs of an SM
constexpr uint32_t kTmemCols = 256, kOutCol = 128;    // S and P at 0, O at 128
constexpr int kRing = 64 * 1024;
constexpr int kEntries = 1024;  // prefix sums of the plan: of every ceil(B / 1024)th sequence
constexpr int kSegCost = 2;     // a segment's start and end, in blocks
constexpr int kMinShare = 2;    // least cost of a CTA's stretch
constexpr float kBias = 7.f;    // log2 of the factor that the weights carry
constexpr int kMaskWords = KVQ_TREE_MAX_NODES / 32;

struct TreeParams {
  const uint16_t* q;
  const int32_t* cu_q;
  const int32_t* parents;  // NULL: a chain
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const uint8_t* vc;  // for the rows that NaN are put back into
  int max_blocks, B, Hq, Hkv, G;
  int64_t num_blocks, total_q;
  int window;
  const float* qs;  // KVQ_Q_FP8
  const float* ks;
  const float* vs;
  int q_per_head, per_head;
  float logit_scale;  // log2(e) / sqrt(dh)
  int4* ws_rec;       // [CTA] the segment that is cut and starts there: rows, last CTA, first query token, head
  float2* ws_ml;      // [2 CTA + whether the piece starts its segment][kRows]
  float* ws_o;        // [..][kRows][DH]
  uint16_t* out;
  uint32_t* status;
  int withhold;  // test builds: position of CTA 0's stream that is never copied; -1
};

struct TreeWs {
  size_t ml, o, total;
};
inline TreeWs tree_ws(int DH, int ctas) {
  const size_t rows = static_cast<size_t>(ctas) * 2 * kRows;
  TreeWs w;
  w.ml = round256(static_cast<size_t>(ctas) * sizeof(int4));
  w.o = w.ml + round256(rows * sizeof(float2));
  w.total = w.o + round256(rows * DH * sizeof(float));
  return w;
}

template <int FMT, int DH>
struct TreeCfg {
  static constexpr bool kBf = FMT == KVQ_FMT_BF16;
  static constexpr int kElem = kBf ? 2 : 1;
  static constexpr int kRow = DH * kElem;                 // bytes of a token's row
  static constexpr int kSpan = kRow > 128 ? 128 : kRow;   // of a tile's row; wider rows take two tiles side by side
  static constexpr int kKeys = kRow > 128 ? 64 : 128;     // keys of a block
  static constexpr int kPages = kKeys / kBS;
  static constexpr int kTile = kKeys * kRow;              // a block's K or V
  static constexpr int kSlots = kRing / kTile;            // 4 or 8
  static constexpr int kQTile = kRows * kRow;             // one part of Q
  static constexpr int kQParts = kBf ? 1 : 2;
  static constexpr int kChunks = kKeys / 64;              // of 32 keys, of a half block
  static constexpr int kPageBytes = kBS * kRow;
};

template <int FMT, int DH, bool TS>
struct TreeSmem {
  using C = TreeCfg<FMT, DH>;
  static constexpr int S = C::kSlots;
  static constexpr int q = 0;
  static constexpr int ring = q + C::kQParts * C::kQTile;
  static constexpr int tsc = ring + kRing;  // per-(token, head) scales, K's and V's, that land with a V
  static constexpr int bars = tsc + (TS ? S * C::kKeys * 4 : 0);
  static constexpr int kBars = 2 * S + 9;
  static constexpr int misc = bars + kBars * 8;  // tmem address, abort, NaN mark, -, bad[S], issued[S], warp sums
  static constexpr int mx = misc + (4 + 2 * S + kTreeThreads / 32) * 4;  // [2][2][kRows] maxima, [2][kRows] sums
  static constexpr int lo = mx + 6 * kRows * 4;                          // [kRows] first visible token
  static constexpr int anc = lo + kRows * 4;                             // [kMaskWords][kRows] ancestors
  static constexpr int plan = anc + kMaskWords * kRows * 4;
  static constexpr int total = plan + (kEntries + 1) * 4 + 1024;
  static_assert(total <= 113 * 1024, "two CTAs an SM");
};

// What the plan needs to know of a sequence.
struct Seq {
  int q0, n, L;
  int first;   // first key of its blocks, a page's first
  int blocks;  // 0: no rows to work on
  int tiles;
  int cost;    // of all its segments
  bool bad_q, bad_len;
};

template <int KEYS>
KVQ_DEVI Seq seq_of(const TreeParams& p, int b) {
  Seq s;
  s.q0 = __ldg(p.cu_q + b);
  const int q1 = __ldg(p.cu_q + b + 1);
  s.L = __ldg(p.seq_lens + b);
  s.bad_q = s.q0 < 0 || q1 < s.q0 || q1 > p.total_q || q1 - s.q0 > KVQ_TREE_MAX_NODES;
  s.n = s.bad_q ? 0 : q1 - s.q0;
  s.bad_len = s.n > 0 && (s.L < s.n || s.L > p.max_blocks * kBS);
  s.first = s.blocks = s.tiles = s.cost = 0;
  if (s.n > 0 && !s.bad_len) {
    const int tq = kRows / p.G;
    s.tiles = (s.n + tq - 1) / tq;
    const int lo = p.window > 0 ? s.L - s.n - p.window + 1 : 0;  // of the nodes without ancestors
    s.first = lo > 0 ? lo / kBS * kBS : 0;
    s.blocks = (s.L - s.first + KEYS - 1) / KEYS;
    s.cost = s.tiles * p.Hkv * (s.blocks + kSegCost);
  }
  return s;
}

// A CTA's part of a segment: blocks [i0, i1).
struct Piece {
  Seq s;
  int b, head, tile, i0, i1;
  int base;  // cost position of the segment
  KVQ_DEVI bool whole() const { return i0 == 0 && i1 == s.blocks; }
};

// The pieces of a stretch [v, end) of cost positions, in order.  A segment of n blocks takes
// kSegCost + n positions; block i is the CTA's that has position base + kSegCost + i.
template <int KEYS>
struct Pieces {
  const int32_t* plan;
  int per, entries;  // sequences of an entry
  int v, end;
  int b, at;  // the present sequence (-1: none), and its first position
  Seq s;
  KVQ_DEVI Pieces(const int32_t* plan_, int B, int v_, int end_) : plan(plan_), v(v_), end(end_), b(-1), at(0) {
    per = (B + kEntries - 1) / kEntries;
    entries = (B + per - 1) / per;
  }
  KVQ_DEVI bool next(const TreeParams& p, Piece& out) {
    while (v < end) {
      if (b < 0 || v >= at + s.cost) {
        const int e = find_seq(plan, entries, v);
        b = e * per;
        at = plan[e];
        s = seq_of<KEYS>(p, b);
        while (v >= at + s.cost) {
          at += s.cost;
          s = seq_of<KEYS>(p, ++b);
        }
      }
      const int len = s.blocks + kSegCost, seg = (v - at) / len;
      out.s = s;
      out.b = b;
      out.head = seg / s.tiles;  // tiles of a head side by side: they read the same pages
      out.tile = seg - out.head * s.tiles;
      out.base = at + seg * len;
      out.i0 = max(0, v - out.base - kSegCost);
      out.i1 = min(s.blocks, end - out.base - kSegCost);
      v = min(end, out.base + len);
      if (out.i1 > out.i0) return true;
    }
    return false;
  }
};

// Bits 0 .. 31 of the keys below `end` of 32 from key 0 on.
KVQ_DEVI uint32_t below(int end) { return end >= 32 ? 0xFFFFFFFFu : end <= 0 ? 0u : (1u << end) - 1u; }

// Bytes (halves) of a word that are NaN or infinite, as 0xFF (0xFFFF).
template <int FMT>
KVQ_DEVI uint32_t not_finite(uint32_t w) {
  if (FMT == KVQ_FMT_E4M3) return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  if (FMT == KVQ_FMT_E5M2) return __vcmpgeu4(w & 0x7F7F7F7Fu, 0x7C7C7C7Cu);
  return __vcmpgeu2(w & 0x7FFF7FFFu, 0x7F807F80u);
}

template <int FMT>
KVQ_DEVI float code_value(const uint8_t* row, int d) {
  if (FMT == KVQ_FMT_BF16) return bf16lo_to_f32(reinterpret_cast<const uint16_t*>(row)[d]);
  return f16lo_to_f32(fp8x2_to_f16x2<FMT>(row[d]));
}

KVQ_DEVI uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two f16 -> two E5M2 codes in the low half.
KVQ_DEVI uint32_t f16x2_to_e5m2x2(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  return c;
}
// And back: an E5M2 code is the upper byte of its f16.
KVQ_DEVI uint32_t e5m2x2_to_f16x2(uint32_t c) { return prmt(c, 0u, 0x1404u); }

// The three E5M2 parts of two weights (f16), each in the low half of c[k].
KVQ_DEVI void weight_parts(uint32_t h, uint32_t (&c)[3]) {
  c[0] = f16x2_to_e5m2x2(h);
  h = hsub2(h, e5m2x2_to_f16x2(c[0]));
  c[1] = f16x2_to_e5m2x2(h);
  h = hsub2(h, e5m2x2_to_f16x2(c[1]));
  c[2] = f16x2_to_e5m2x2(h);
}

// Byte `b` of row r in a tile of swizzled rows; rows past 128 bytes go on in a second tile.
template <int SPAN>
KVQ_DEVI uint32_t tile_at(int r, int b) {
  if (SPAN == 64) return static_cast<uint32_t>(r * 64 + (((b >> 4) ^ ((r >> 1) & 3)) << 4) + (b & 15));
  return static_cast<uint32_t>((b >> 7) * (kRows * 128) + r * 128 + ((((b & 127) >> 4) ^ (r & 7)) << 4) + (b & 15));
}

template <int FMT, int DH, bool TS>
__global__ void __launch_bounds__(kTreeThreads, kTreeCtas)
    tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv) {
  using C = TreeCfg<FMT, DH>;
  using SM = TreeSmem<FMT, DH, TS>;
  constexpr int S = C::kSlots, KEYS = C::kKeys;
  constexpr bool BF = C::kBf;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  // Position 2 g of the stream is the K of the CTA's block g, 2 g + 1 its V; slot: position % S.
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::bars);  // [S] a slot landed
  uint64_t* empty = full + S;     // [S] read by the matrix steps (commit)
  uint64_t* sfull = empty + S;    // S of a block written (commit, and the issuer's arrival)
  uint64_t* pfull = sfull + 1;    // P of a block written, O rescaled (8 warps)
  uint64_t* pdone = pfull + 1;    // O += P V of a block done (commit, and the issuer's arrival)
  uint64_t* qready = pdone + 1;   // Q of a piece written (8 warps)
  uint64_t* xch = qready + 1;     // [4] a row quarter's two warps have left words for each other
  uint64_t* fin = xch + 4;        // every matrix step done (commit)
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + SM::misc);
  volatile uint32_t* tmem_slot = misc;
  volatile uint32_t* abort_flag = misc + 1;
  volatile uint32_t* vnan = misc + 2;   // 1 + the last piece that met a NaN or infinity to put back
  volatile uint32_t* bad = misc + 4;    // [S] masked pages of block g at [g % S]: rewritten for block
                                        // g + S, whose K waits for the S of a block after g
  volatile int32_t* issued = reinterpret_cast<volatile int32_t*>(misc + 4 + S);  // [S] last position
  volatile int32_t* warp_sum = reinterpret_cast<volatile int32_t*>(misc + 4 + 2 * S);
  float* mx_s = reinterpret_cast<float*>(smem + SM::mx);
  float* l_s = mx_s + 4 * kRows;
  int32_t* lo_s = reinterpret_cast<int32_t*>(smem + SM::lo);
  uint32_t* anc = reinterpret_cast<uint32_t*>(smem + SM::anc);
  int32_t* plan = reinterpret_cast<int32_t*>(smem + SM::plan);

  // A parity wait for phase k of a barrier is sound while it has completed k or k + 1 phases.  The
  // issuer, the producer and the softmax take their barriers' phases in order, one a block (a piece:
  // qready).  The softmax also looks at a V slot's full barrier, for some blocks only: all earlier
  // phases of it are complete then, as the S of block g comes after the PV of block g - 1, and the
  // next one waits for this softmax.  (Not at a K slot's: the next K may land while a warp is late.)

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
      issued[i] = -1;
    }
    mbar_init(sfull, 2);
    mbar_init(pfull, kSoftWarps);
    mbar_init(pdone, 2);
    mbar_init(qready, kSoftWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&xch[i], 2);
    mbar_init(fin, 1);
    *abort_flag = 0u;
    *vnan = 0u;
    fence_mbar_init();
  }
  if (warp == kProdWarp && lane == 0) {
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  if (warp == kMmaWarp) tc::tmem_alloc(const_cast<uint32_t*>(tmem_slot), kTmemCols);
  pdl_wait();
  pdl_allow_next();

  // ---- the plan: prefix sums of the sequences' costs
  const int cta = blockIdx.x;
  int V;
  {
    const int per = (p.B + kEntries - 1) / kEntries, entries = (p.B + per - 1) / per;
    constexpr int kMine = (kEntries + kTreeThreads - 1) / kTreeThreads;
    const int each = (entries + kTreeThreads - 1) / kTreeThreads;
    int sum[kMine], mine = 0;
#pragma unroll
    for (int y = 0; y < kMine; ++y) {
      sum[y] = 0;
      const int e = tid * each + y;
      if (y < each && e < entries)
        for (int b = e * per; b < min(p.B, (e + 1) * per); ++b) sum[y] += seq_of<KEYS>(p, b).cost;
      mine += sum[y];
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(kFull, incl, off);
      if (lane >= off) incl += t;
    }
    if (lane == 31) warp_sum[warp] = incl;
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    int at = incl - mine;
    V = 0;
    for (int w = 0; w < kTreeThreads / 32; ++w) {
      at += w < warp ? warp_sum[w] : 0;
      V += warp_sum[w];
    }
#pragma unroll
    for (int y = 0; y < kMine; ++y) {
      const int e = tid * each + y;
      if (y < each && e < entries) plan[e] = at;
      at += sum[y];
    }
    if (tid == 0) p.ws_rec[cta] = make_int4(0, 0, 0, 0);
  }
  // sequences without work: errors, and zero rows
  for (int b = cta; b < p.B; b += gridDim.x) {
    const Seq s = seq_of<KEYS>(p, b);
    if (tid == 0 && s.bad_q) flag_status(p.status, KVQ_DEV_BAD_QLEN);
    if (!s.bad_len) continue;
    if (tid == 0) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
    uint4* row = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(s.q0) * p.Hq * DH);
    for (int64_t i = tid; i < static_cast<int64_t>(s.n) * p.Hq * DH / 8; i += kTreeThreads) row[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  // few blocks go to fewer CTAs
  const int Pe = max(1, min(static_cast<int>(gridDim.x), V / kMinShare));
  const CostSplit split(V, Pe);
  const int v0 = cta < Pe ? split(cta) : 0, v1 = cta < Pe ? (cta + 1 == Pe ? V : split(cta + 1)) : 0;

  auto fail = [&] {
    if (!*abort_flag) {
      *abort_flag = 1u;
      flag_status(p.status, KVQ_DEV_WAIT_TIMEOUT);
    }
  };
  auto wait_w = [&](uint64_t* bar, int phase) {  // warp-uniform
    return __all_sync(kFull, wait_or_abort(bar, static_cast<uint32_t>(phase & 1), abort_flag));
  };

  if (warp == kProdWarp) {
    // ------------------------------------------------------------ producer
    constexpr int kAhead = 32 / C::kPages;  // blocks of which the lanes hold the block ids
    Pieces<KEYS> it(plan, p.B, v0, v1);
    Piece pc;
    int g = 0;
    bool ok = true;
    while (ok && it.next(p, pc)) {
      const int pages = (pc.s.L + kBS - 1) / kBS, page0 = pc.s.first / kBS;
      const int32_t* table = p.block_tables + static_cast<int64_t>(pc.b) * p.max_blocks;
      // the cache row of page `page0 + kPages i + lane`, -1: masked out, -2: past the sequence
      auto row_of = [&](int i) {
        const int page = page0 + C::kPages * i + lane;
        if (page >= pages || i >= pc.i1 + kAhead) return -2;
        const int blk = __ldg(table + page);
        if (blk < 0 || blk >= p.num_blocks) return -1;
        return (blk * p.Hkv + pc.head) * kBS;
      };
      int rows = row_of(pc.i0), rows_next = row_of(pc.i0 + kAhead);
      for (int i = pc.i0; i < pc.i1 && ok; ++i, ++g) {
        const int j = (i - pc.i0) % kAhead;
        if (j == 0 && i > pc.i0) {
          rows = rows_next;
          rows_next = row_of(i + kAhead);
        }
        const int row = __shfl_sync(kFull, rows, C::kPages * j + lane % C::kPages);
        const bool good = lane < C::kPages && row >= 0;
        const uint32_t goods = __ballot_sync(kFull, good);
        if (lane < C::kPages && row == -1) flag_status(p.status, KVQ_DEV_BAD_BLOCK);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int pos = 2 * g + t, s = pos % S;
          ok = pos < S || wait_w(&empty[s], pos / S - 1);
          if (__any_sync(kFull, !ok || *abort_flag != 0u)) {
            if (lane == 0) fail();
            ok = false;
            break;
          }
#ifdef KVQ_TEST_HOOKS
          if (cta == 0 && pos == p.withhold) continue;  // its full barrier never completes
#endif
          if (lane == 0) {
            if (t == 0) bad[g % S] = ~goods & ((1u << C::kPages) - 1u);
            issued[s] = pos;
            if (goods == 0)
              mbar_arrive(&full[s]);  // nothing to copy
            else
              mbar_arrive_expect_tx(&full[s], __popc(goods) * (C::kPageBytes + (TS && t == 1 ? 2 * kBS * 4 : 0)));
          }
          __syncwarp();
          if (good) {
            uint8_t* dst = smem + SM::ring + s * C::kTile + lane * (kBS * C::kSpan);
            const CUtensorMap* map = t ? &tmv : &tmk;
            tma_load_2d(dst, map, 0, row, &full[s]);
            if (C::kRow > 128) tma_load_2d(dst + KEYS * 128, map, 64, row, &full[s]);
            if (TS && t == 1) {  // (K's own slot goes on to the next K before the softmax is done)
              uint8_t* sc = smem + SM::tsc + (g % (S / 2) * 2 * KEYS + lane * kBS) * 4;
              bulk_load(sc, p.ks + row, kBS * 4, &full[s]);
              bulk_load(sc + KEYS * 4, p.vs + row, kBS * 4, &full[s]);
            }
          }
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ matrix steps
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    if (tc::elect_one()) {
      const bool qf8 = !BF && p.qs != nullptr;
      const uint32_t id_qk = BF ? tc::idesc_bf16(kRows, KEYS)
                                : tc::idesc_f8(kRows, KEYS, qf8 ? tc::tc_type(FMT) : tc::kTcE4M3, tc::tc_type(FMT), false, false);
      const uint32_t id_pv = BF ? tc::idesc_bf16(kRows, DH) | (1u << 16)
                                : tc::idesc_f8(kRows, DH, tc::kTcE5M2, tc::tc_type(FMT), false, true);
      const int parts = BF || qf8 ? 1 : 2;
      auto wait = [&](uint64_t* bar, int phase) { return wait_or_abort(bar, static_cast<uint32_t>(phase & 1), abort_flag); };
      auto desc = [&](uint32_t a) { return C::kSpan == 64 ? tc::sw64_desc(a) : tc::sw128_desc(a); };
      Pieces<KEYS> it(plan, p.B, v0, v1);
      Piece pc;
      int g = 0, piece = 0;
      bool ok = true;
      while (ok && it.next(p, pc)) {
        if (!(ok = wait(qready, piece++))) break;
        for (int i = pc.i0; i < pc.i1; ++i, ++g) {
          const int ks = 2 * g % S, vs = (2 * g + 1) % S;
          if (!(ok = wait(&full[ks], 2 * g / S))) break;
          if (g > 0 && !(ok = wait(pdone, g - 1))) break;  // S's columns hold the P that this has read
          tc::tc_fence_after();
          const uint32_t a = sbase + SM::q, bk = sbase + SM::ring + ks * C::kTile;
#pragma unroll
          for (int k = 0; k < C::kRow / 32; ++k) {  // 32 bytes of a row a step
            const uint32_t oa = (k >> 2) * (kRows * 128) + (k & 3) * 32, ob = (k >> 2) * (KEYS * 128) + (k & 3) * 32;
            if (BF) {
              tc::mma_f16_ss(tm, desc(a + oa), desc(bk + ob), id_qk, k > 0 ? 1u : 0u);
            } else {
              tc::mma_f8_ss(tm, desc(a + oa), desc(bk + ob), id_qk, k > 0 ? 1u : 0u);
              if (parts > 1) tc::mma_f8_ss(tm, desc(a + C::kQTile + oa), desc(bk + ob), id_qk, 1u);
            }
          }
          mbar_arrive(sfull);  // hands on what the K slot's arrival showed (bad)
          tc::mma_commit(sfull);
          tc::mma_commit(&empty[ks]);
          if (!(ok = wait(&full[vs], (2 * g + 1) / S) && wait(pfull, g))) break;
          tc::tc_fence_after();
          const uint32_t bv = sbase + SM::ring + vs * C::kTile;
          const uint32_t more = i > pc.i0 ? 1u : 0u;
          if (BF) {
#pragma unroll
            for (int k = 0; k < KEYS / 16; ++k) {
              const uint64_t d = tc::sw128_desc(bv + k * 2048, KEYS * 128, 1024);
              const uint32_t at = tm + (k >> 1) * 32 + (k & 1) * 8;
              tc::mma_f16_ts(tm + kOutCol, at, d, id_pv, k > 0 ? 1u : more);
              tc::mma_f16_ts(tm + kOutCol, at + 16, d, id_pv, 1u);
            }
          } else {
#pragma unroll
            for (int k = 0; k < KEYS / 32; ++k) {
              const uint64_t d = desc(bv + k * 32 * C::kSpan);
#pragma unroll
              for (int y = 0; y < 3; ++y)
                tc::mma_f8_ts(tm + kOutCol, tm + k * 32 + y * 8, d, id_pv, k > 0 || y > 0 ? 1u : more);
            }
          }
          mbar_arrive(pdone);  // hands on what the softmax warps' arrivals showed (vnan)
          tc::mma_commit(pdone);
          tc::mma_commit(&empty[vs]);
        }
      }
      if (!ok) fail();
      tc::mma_commit(fin);
      if (!mbar_wait(fin, 0u)) fail();
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3, half = warp >> 2, r = quad * 32 + lane;
    const uint32_t tm = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    Pieces<KEYS> it(plan, p.B, v0, v1);
    Piece pc;
    int g = 0, piece = 0, xphase = 0;
    bool ok = true;
    // the two warps of a row quarter wait for each other
    auto exchange = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&xch[quad]);
      return wait_w(&xch[quad], xphase++);
    };
    while (ok && it.next(p, pc)) {
      const int TQ = kRows / p.G, j0 = pc.tile * TQ;
      const int rows = min(pc.s.n - j0, TQ) * p.G;
      const bool live = r < rows, some = quad * 32 < rows;
      const int node = j0 + (live ? r / p.G : 0), hq = pc.head * p.G + (live ? r % p.G : 0);
      const int64_t qrow = (static_cast<int64_t>(pc.s.q0) + node) * p.Hq + hq;
      const int P = pc.s.L - pc.s.n;  // tokens before the tree
      float lscale = (BF || TS ? 1.f : __ldg(p.ks + (p.per_head ? pc.head : 0))) * p.logit_scale;
      // ---- the query row: its half of the dims
      if (some) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + qrow * DH);
        if (BF) {
#pragma unroll 4
          for (int c = half * (DH / 16); c < (half + 1) * (DH / 16); ++c) {
            const uint4 w = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            tc::sts128(sbase + SM::q + tile_at<C::kSpan>(r, 16 * c), w.x, w.y, w.z, w.w);
          }
        } else {
          float up = 1.f, sq = 1.f;
          if (p.qs) {
            sq = __ldg(p.qs + (p.q_per_head ? hq : 0));
            lscale *= sq;
          } else {
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < DH / 8; ++c) {
              const uint4 w = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
              const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(bf16lo_to_f32(u[e])), fabsf(bf16hi_to_f32(u[e]))));
            }
            int a = 0;
            if (amax > 0.f) {
              a = 7 - (static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu) - 127);
              a = a > 126 ? 126 : (a < -126 ? -126 : a);
            }
            up = __int_as_float((a + 127) << 23);
            lscale *= __int_as_float((127 - a) << 23);
          }
#pragma unroll 2
          for (int c = half * (DH / 32); c < (half + 1) * (DH / 32); ++c) {  // 16 dims
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint4 w = live ? __ldg(src + 2 * c + y) : make_uint4(0u, 0u, 0u, 0u);
              const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x[4] = {bf16lo_to_f32(u[2 * e]), bf16hi_to_f32(u[2 * e]), bf16lo_to_f32(u[2 * e + 1]), bf16hi_to_f32(u[2 * e + 1])};
                if (p.qs) {
                  constexpr int F = FMT == KVQ_FMT_E5M2 ? KVQ_FMT_E5M2 : KVQ_FMT_E4M3;
#pragma unroll
                  for (int z = 0; z < 4; ++z) x[z] = __fdiv_rn(x[z], sq);
                  hi[2 * y + e] = f32x2_to_fp8x2<F>(x[0], x[1]) | (static_cast<uint32_t>(f32x2_to_fp8x2<F>(x[2], x[3])) << 16);
                  lo[2 * y + e] = 0u;
                } else {
#pragma unroll
                  for (int z = 0; z < 4; ++z) x[z] *= up;  // exact: a power of two, no overflow
                  const uint32_t c0 = f32x2_to_fp8x2<KVQ_FMT_E4M3>(x[0], x[1]), c1 = f32x2_to_fp8x2<KVQ_FMT_E4M3>(x[2], x[3]);
                  const uint32_t h0 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(c0));
                  const uint32_t h1 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(c1));
                  const uint32_t d0 = f32x2_to_fp8x2<KVQ_FMT_E4M3>(x[0] - f16lo_to_f32(h0), x[1] - f16hi_to_f32(h0));
                  const uint32_t d1 = f32x2_to_fp8x2<KVQ_FMT_E4M3>(x[2] - f16lo_to_f32(h1), x[3] - f16hi_to_f32(h1));
                  hi[2 * y + e] = c0 | (c1 << 16);
                  lo[2 * y + e] = d0 | (d1 << 16);
                }
              }
            }
            const uint32_t at = sbase + SM::q + tile_at<C::kSpan>(r, 16 * c);
            tc::sts128(at, hi[0], hi[1], hi[2], hi[3]);
            if (!p.qs) tc::sts128(at + C::kQTile, lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qready);
      lscale = fp4::bounded_scale(lscale);
      // ---- the row's ancestors, and the first token that it sees
      const int far = p.window > 0 ? p.window : INT_MAX;
      if (some && half == 0 && live && (p.window > 0 || pc.s.first + pc.i1 * KEYS > P)) {
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) anc[w * kRows + r] = 0u;
        int depth = -1;
        for (int at = node; at >= 0; ++depth) {
          if (depth + 1 < far) anc[(at >> 5) * kRows + r] |= 1u << (at & 31);
          int up = at - 1;
          if (p.parents) {
            up = __ldg(p.parents + pc.s.q0 + at);
            if (up >= at || up < -1) {
              flag_status(p.status, KVQ_DEV_BAD_TREE);
              up = -1;
            }
          }
          at = up;
        }
        lo_s[r] = p.window > 0 ? max(0, P + depth - p.window + 1) : 0;
      }
      if (some && !(ok = exchange())) break;
      const int lo = some && live && p.window > 0 ? lo_s[r] : 0;
      const int lo_most = p.window > 0 ? P + pc.s.n - p.window : 0;  // no row's first token lies past it
      // Keys of the 32 from key k on that the row sees, on good pages (bit y: page k / 16 + y is bad).
      auto seen32 = [&](int k, uint32_t bm) {
        uint32_t s = below(P - k) & ~below(lo - k);
        const int i = k - P;  // the first key's node
        if (i > -32 && i < KVQ_TREE_MAX_NODES) {
          const int w = i >> 5;
          const uint32_t a = w >= 0 ? anc[w * kRows + r] : 0u, z = w + 1 < kMaskWords ? anc[(w + 1) * kRows + r] : 0u;
          s |= __funnelshift_r(a, z, i & 31);
        }
        return s & ~((bm & 1u ? 0xFFFFu : 0u) | (bm & 2u ? 0xFFFF0000u : 0u));
      };
      float m = -INFINITY, l = 0.f, sig = 0.f;
      const float rise = kRescaleThreshold / lscale;
      for (int i = pc.i0; i < pc.i1; ++i, ++g) {
        const int k0 = pc.s.first + i * KEYS;
        const int vslot = (2 * g + 1) % S;
        if (!(ok = wait_w(sfull, g))) break;
        const uint32_t bm = bad[g % S];
        const bool edge = bm != 0u || k0 + KEYS > P || k0 < lo_most;
        if (edge || TS)
          if (!(ok = wait_w(&full[vslot], (2 * g + 1) / S))) break;
        if (edge) {
          // V's rows that no row sees become zeros; the others lose what is not finite
#pragma unroll
          for (int y = 0; y < C::kTile / (kSoftWarps * 32 * 16); ++y) {
            const int c = tid + y * kSoftWarps * 32;  // 16 bytes
            const int key = c / (C::kSpan / 16) % KEYS, t = k0 + key;
            uint4* at = reinterpret_cast<uint4*>(smem + SM::ring + vslot * C::kTile) + c;
            if (t >= pc.s.L || (bm >> (key / kBS) & 1u)) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else if (t >= P || t < lo_most) {
              uint4 w = *at;
              const uint4 f = make_uint4(not_finite<FMT>(w.x), not_finite<FMT>(w.y), not_finite<FMT>(w.z), not_finite<FMT>(w.w));
              if (f.x | f.y | f.z | f.w) {
                *at = make_uint4(w.x & ~f.x, w.y & ~f.y, w.z & ~f.z, w.w & ~f.w);
                *vnan = 1u + piece;
              }
            }
          }
          fence_proxy_async_smem();  // generic writes -> the tensor core's reads
        }
        tc::tc_fence_after();
        if (some) {
          const int kh = half * (KEYS / 2);
          const float* sk = reinterpret_cast<const float*>(smem + SM::tsc) + g % (S / 2) * 2 * KEYS + kh;
          const float* sv = sk + KEYS;
          // 32 logits (as raw products) of the half's chunk c, masked
          auto load = [&](int c, float (&x)[32]) {
            tc::tmem_ld32(tm + kh + 32 * c, x);
            if (TS) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 s4 = *reinterpret_cast<const float4*>(sk + 32 * c + e);
                x[e] *= s4.x;
                x[e + 1] *= s4.y;
                x[e + 2] *= s4.z;
                x[e + 3] *= s4.w;
              }
            }
            if (edge) {
              const uint32_t s = seen32(k0 + kh + 32 * c, bm >> ((kh + 32 * c) / kBS));
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = s >> e & 1u ? x[e] : -INFINITY;
              return s;
            }
            return 0xFFFFFFFFu;
          };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < C::kChunks; ++c) {
            float x[32];
            load(c, x);
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              a = tc::fmax3(a, x[e], x[e + 1]);
              b = tc::fmax3(b, x[e + 2], x[e + 3]);
            }
            mx = tc::fmax3(mx, a, b);
          }
          float* slot = mx_s + (g & 1) * 2 * kRows;
          slot[half * kRows + r] = mx;
          if (!(ok = exchange())) break;
          mx = fmaxf(mx, slot[(half ^ 1) * kRows + r]);
          const bool grow = mx > m + rise;
          float fs = 1.f;
          if (TS) {  // the largest value scale of the block's tokens, to a power of two
            float s = 0.f;
#pragma unroll
            for (int y = 0; y < KEYS / 32; ++y) {
              const int key = lane + 32 * y;
              const float v = sv[key - kh];
              if (k0 + key < pc.s.L && !(bm >> (key / kBS) & 1u)) s = fmaxf(s, v);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) s = fmaxf(s, __shfl_xor_sync(kFull, s, off));
            s = __uint_as_float(min((__float_as_uint(s) + 0x7FFFFFu) & 0x7F800000u, 0x7E800000u));
            if (s > sig) {
              fs = sig / s;
              sig = s;
            }
          }
          if (__any_sync(kFull, grow) || (TS && fs != 1.f)) {
            const float a = m == -INFINITY ? 0.f : fast_exp2((m - mx) * lscale);
            if (i > pc.i0) {  // (O's last writer is done: S came after it)
              const float f = (grow ? a : 1.f) * fs;
#pragma unroll 1
              for (int c = half * (DH / 2); c < (half + 1) * (DH / 2); c += 16) {
                uint32_t o[16];
                tc::tmem_ld16(tm + kOutCol + c, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tc::tmem_st16(tm + kOutCol + c, o);
              }
            }
            if (grow) {
              l *= a;
              m = mx;
            }
          }
          const float fm = m == -INFINITY ? 0.f : -m;
          const float inv_sig = TS && sig > 0.f ? 1.f / sig : 0.f;
          const tc::f32x2 fm2 = tc::f32x2_pack(fm, fm), ls2 = tc::f32x2_pack(lscale, lscale), b2 = tc::f32x2_pack(kBias, kBias);
          tc::f32x2 l2 = tc::f32x2_pack(0.f, 0.f);
#pragma unroll 1
          for (int c = 0; c < C::kChunks; ++c) {
            float x[32];
            const uint32_t s = load(c, x);
            // the maximum is subtracted before the scale: its own weight is 2^7 exactly, however large
            uint32_t w[3][8];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float y[4];
#pragma unroll
              for (int z = 0; z < 4; z += 2) {
                tc::f32x2_unpack(tc::f32x2_fma(tc::f32x2_add(tc::f32x2_pack(x[e + z], x[e + z + 1]), fm2), ls2, b2), y[z], y[z + 1]);
                y[z] = fast_exp2(y[z]);
                y[z + 1] = fast_exp2(y[z + 1]);
                l2 = tc::f32x2_add(l2, tc::f32x2_pack(y[z], y[z + 1]));
              }
              if (TS) {
                const float4 s4 = *reinterpret_cast<const float4*>(sv + 32 * c + e);
                y[0] = s >> e & 1u ? y[0] * (s4.x * inv_sig) : 0.f;
                y[1] = s >> (e + 1) & 1u ? y[1] * (s4.y * inv_sig) : 0.f;
                y[2] = s >> (e + 2) & 1u ? y[2] * (s4.z * inv_sig) : 0.f;
                y[3] = s >> (e + 3) & 1u ? y[3] * (s4.w * inv_sig) : 0.f;
              }
              if (BF) {  // two keys a column; hi of 16 keys a step, lo of them 16 columns on
                const uint32_t h0 = f32x2_to_bf16x2(y[0], y[1]), h1 = f32x2_to_bf16x2(y[2], y[3]);
                const uint32_t l0 = f32x2_to_bf16x2(y[0] - bf16lo_to_f32(h0), y[1] - bf16hi_to_f32(h0));
                const uint32_t l1 = f32x2_to_bf16x2(y[2] - bf16lo_to_f32(h1), y[3] - bf16hi_to_f32(h1));
                const uint32_t at = tm + kh + 32 * c + e / 2;
                asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(at), "r"(h0), "r"(h1) : "memory");
                asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(at + 16), "r"(l0), "r"(l1) : "memory");
              } else {
                uint32_t c0[3], c1[3];
                weight_parts(f32x2_to_f16x2(y[0], y[1]), c0);
                weight_parts(f32x2_to_f16x2(y[2], y[3]), c1);
#pragma unroll
                for (int k = 0; k < 3; ++k) w[k][e / 4] = prmt(c0[k], c1[k], 0x5410u);
              }
            }
            if (!BF)
#pragma unroll
              for (int k = 0; k < 3; ++k) tc::tmem_st8(tm + kh + 32 * c + 8 * k, w[k]);
          }
          float l0, l1;
          tc::f32x2_unpack(l2, l0, l1);
          l += l0 + l1;
          tc::tmem_st_wait();
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
      }
      if (!ok) break;
      // ---- the piece's end: rows of O, normalised
      if (!(ok = wait_w(pdone, g - 1))) break;
      tc::tc_fence_after();
      if (tid == 0 && !pc.whole() && pc.i0 == 0)
        p.ws_rec[cta] = make_int4(rows, split.cta_of(pc.base + kSegCost + pc.s.blocks - 1), pc.s.q0 + j0, pc.head);
      const bool put_back = *vnan == 1u + piece;
      ++piece;
      if (!some) continue;
      l_s[half * kRows + r] = l;
      if (!(ok = exchange())) break;
      l = l_s[r] + l_s[kRows + r];
      const float svs = TS ? sig : BF ? 1.f : __ldg(p.vs + (p.per_head ? pc.head : 0));
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const int64_t part = static_cast<int64_t>(2 * cta + (pc.i0 == 0)) * kRows + r;
      if (!pc.whole() && live && half == 0) p.ws_ml[part] = make_float2(fp4::merge_max(m, lscale), l);
#pragma unroll 1
      for (int c = half * (DH / 2); c < (half + 1) * (DH / 2); c += 32) {
        float o[32];
        tc::tmem_ld32(tm + kOutCol + c, o);
        if (put_back && live) {
          const int32_t* table = p.block_tables + static_cast<int64_t>(pc.b) * p.max_blocks;
          for (int k = pc.s.first + pc.i0 * KEYS; k < min(pc.s.L, pc.s.first + pc.i1 * KEYS); ++k) {
            if (k >= lo_most && k < P) {
              k = P - 1;
              continue;
            }
            if (!(seen32(k, 0u) & 1u)) continue;
            const int blk = __ldg(table + k / kBS);
            if (blk < 0 || blk >= p.num_blocks) continue;
            const uint8_t* row = p.vc + ((static_cast<int64_t>(blk) * p.Hkv + pc.head) * kBS + k % kBS) * C::kRow;
#pragma unroll 1
            for (int e = 0; e < 32; ++e) {
              const float v = code_value<FMT>(row, c + e);
              if (!(fabsf(v) <= 3.4028235e38f)) {
#pragma unroll
                for (int z = 0; z < 32; ++z) o[z] = z == e ? o[z] + v : o[z];
              }
            }
          }
        }
        if (live && pc.whole()) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + qrow * DH + c);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            dst[y] = make_uint4(fp4::output2(o[8 * y], o[8 * y + 1], inv, svs), fp4::output2(o[8 * y + 2], o[8 * y + 3], inv, svs),
                                fp4::output2(o[8 * y + 4], o[8 * y + 5], inv, svs), fp4::output2(o[8 * y + 6], o[8 * y + 7], inv, svs));
        } else if (live) {
          float4* dst = reinterpret_cast<float4*>(p.ws_o + part * DH + c);
#pragma unroll
          for (int y = 0; y < 8; ++y)
            dst[y] = make_float4(o[4 * y] * inv * svs, o[4 * y + 1] * inv * svs, o[4 * y + 2] * inv * svs, o[4 * y + 3] * inv * svs);
        }
      }
      if (put_back && !(ok = exchange())) break;  // (the next piece's ancestors are written over these)
      tc::tc_fence_before();
    }
    if (!ok) {
      tc::tmem_st_wait();
      fail();
    }
  }

  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  // After an abort: wait (bounded) for the copies in flight; the issuer waited for its steps.
  if (*abort_flag && tid == 0)
    for (int s = 0; s < S; ++s)
      if (issued[s] >= 0) mbar_wait(&full[s], static_cast<uint32_t>((issued[s] / S) & 1));
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- the rows of segments that were cut: a warp a row.  A piece's state is (maximum, sum,
// normalised row); the rows add with weights sum 2^maximum.
constexpr int kMergeThreads = 256;
constexpr int kMaxCtas = 512;

template <int DH>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ TreeParams p, int ctas) {
  __shared__ int off[kMaxCtas + 1];
  __shared__ int warp_sum[kMergeThreads / 32];
  pdl_wait();
  pdl_allow_next();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = kMaxCtas / kMergeThreads;
  int rows[kPer], mine = 0;
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    const int c = kPer * tid + y;
    rows[y] = c < ctas ? __ldcg(p.ws_rec + c).x : 0;
    mine += rows[y];
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int at = incl - mine, total = 0;
  for (int w = 0; w < kMergeThreads / 32; ++w) {
    at += w < warp ? warp_sum[w] : 0;
    total += warp_sum[w];
  }
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    off[kPer * tid + y] = at;
    at += rows[y];
  }
  if (tid == 0) off[kMaxCtas] = total;
  __syncthreads();
  constexpr int E = DH / 32;  // values of a lane
  for (int x = blockIdx.x * (kMergeThreads / 32) + warp; x < total; x += gridDim.x * (kMergeThreads / 32)) {
    const int c0 = find_seq(off, kMaxCtas, x), r = x - off[c0];
    const int4 rec = __ldcg(p.ws_rec + c0);
    const int n = rec.y - c0 + 1;  // pieces
    auto part = [&](int y) { return static_cast<int64_t>(2 * (c0 + y) + (y == 0)) * kRows + r; };
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int y0 = 0; y0 < n; y0 += 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (y0 + lane < n) ml = __ldcg(p.ws_ml + part(y0 + lane));
      float nm = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) nm = fmaxf(nm, __shfl_xor_sync(kFull, nm, o));
      nm = fmaxf(nm, M);
      const float a = M == -INFINITY ? 0.f : fast_exp2((M - nm) * fp4::kMergeUnit);
      // (a piece without a maximum has a sum of 0, or a NaN, which stays)
      const float w = ml.y * (ml.x == -INFINITY ? 1.f : fast_exp2((ml.x - nm) * fp4::kMergeUnit));
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      L = L * a + sum;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= a;
      M = nm;
      const int k = min(32, n - y0);
#pragma unroll 8
      for (int y = 0; y < k; ++y) {
        const float wy = __shfl_sync(kFull, w, y);
        const float* o = p.ws_o + part(y0 + y) * DH + E * lane;
        float v[E];
        if (E == 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(o));
          v[0] = f.x;
          v[1] = f.y;
          v[E - 2] = f.z;
          v[E - 1] = f.w;
        } else {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(o));
          v[0] = f.x;
          v[1] = f.y;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wy, v[e], acc[e]);
      }
    }
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
    uint16_t* dst = p.out + ((static_cast<int64_t>(rec.z) + r / p.G) * p.Hq + rec.w * p.G + r % p.G) * DH + E * lane;
    uint32_t* d32 = reinterpret_cast<uint32_t*>(dst);
#pragma unroll
    for (int e = 0; e < E; e += 2) d32[e / 2] = f32x2_to_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  }
}

}  // namespace tree
}  // namespace kvq
