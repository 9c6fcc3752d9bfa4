// kvq_tree.cuh -- attention of trees of drafted tokens over the paged cache, on the
// 5th-generation tensor cores straight on the cache's codes.
//
//   O_j = softmax(q_j K^^T / sqrt(dh)) V^ over the tokens before the tree (in the window)
//   and node j's ancestors and itself,  K^ = float(code) sK
//
// A row is a (node, query head of the group) pair, a tile 128 of them (128 / G nodes) of a
// sequence and KV head: the M of both products.  A segment is a tile's keys, in blocks of 64.
// The segments are laid end to end and cut into equal stretches, one a CTA, a CTA an SM, so that a
// batch of any lengths keeps all SMs busy to the end; a segment that is cut leaves its rows'
// states in the workspace, which a second, dependent launch merges.  (A last arriver would read a
// piece of 64 KB of each of, say, 19 CTAs alone.)
//
//   warps 12, 13 (producers of K, of V)  copy a block's pages by TMA into rings of 64 KB; the first
//     also works out the CTA's pieces, one ahead, and describes them to the others in shared memory
//   warp 14 (issuer)  one lane: S = Q K^T (M 128, N 64), up to six blocks ahead
//   warp 15 (issuer)  one lane: O += P V (M 128, N dh), V as it lies (token-major: an MN-major operand)
//   warps 0-3, 4-7, 8-11 (softmax of every third block)  thread = row (TMEM lane): mask, running
//     maximum, P over the S columns that it came from.  The maximum is handed from block to block, a
//     warp of one group to the next one's (m_s): it is wanted before the weights, and changes rarely
// Tensor memory: six buffers of S and P (64 columns each) and O (128).  A block's way through S,
// softmax and PV takes about 5000 cycles, of which the matrix steps' and barriers' latencies are most;
// six blocks in flight hide it.  Q lies in shared memory, twice: the next piece's is written while this
// one's is in use.
//
// What bounds it: instructions.  64 keys of 128 rows take 0.63 us of a CTA, some 1250 cycles, of which the
// tensor cores are busy 770, and each scheduler issues some 900 instructions: 64 weights of a row and
// their parts are about 9 each (a softmax thread), the roles beside it the rest.  A segment's start and end
// cost ten blocks.  32 trees of 16 nodes (64 rows) over 2049 tokens of 8 KV heads, 134 MB: 58 to 60 us, of
// which the merge 6; one of 64 nodes over 32768: 56 to 61; 128 of 24 over 17 to 16384 with a window of 4096:
// 166 to 169; with scales per (token, head) the first takes 82.  What was tried and is slower, in us for the
// first and the second of these, then at 57 and 56 (weights of 9 bits): two CTAs an SM
// with two buffers each 77 and 78; two groups, four buffers and Q in tensor memory (steps of 32 cycles
// and not 48) 58 and 58; the maximum handed on behind S's loads, so that the groups go in step, 61 and
// 60; two producers each of K and V and two issuers of S, the logits read twice so that 608 threads
// find registers, 62 and 63; the next piece's Q written between blocks 66 and 63 (code that is rare
// but lies in the loop).
// The products run on the codes as they are: no conversion, no registers between memory and the
// tensor cores.  For that Q and P are split into parts that 8 bits hold:
//   q  2^a q = q1 + q2, E4M3 both, 2^a taking the row's largest to [2^7, 2^8): bf16's 8 bits are
//     4 + 4, so exact within 2^8 of the largest; the parts add in one accumulator
//   P  weights times 2^7 as f16, then p1 + p2 + p3, E5M2 each: f16's upper byte is an E5M2 number,
//     so a part is the rounded byte of what the parts before left, subtracted exactly in f16.  What the
//     first two leave of 11 bits is a multiple of 1 and at most 8 in units of the last one, 3 bits: the
//     parts add up to the f16, but for what lies below E5M2's least step: 2^-11 of the weight and 2^-24 of
//     the row's largest.  (Parts cut and not rounded, the last one excepted, have 9 bits and take 5
//     instructions a pair of weights, not 7: 1 to 3 % of the time.)  Three
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
constexpr int kGroups = 3, kGroupWarps = 4, kSoftWarps = kGroups * kGroupWarps, kProdWarp = kSoftWarps, kMmaWarp = kProdWarp + 2;
constexpr int kTreeThreads = 32 * (kMmaWarp + 2);
constexpr int kKeys = 64;                             // keys of a block
constexpr int kBufs = 6;                              // of S and P
constexpr uint32_t kTmemCols = 512, kOutCol = 384;    // the buffers at 0, O at 384
constexpr int kRing = 64 * 1024;  // of K, and of V
constexpr int kEntries = 1024;  // prefix sums of the plan: of every ceil(B / 1024)th sequence
constexpr int kKept = 256;      // sequences up to which their lengths are kept beside the prefix sums
// A segment's start and end, in blocks.  Swept on 128 mixed sequences, in us, with weights of 9 bits: 4 195,
// 8 168, 10 161, 12 159, 16 168; 16 bf16 ones: 4 41, 8 and 10 37, 12 39.
constexpr int kSegCost = 10;
constexpr int kMinShare = 4;    // least cost of a CTA's stretch
constexpr float kBias = 7.f;    // log2 of the factor that the weights carry
constexpr int kPieces = 32;     // descriptions of pieces
constexpr int kBadRing = 32;
constexpr int kMaskWords = KVQ_TREE_MAX_NODES / 32;
constexpr int kScaleBufs = 3;   // pieces whose logits' scales are in shared memory
constexpr int kNanMarks = 2;    // pieces whose mark of a NaN or infinity is

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
  int late;      // test builds: softmax warp that sleeps before it reads what other quarters' warps write; -1
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
  static constexpr int kPages = kKeys / kBS;
  static constexpr int kTile = kKeys * kRow;              // a block's K or V
  static constexpr int kSlots = kRing / kTile;            // 4, 8 or 16
  static constexpr int kQParts = kBf ? 1 : 2;
  static constexpr int kPageBytes = kBS * kRow;
  static constexpr int kQTile = kRows * kRow;             // one part of Q
};

template <int FMT, int DH, bool TS>
struct TreeSmem {
  using C = TreeCfg<FMT, DH>;
  static constexpr int S = C::kSlots;
  static constexpr int q = 0;  // [2] Q, by piece
  static constexpr int ring = q + 2 * C::kQParts * C::kQTile;
  static constexpr int tsc = ring + 2 * kRing;  // per-(token, head) scales, K's and V's, that land with a V
  static constexpr int bars = tsc + (TS ? 2 * S * kKeys * 4 : 0);
  static constexpr int kBars = 4 * S + 3 * kBufs + 2 + 1 + kGroups * 4 + 4 + 2 + 1 + kPieces;
  // tmem address, abort, bad sequences, NaN marks, bad[kBadRing], issued[2], warp sums
  static constexpr int misc = bars + kBars * 8;
  // [kRows] running maximum; (TS) [kRows] largest value scale that the row has seen, [2][kRows] that at a piece's end
  static constexpr int m = misc + (5 + kNanMarks + kBadRing + kTreeThreads / 32) * 4;
  static constexpr int l = (m + (TS ? 4 : 1) * kRows * 4 + 7) / 8 * 8;  // [2][kGroups][kRows] sums and their maxima, by piece
  static constexpr int ls = l + 2 * kGroups * kRows * 8;                 // [kScaleBufs][kRows] logits' scales, by piece
  static constexpr int anc = ls + kScaleBufs * kRows * 4;               // [kGroups][kMaskWords][kRows] ancestors
  static constexpr int pieces = (anc + kGroups * kMaskWords * kRows * 4 + 15) / 16 * 16;  // [kPieces] of 12 words
  static constexpr int plan = pieces + kPieces * 48;
  static constexpr int total = plan + (kEntries + 1) * 4 + 1024;
  static_assert(total <= 227 * 1024, "shared memory");
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

KVQ_DEVI Seq seq_from(const TreeParams& p, int q0, int q1, int L) {
  Seq s;
  s.q0 = q0;
  s.L = L;
  s.bad_q = s.q0 < 0 || q1 < s.q0 || q1 > p.total_q || q1 - s.q0 > KVQ_TREE_MAX_NODES;
  s.n = s.bad_q ? 0 : q1 - s.q0;
  s.bad_len = s.n > 0 && (s.L < s.n || s.L > p.max_blocks * kBS);
  s.first = s.blocks = s.tiles = s.cost = 0;
  if (s.n > 0 && !s.bad_len) {
    const int tq = kRows / p.G;
    s.tiles = (s.n + tq - 1) / tq;
    const int lo = p.window > 0 ? s.L - s.n - p.window + 1 : 0;  // of the nodes without ancestors
    s.first = lo > 0 ? lo / kBS * kBS : 0;
    s.blocks = (s.L - s.first + kKeys - 1) / kKeys;
    s.cost = s.tiles * p.Hkv * (s.blocks + kSegCost);
  }
  return s;
}

KVQ_DEVI Seq seq_of(const TreeParams& p, int b) {
  return seq_from(p, __ldg(p.cu_q + b), __ldg(p.cu_q + b + 1), __ldg(p.seq_lens + b));
}
// From the plan, whose words kKept + 3 b .. are q0, q1 and L of sequence b where there are few.
KVQ_DEVI Seq seq_of(const TreeParams& p, const int32_t* plan, int b) {
  const int32_t* w = plan + kKept + 3 * b;
  return p.B <= kKept ? seq_from(p, w[0], w[1], w[2]) : seq_of(p, b);
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
        s = seq_of(p, plan, b);
        while (v >= at + s.cost) {
          at += s.cost;
          s = seq_of(p, plan, ++b);
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
// 1 / s of a power of two from 2^-126 to 2^126.
KVQ_DEVI float inverse_power(float s) { return __uint_as_float(0x7F000000u - __float_as_uint(s)); }

// The E5M2 parts of two weights (f16, not negative, at most 2^15), each the upper byte of a half of c[k].
// Half a step added rounds a magnitude; no carry leaves a half.  A NaN becomes a zero: it is in the row's sum.
KVQ_DEVI void weight_parts(uint32_t h, uint32_t (&c)[3]) {
  c[0] = h + 0x00800080u;
  const uint32_t r1 = hsub2(h, c[0] & 0xFF00FF00u);
  c[1] = r1 + 0x00800080u;
  c[2] = hsub2(r1, c[1] & 0xFF00FF00u) + 0x00800080u;
}

// Byte `b` of row r in a tile of swizzled rows; rows past 128 bytes go on in a second tile.
template <int SPAN>
KVQ_DEVI uint32_t tile_at(int r, int b) {
  if (SPAN == 64) return static_cast<uint32_t>(r * 64 + (((b >> 4) ^ ((r >> 1) & 3)) << 4) + (b & 15));
  return static_cast<uint32_t>((b >> 7) * (kRows * 128) + r * 128 + ((((b & 127) >> 4) ^ (r & 7)) << 4) + (b & 15));
}

template <int FMT, int DH, bool TS>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv) {
  using C = TreeCfg<FMT, DH>;
  using SM = TreeSmem<FMT, DH, TS>;
  constexpr int S = C::kSlots;
  constexpr bool BF = C::kBf;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  // The K (V) of the CTA's block g takes slot g % S of its ring; full and empty: [0, S) K's, [S, 2 S) V's.
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::bars);  // [2 S] a slot landed
  uint64_t* empty = full + 2 * S;  // [2 S] read by the matrix steps (commit)
  uint64_t* sfull = empty + 2 * S;      // [kBufs] S of a block written (commit, and the issuer's arrival)
  uint64_t* pfull = sfull + kBufs;      // [kBufs] P of a block written, O rescaled (4 warps)
  uint64_t* pdone = pfull + kBufs;      // [kBufs] O += P V of a block done (commit)
  uint64_t* qready = pdone + kBufs;     // [2] Q of a piece written (12 warps)
  uint64_t* ofree = qready + 2;         // O of a piece read (12 warps)
  uint64_t* token = ofree + 1;          // [kGroups][4] a block's maximum is in m_s: by quarter of the rows
  uint64_t* lfull = token + kGroups * 4;  // [4] a piece's sums of a quarter are in l_s (3 warps)
  uint64_t* fin = lfull + 4;            // [2] every S, every PV done (commit)
  uint64_t* odone = fin + 2;            // a piece's last O += P V done (commit, and the issuer's arrival)
  uint64_t* known = odone + 1;          // [kPieces] a piece's description is there
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + SM::misc);
  volatile uint32_t* tmem_slot = misc;
  volatile uint32_t* abort_flag = misc + 1;
  volatile uint32_t* any_bad = misc + 2;  // a sequence has an error
  volatile uint32_t* vnan = misc + 3;   // [kNanMarks] 1 + the last piece that met a NaN or infinity to put back
  volatile uint32_t* bad = vnan + kNanMarks;  // [kBadRing] masked pages of block g: rewritten for block g + 32,
                                        // whose K waits for the S of block g + 32 - S, and that for the PV of
                                        // block g + 26 - S
  volatile int32_t* issued = reinterpret_cast<volatile int32_t*>(bad + kBadRing);  // [2] blocks copied
  volatile int32_t* warp_sum = issued + 2;
  // Piece n's description in [n % kPieces].  It is rewritten for piece n + 32, when all blocks of piece
  // n + 30 but its last have their K's slots: the PV of block g - S - 7 of the last block g is done then, and
  // every role past the piece that has it, which at a block a piece is n + 30 - S - 7 > n.
  int4* pieces_s = reinterpret_cast<int4*>(smem + SM::pieces);
  float* m_s = reinterpret_cast<float*>(smem + SM::m);
  float* sig_s = m_s + kRows;
  float* sige_s = sig_s + kRows;
  float2* l_s = reinterpret_cast<float2*>(smem + SM::l);
  float* ls_s = reinterpret_cast<float*>(smem + SM::ls);
  int32_t* plan = reinterpret_cast<int32_t*>(smem + SM::plan);

  // A parity wait for phase k of a barrier is sound while it has completed k or k + 1 phases.  All roles
  // take their barriers' phases in order, except that the softmax looks at V's full barriers (edge blocks)
  // and at pdone now and then.  All earlier phases are complete then: the S of block g comes after the PV
  // of block g - 6, PVs go in order, and a V's slot has had its last V once the PV of block g - S is done.
  // And the next phases come after a block that this warp has not begun with.  (Not at a K slot's full
  // barrier: the next K may land while a warp is late.  Nor at pdone for a piece's end: a group that had
  // no block of it may be several phases behind.)
  //
  // What a softmax warp writes for others between pieces: at the start of piece n the logits' scales of piece
  // n + 1 (rows of any quarter), in its edge blocks the mark of a NaN, at its end its group's sums.  A piece's
  // end holds up only a quarter's three warps (lfull), so a warp of another quarter may still be at the start
  // of piece n, its scales not read, when one is in piece n + 1; not in n + 2, whose way leads through the PV
  // of piece n + 1 (odone) and so through every warp's end of piece n (ofree).  So scales are kept for three
  // pieces, marks for two (sums too, though a warp that writes them is past that PV).

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 2 * S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    issued[0] = issued[1] = 0;
    *any_bad = 0u;
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sfull[i], 2);
      mbar_init(&pfull[i], kGroupWarps);
      mbar_init(&pdone[i], 1);
    }
    mbar_init(&qready[0], kSoftWarps);
    mbar_init(&qready[1], kSoftWarps);
    mbar_init(ofree, kSoftWarps);
    for (int i = 0; i < kGroups * 4; ++i) mbar_init(&token[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&lfull[i], kGroups);
    for (int i = 0; i < kPieces; ++i) mbar_init(&known[i], 1);
    mbar_init(odone, 2);
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    *abort_flag = 0u;
    for (int i = 0; i < kNanMarks; ++i) vnan[i] = 0u;
    fence_mbar_init();
  }
  if (warp == kProdWarp && lane == 0) {
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  __syncthreads();  // (any_bad)
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
        for (int b = e * per; b < min(p.B, (e + 1) * per); ++b) {
          const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), L = __ldg(p.seq_lens + b);
          const Seq s = seq_from(p, q0, q1, L);
          if (p.B <= kKept) {
            plan[kKept + 3 * b] = q0;
            plan[kKept + 3 * b + 1] = q1;
            plan[kKept + 3 * b + 2] = L;
          }
          sum[y] += s.cost;
          if (s.bad_q || s.bad_len) *any_bad = 1u;
        }
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
  __syncthreads();
  // sequences with errors: reported, and zero rows
  for (int b = cta; *any_bad && b < p.B; b += gridDim.x) {
    const Seq s = seq_of(p, b);
    if (tid == 0 && s.bad_q) flag_status(p.status, KVQ_DEV_BAD_QLEN);
    if (!s.bad_len) continue;
    if (tid == 0) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
    uint4* row = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(s.q0) * p.Hq * DH);
    for (int64_t i = tid; i < static_cast<int64_t>(s.n) * p.Hq * DH / 8; i += kTreeThreads) row[i] = make_uint4(0u, 0u, 0u, 0u);
  }
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
  auto wait = [&](uint64_t* bar, int phase) { return wait_or_abort(bar, static_cast<uint32_t>(phase & 1), abort_flag); };
  auto wait_w = [&](uint64_t* bar, int phase) { return __all_sync(kFull, wait(bar, phase)); };  // warp-uniform

  // Piece n, as the producer of K describes it; without blocks: the end.
  auto piece_at = [&](int n, Piece& pc) {
    if (!wait(&known[n % kPieces], n / kPieces)) return false;
    const int4 a = pieces_s[3 * (n % kPieces)], b = pieces_s[3 * (n % kPieces) + 1], c = pieces_s[3 * (n % kPieces) + 2];
    pc.i0 = a.x;
    pc.i1 = a.y;
    pc.head = a.z;
    pc.tile = a.w;
    pc.s.q0 = b.x;
    pc.s.n = b.y;
    pc.s.L = b.z;
    pc.s.first = b.w;
    pc.s.blocks = c.x;
    pc.b = c.y;
    pc.base = c.z;
    return true;
  };

  if (warp >= kProdWarp) {
  if (warp < kMmaWarp) {
    // ------------------------------------------------------------ producers: K, V
    const int t = __shfl_sync(kFull, warp, 0) - kProdWarp;
    constexpr int kAhead = 32 / C::kPages;  // blocks of which the lanes hold the block ids
    const CUtensorMap* map = t ? &tmv : &tmk;
    const uint64_t policy = l2_evict_first_policy();  // (what is read once does not push out the queries, states and code)
    Pieces it(plan, p.B, v0, v1);
    Piece pc;
    pc.i0 = pc.i1 = 0;
    int described = 0, begun = 0, i = 0, rows = 0, rows_next = 0;
    bool ok = true, fetch = t == 0;
    for (int g = 0;; ++g) {
      if (fetch) {  // (K's) a piece is described once the one before has begun: the softmax wants its queries
        Piece nx = {};
        const bool more = it.next(p, nx);
        if (lane == 0) {
          int4* d = pieces_s + 3 * (described % kPieces);
          d[0] = more ? make_int4(nx.i0, nx.i1, nx.head, nx.tile) : make_int4(0, 0, 0, 0);
          d[1] = make_int4(nx.s.q0, nx.s.n, nx.s.L, nx.s.first);
          d[2] = make_int4(nx.s.blocks, nx.b, nx.base, 0);
          mbar_arrive(&known[described % kPieces]);
        }
        __syncwarp();
        ++described;
        fetch = false;
      }
      const bool begins = i == pc.i1;
      if (begins) {
        if (!(ok = __all_sync(kFull, piece_at(begun++, pc))) || pc.i1 == 0) break;
        i = pc.i0;
      }
      const int pages = (pc.s.L + kBS - 1) / kBS, page0 = pc.s.first / kBS;
      const int32_t* table = p.block_tables + static_cast<int64_t>(pc.b) * p.max_blocks;
      // the cache row of page `page0 + kPages i + lane`, -1: masked out, -2: past the sequence
      auto row_of = [&](int i) {
        const int page = page0 + C::kPages * i + lane;
        if (page >= pages || i >= pc.i1 + kAhead) return -2;
        const int blk = __ldg(table + page);
        if (blk < 0 || blk >= p.num_blocks) {
          if (page < page0 + C::kPages * pc.i1) flag_status(p.status, KVQ_DEV_BAD_BLOCK);
          return -1;
        }
        return (blk * p.Hkv + pc.head) * kBS;
      };
      const int j = (i - pc.i0) % kAhead, s = g % S;
      if (begins) rows_next = row_of(i);
      if (j == 0) {
        rows = rows_next;
        rows_next = row_of(i + kAhead);
      }
      {
        const uint32_t goods = (__ballot_sync(kFull, rows >= 0) >> (C::kPages * j)) & ((1u << C::kPages) - 1u);
        if (g >= S && !(ok = wait_w(&empty[t * S + s], g / S - 1))) break;
        bool copies = true;
#ifdef KVQ_TEST_HOOKS
        copies = cta != 0 || 2 * g + t != p.withhold;  // (its full barrier never completes)
#endif
        uint8_t* dst = smem + SM::ring + t * kRing + s * C::kTile;
        int row[C::kPages];
#pragma unroll
        for (int y = 0; y < C::kPages; ++y) row[y] = __shfl_sync(kFull, rows, C::kPages * j + y);
        if (copies && tc::elect_one()) {
          if (t == 0) bad[g % kBadRing] = ~goods & ((1u << C::kPages) - 1u);
          issued[t] = g + 1;
          if (goods == 0)
            mbar_arrive(&full[t * S + s]);  // nothing to copy
          else
            mbar_arrive_expect_tx(&full[t * S + s], __popc(goods) * (C::kPageBytes + (TS && t == 1 ? 2 * kBS * 4 : 0)));
#pragma unroll
          for (int y = 0; y < C::kPages; ++y) {
            if (row[y] < 0) continue;
            tma_load_2d_hint(dst + y * (kBS * C::kSpan), map, 0, row[y], &full[t * S + s], policy);
            if (C::kRow > 128) tma_load_2d_hint(dst + y * (kBS * C::kSpan) + kKeys * 128, map, 64, row[y], &full[t * S + s], policy);
            if (TS && t == 1) {  // (K's own slot goes on to the next K before the softmax is done)
              uint8_t* sc = smem + SM::tsc + (s * 2 * kKeys + y * kBS) * 4;
              bulk_load(sc, p.ks + row[y], kBS * 4, &full[t * S + s]);
              bulk_load(sc + kKeys * 4, p.vs + row[y], kBS * 4, &full[t * S + s]);
            }
          }
        }
        __syncwarp();
      }
      ++i;
      fetch = t == 0 && begins;
    }
    if (!ok && lane == 0) fail();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ S = Q K^T
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    if (tc::elect_one()) {
      const bool qf8 = !BF && p.qs != nullptr;
      const uint32_t id_qk = BF ? tc::idesc_bf16(kRows, kKeys)
                                : tc::idesc_f8(kRows, kKeys, qf8 ? tc::tc_type(FMT) : tc::kTcE4M3, tc::tc_type(FMT), false, false);
      const int parts = BF || qf8 ? 1 : 2;
      auto desc = [&](uint32_t a) { return C::kSpan == 64 ? tc::sw64_desc(a) : tc::sw128_desc(a); };
      Piece pc;
      int g = 0, piece = 0;
      bool ok = true;
      while (ok && (ok = piece_at(piece, pc)) && pc.i1 > 0) {
        if (!(ok = wait(&qready[piece & 1], piece >> 1))) break;
        const uint32_t a = sbase + SM::q + (piece & 1) * C::kQParts * C::kQTile;
        ++piece;
        for (int i = pc.i0; i < pc.i1; ++i, ++g) {
          const int s = g % S, buf = g % kBufs;
          // (over the P that the PV of block g - 6 has read)
          if (!(ok = wait(&full[s], g / S) && (g < kBufs || wait(&pdone[buf], g / kBufs - 1)))) break;
          tc::tc_fence_after();
          const uint32_t bk = sbase + SM::ring + s * C::kTile, d = tm + buf * kKeys;
#pragma unroll
          for (int k = 0; k < C::kRow / 32; ++k) {  // 32 bytes of a row a step
            const uint32_t oa = (k >> 2) * (kRows * 128) + (k & 3) * 32, ob = (k >> 2) * (kKeys * 128) + (k & 3) * 32;
            if (BF) {
              tc::mma_f16_ss(d, desc(a + oa), desc(bk + ob), id_qk, k > 0 ? 1u : 0u);
            } else {
              tc::mma_f8_ss(d, desc(a + oa), desc(bk + ob), id_qk, k > 0 ? 1u : 0u);
              if (parts > 1) tc::mma_f8_ss(d, desc(a + C::kQTile + oa), desc(bk + ob), id_qk, 1u);
            }
          }
          mbar_arrive(&sfull[buf]);  // hands on what the K slot's arrival showed (bad)
          tc::mma_commit(&sfull[buf]);
          tc::mma_commit(&empty[s]);
        }
      }
      if (!ok) fail();
      tc::mma_commit(&fin[0]);
      if (!mbar_wait(&fin[0], 0u)) fail();
    }
  } else if (warp == kMmaWarp + 1) {
    // ------------------------------------------------------------ O += P V
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    if (tc::elect_one()) {
      const uint32_t id_pv = BF ? tc::idesc_bf16(kRows, DH) | (1u << 16)
                                : tc::idesc_f8(kRows, DH, tc::kTcE5M2, tc::tc_type(FMT), false, true);
      auto desc = [&](uint32_t a) { return C::kSpan == 64 ? tc::sw64_desc(a) : tc::sw128_desc(a); };
      Piece pc;
      int g = 0, piece = 0;
      bool ok = true;
      while (ok && (ok = piece_at(piece, pc)) && pc.i1 > 0) {
        if (piece > 0 && !(ok = wait(ofree, piece - 1))) break;
        ++piece;
        for (int i = pc.i0; i < pc.i1; ++i, ++g) {
          const int s = g % S, buf = g % kBufs;
          if (!(ok = wait(&full[S + s], g / S) && wait(&pfull[buf], g / kBufs))) break;
          tc::tc_fence_after();
          const uint32_t bv = sbase + SM::ring + kRing + s * C::kTile, tp = tm + buf * kKeys;
          const uint32_t more = i > pc.i0 ? 1u : 0u;
          if (BF) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k) {
              const uint64_t d = tc::sw128_desc(bv + k * 2048, kKeys * 128, 1024);
              const uint32_t at = tp + (k >> 1) * 32 + (k & 1) * 8;
              tc::mma_f16_ts(tm + kOutCol, at, d, id_pv, k > 0 ? 1u : more);
              tc::mma_f16_ts(tm + kOutCol, at + 16, d, id_pv, 1u);
            }
          } else {
#pragma unroll
            for (int k = 0; k < kKeys / 32; ++k) {
              const uint64_t d = desc(bv + k * 32 * C::kSpan);
#pragma unroll
              for (int y = 0; y < 3; ++y)
                tc::mma_f8_ts(tm + kOutCol, tp + k * 32 + y * 8, d, id_pv, k > 0 || y > 0 ? 1u : more);
            }
          }
          tc::mma_commit(&pdone[buf]);
          tc::mma_commit(&empty[S + s]);
        }
        mbar_arrive(odone);  // hands on what the softmax warps' arrivals showed (vnan)
        tc::mma_commit(odone);
      }
      if (!ok) fail();
      tc::mma_commit(&fin[1]);
      if (!mbar_wait(&fin[1], 0u)) fail();
    }
  }
  } else {
    // ------------------------------------------------------------ softmax
    const int group = warp / kGroupWarps, quad = warp % kGroupWarps, r = quad * 32 + lane;
    const uint32_t tm = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    uint32_t* anc = reinterpret_cast<uint32_t*>(smem + SM::anc) + group * kMaskWords * kRows;
    // The query rows of piece number n into shared memory, scaled, and their logits' scales, while the
    // piece before is worked on: a warp two rows (dh 64: four) at a time, three such steps in flight.
    // (Code that runs once a piece is fetched as slowly as data, so it is kept short: a thread a row and
    // its 128 dims unrolled took 9000 to 19000 cycles, in loops 7000 with the small L1 missed twice.)
    auto write_q = [&](const Piece& pc, int n) {
      constexpr int kLanes = DH / 8, kStep = kSoftWarps * (32 / kLanes);
      const int TQ = kRows / p.G, j0 = pc.tile * TQ, rows = min(pc.s.n - j0, TQ) * p.G, ql = lane % kLanes;
      const float lscale0 = (BF || TS ? 1.f : __ldg(p.ks + (p.per_head ? pc.head : 0))) * p.logit_scale;
      const uint32_t to = sbase + SM::q + (n & 1) * C::kQParts * C::kQTile;
#pragma unroll 1
      for (int r0 = warp * (32 / kLanes) + lane / kLanes; __any_sync(kFull, r0 < rows); r0 += 3 * kStep) {
        uint4 w[3];
        float qs[3];
#pragma unroll
        for (int y = 0; y < 3; ++y) {
          const int at = r0 + y * kStep < rows ? r0 + y * kStep : 0, hq = pc.head * p.G + at % p.G;
          w[y] = __ldg(reinterpret_cast<const uint4*>(p.q + ((static_cast<int64_t>(pc.s.q0) + j0 + at / p.G) * p.Hq + hq) * DH) + ql);
          qs[y] = p.qs ? __ldg(p.qs + (p.q_per_head ? hq : 0)) : 1.f;
        }
#pragma unroll
        for (int y = 0; y < 3; ++y) {
          const int at = r0 + y * kStep;
          float lscale = lscale0;
          uint32_t u[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
          if (BF) {  // (infinities as NaN: logits of -inf alone would be a row that sees nothing)
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] |= __vcmpeq2(u[e] & 0x7FFF7FFFu, 0x7F807F80u) & 0x00400040u;
            if (at < rows) tc::sts128(to + tile_at<C::kSpan>(at, 16 * ql), u[0], u[1], u[2], u[3]);
          } else {
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[2 * e] = bf16lo_to_f32(u[e]);
              x[2 * e + 1] = bf16hi_to_f32(u[e]);
            }
            uint32_t hi[2], lo[2] = {0u, 0u};
            if (p.qs) {
              constexpr int F = FMT == KVQ_FMT_E5M2 ? KVQ_FMT_E5M2 : KVQ_FMT_E4M3;
              lscale *= qs[y];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(x[e], qs[y]);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                hi[e] = f32x2_to_fp8x2<F>(x[4 * e], x[4 * e + 1]) | (static_cast<uint32_t>(f32x2_to_fp8x2<F>(x[4 * e + 2], x[4 * e + 3])) << 16);
            } else {
              uint32_t top = __vmaxu2(__vmaxu2(u[0] & 0x7FFF7FFFu, u[1] & 0x7FFF7FFFu), __vmaxu2(u[2] & 0x7FFF7FFFu, u[3] & 0x7FFF7FFFu));
#pragma unroll
              for (int off = 1; off < kLanes; off <<= 1) top = __vmaxu2(top, __shfl_xor_sync(kFull, top, off));
              const int e = static_cast<int>(max(top & 0xFFFFu, top >> 16) >> 7);  // its exponent, 0 for subnormals
              const int a = top == 0u ? 0 : min(126, 134 - max(e, 8));  // (-121 .. 126)
              // exact: a power of two, no overflow; in a row with a NaN or an infinity 0, which leaves NaN for these
              const float by = e == 255 ? 0.f : __int_as_float((a + 127) << 23);
              lscale *= __int_as_float((127 - a) << 23);
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] *= by;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t c0 = f32x2_to_fp8x2<KVQ_FMT_E4M3>(x[4 * e], x[4 * e + 1]);
                const uint32_t c1 = f32x2_to_fp8x2<KVQ_FMT_E4M3>(x[4 * e + 2], x[4 * e + 3]);
                const uint32_t h0 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(c0));
                const uint32_t h1 = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(c1));
                hi[e] = c0 | (c1 << 16);
                lo[e] = f32x2_to_fp8x2<KVQ_FMT_E4M3>(x[4 * e] - f16lo_to_f32(h0), x[4 * e + 1] - f16hi_to_f32(h0)) |
                        (static_cast<uint32_t>(f32x2_to_fp8x2<KVQ_FMT_E4M3>(x[4 * e + 2] - f16lo_to_f32(h1), x[4 * e + 3] - f16hi_to_f32(h1))) << 16);
              }
            }
            if (at < rows) {
              uint8_t* dst = smem + SM::q + (n & 1) * C::kQParts * C::kQTile + tile_at<C::kSpan>(at, 8 * ql);
              *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
              if (!p.qs) *reinterpret_cast<uint2*>(dst + C::kQTile) = make_uint2(lo[0], lo[1]);
            }
          }
          if (at < rows && ql == 0) ls_s[(n % kScaleBufs) * kRows + at] = fp4::bounded_scale(lscale);
        }
      }
      fence_proxy_async_smem();  // generic writes -> the tensor core's reads
      __syncwarp();
      if (lane == 0) mbar_arrive(&qready[n & 1]);
    };
    auto late = [&] {
#ifdef KVQ_TEST_HOOKS
      if (warp == p.late) __nanosleep(20000);
#endif
    };
    int g = 0, piece = 0, written = 0;
    bool ok = true;
    for (;;) {
      Piece pc;
      while (written <= piece + 1) {  // (the S of the piece that this Q's place was of are done)
        if (!(ok = __all_sync(kFull, piece_at(written, pc))) || pc.i1 == 0) break;
        write_q(pc, written++);
      }
      if (!ok || !(ok = __all_sync(kFull, piece_at(piece, pc))) || pc.i1 == 0) break;
      // the logits' scales are other warps'
      if (!(ok = wait_w(&qready[piece & 1], piece >> 1))) break;
      const int TQ = kRows / p.G, j0 = pc.tile * TQ;
      const int rows = min(pc.s.n - j0, TQ) * p.G;
      const bool live = r < rows, some = quad * 32 < rows;
      const int node = j0 + (live ? r / p.G : 0);
      const int P = pc.s.L - pc.s.n;  // tokens before the tree
      // ---- the row's ancestors, and the first token that it sees
      int lo = 0;
      if (live && (p.window > 0 || pc.s.first + pc.i1 * kKeys > P)) {
        const int far = p.window > 0 ? p.window : INT_MAX;
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
        if (p.window > 0) lo = max(0, P + depth - p.window + 1);
      }
      __syncwarp();
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
      late();
      const float lscale = live ? ls_s[(piece % kScaleBufs) * kRows + r] : 1.f;
      const int last = g + pc.i1 - pc.i0 - 1;  // the piece's last block
      for (int i = pc.i0; i < pc.i1; ++i, ++g) {
        if (g % kGroups != group) continue;
        const int k0 = pc.s.first + i * kKeys, buf = g % kBufs;
        const int vslot = g % S;
        // what the block before left
        if (g > 0 && !(ok = wait_w(&token[(group + kGroups - 1) % kGroups * 4 + quad], (g - 1) / kGroups))) break;
        const float before = i > pc.i0 ? m_s[r] : -INFINITY;
        if (!(ok = wait_w(&sfull[buf], g / kBufs))) break;
        const uint32_t bm = bad[g % kBadRing];
        const bool edge = bm != 0u || k0 + kKeys > P || k0 < lo_most;
        if (edge || TS) {
          // (with rings of fewer blocks than buffers, the slot's last V may still be to come: it is there
          // once the PV of block g - S is done)
          if (S < kBufs && g >= S && !(ok = wait_w(&pdone[(g - S) % kBufs], (g - S) / kBufs))) break;
          if (!(ok = wait_w(&full[S + vslot], g / S))) break;
        }
        if (__builtin_expect(edge, 0)) {
          // V's rows that no row sees become zeros; the others lose what is not finite
#pragma unroll
          for (int y = 0; y < C::kTile / (kGroupWarps * 32 * 16); ++y) {
            const int c = r + y * kGroupWarps * 32;  // 16 bytes
            const int key = c / (C::kSpan / 16) % kKeys, t = k0 + key;
            uint4* at = reinterpret_cast<uint4*>(smem + SM::ring + kRing + vslot * C::kTile) + c;
            if (t >= pc.s.L || (bm >> (key / kBS) & 1u)) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else if (t >= P || t < lo_most) {
              uint4 w = *at;
              const uint4 f = make_uint4(not_finite<FMT>(w.x), not_finite<FMT>(w.y), not_finite<FMT>(w.z), not_finite<FMT>(w.w));
              if (f.x | f.y | f.z | f.w) {
                *at = make_uint4(w.x & ~f.x, w.y & ~f.y, w.z & ~f.z, w.w & ~f.w);
                vnan[piece % kNanMarks] = 1u + piece;
              }
            }
          }
          fence_proxy_async_smem();  // generic writes -> the tensor core's reads
        }
        tc::tc_fence_after();
        if (some) {
          const uint32_t ts = tm + buf * kKeys;
          const float* sk = reinterpret_cast<const float*>(smem + SM::tsc) + vslot * 2 * kKeys;
          const float* sv = sk + kKeys;
          // 64 logits (as raw products), masked
          float x[kKeys];
          tc::tmem_ld64(ts, x);
          if (TS) {
#pragma unroll
            for (int e = 0; e < kKeys; e += 4) {
              const float4 s4 = *reinterpret_cast<const float4*>(sk + e);
              x[e] *= s4.x;
              x[e + 1] *= s4.y;
              x[e + 2] *= s4.z;
              x[e + 3] *= s4.w;
            }
          }
          uint32_t seen[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
          if (__builtin_expect(edge, 0)) {
#pragma unroll
            for (int c = 0; c < 2; ++c) seen[c] = seen32(k0 + 32 * c, bm >> (2 * c));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[32 * c + e] = seen[c] >> e & 1u ? x[32 * c + e] : -INFINITY;
            }
          }
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kKeys; e += 8)
#pragma unroll
            for (int y = 0; y < 4; ++y) mx4[y] = tc::fmax3(mx4[y], x[e + 2 * y], x[e + 2 * y + 1]);
          const float mx = tc::fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]);
          const bool grow = live && mx > before + kRescaleThreshold / lscale;
          if (m != before) {  // (another group raised it)
            l *= m == -INFINITY ? 0.f : fast_exp2((m - before) * lscale);
            m = before;
          }
          float fs = 1.f;
          if (TS) {  // the largest value scale of the block's tokens that the row sees, to a power of two
            uint32_t top = 0u;  // (its bits)
            if (__builtin_expect(edge, 0)) {
#pragma unroll 1
              for (int e = 0; e < kKeys; e += 4) {
                const uint4 s4 = *reinterpret_cast<const uint4*>(sv + e);
                const uint32_t of[4] = {s4.x, s4.y, s4.z, s4.w}, see = (e < 32 ? seen[0] : seen[1]) >> (e & 31);
#pragma unroll
                for (int z = 0; z < 4; ++z) top = max(top, see >> z & 1u ? of[z] & 0x7FFFFFFFu : 0u);
              }
            } else {  // every row sees them all
              const uint32_t* bits = reinterpret_cast<const uint32_t*>(sv);
              top = __reduce_max_sync(kFull, max(bits[lane] & 0x7FFFFFFFu, bits[lane + 32] & 0x7FFFFFFFu));
            }
            if (top > 0x7F800000u) l = __uint_as_float(top);  // (a NaN: no part of a weight is one, the sum is)
            const float s = __uint_as_float(min((top + 0x7FFFFFu) & 0x7F800000u, 0x7E800000u));
            sig = i > pc.i0 ? sig_s[r] : 0.f;
            if (s > sig) {
              fs = sig * inverse_power(s);
              sig = s;
            }
          }
          if (__builtin_expect(__any_sync(kFull, grow || (TS && fs != 1.f)), 0)) {
            const float a = m == -INFINITY ? 0.f : fast_exp2((m - mx) * lscale);
            if (i > pc.i0) {  // O's last writer: the PV of the block before
              if (!(ok = wait_w(&pdone[(g - 1) % kBufs], (g - 1) / kBufs))) break;
              tc::tc_fence_after();
              const float f = (grow ? a : 1.f) * fs;
#pragma unroll 1
              for (int c = 0; c < DH; c += 16) {
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
          m_s[r] = m;
          if (TS) sig_s[r] = sig;
          __syncwarp();
          if (lane == 0) mbar_arrive(&token[group * 4 + quad]);
          const float fm = m == -INFINITY ? 0.f : -m;
          const float inv_sig = TS && sig > 0.f ? inverse_power(sig) : 0.f;
          const tc::f32x2 fm2 = tc::f32x2_pack(fm, fm), ls2 = tc::f32x2_pack(lscale, lscale), b2 = tc::f32x2_pack(kBias, kBias);
          tc::f32x2 l2[2] = {tc::f32x2_pack(0.f, 0.f), tc::f32x2_pack(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // the maximum is subtracted before the scale: its own weight is 2^7 exactly, however large
            uint32_t w[4][8];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const int k = 32 * c + e;
              float y[4];
#pragma unroll
              for (int z = 0; z < 4; z += 2) {
                tc::f32x2_unpack(tc::f32x2_fma(tc::f32x2_add(tc::f32x2_pack(x[k + z], x[k + z + 1]), fm2), ls2, b2), y[z], y[z + 1]);
                y[z] = fast_exp2(y[z]);
                y[z + 1] = fast_exp2(y[z + 1]);
                l2[z >> 1] = tc::f32x2_add(l2[z >> 1], tc::f32x2_pack(y[z], y[z + 1]));
              }
              if (TS) {
                const float4 s4 = *reinterpret_cast<const float4*>(sv + k);
                y[0] = seen[c] >> e & 1u ? y[0] * (s4.x * inv_sig) : 0.f;
                y[1] = seen[c] >> (e + 1) & 1u ? y[1] * (s4.y * inv_sig) : 0.f;
                y[2] = seen[c] >> (e + 2) & 1u ? y[2] * (s4.z * inv_sig) : 0.f;
                y[3] = seen[c] >> (e + 3) & 1u ? y[3] * (s4.w * inv_sig) : 0.f;
              }
              if (BF) {  // two keys a column: w[0], w[1] the hi parts of 16 keys each, w[2], w[3] the lo parts
                const uint32_t h0 = f32x2_to_bf16x2(y[0], y[1]), h1 = f32x2_to_bf16x2(y[2], y[3]);
                w[e >> 4][(e & 15) / 2] = h0;
                w[e >> 4][(e & 15) / 2 + 1] = h1;
                w[2 + (e >> 4)][(e & 15) / 2] = f32x2_to_bf16x2(y[0] - bf16lo_to_f32(h0), y[1] - bf16hi_to_f32(h0));
                w[2 + (e >> 4)][(e & 15) / 2 + 1] = f32x2_to_bf16x2(y[2] - bf16lo_to_f32(h1), y[3] - bf16hi_to_f32(h1));
              } else {  // four keys a column, a part of all 32 in w[0], w[1], w[2] each
                uint32_t c0[3], c1[3];
                weight_parts(f32x2_to_f16x2(y[0], y[1]), c0);
                weight_parts(f32x2_to_f16x2(y[2], y[3]), c1);
#pragma unroll
                for (int z = 0; z < 3; ++z) w[z][e / 4] = prmt(c0[z], c1[z], 0x7531u);
              }
            }
#pragma unroll
            for (int z = 0; z < (BF ? 4 : 3); ++z) tc::tmem_st8(ts + 32 * c + 8 * z, w[z]);
          }
          float l0, l1;
          tc::f32x2_unpack(tc::f32x2_add(l2[0], l2[1]), l0, l1);
          l += l0 + l1;
          tc::tmem_st_wait();
        } else {  // (tokens count blocks)
          if (lane == 0) mbar_arrive(&token[group * 4 + quad]);
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[buf]);
      }
      if (!ok) break;
      // ---- the piece's end: rows of O, normalised, every third run of 16 dims by a group
      if (!(ok = wait_w(odone, piece))) break;
      tc::tc_fence_after();
      if (tid == 0 && !pc.whole() && pc.i0 == 0)
        p.ws_rec[cta] = make_int4(rows, split.cta_of(pc.base + kSegCost + pc.s.blocks - 1), pc.s.q0 + j0, pc.head);
      late();
      const bool put_back = vnan[piece % kNanMarks] == 1u + piece;
      // a group's sum is relative to the maximum of its last block, O to that of the last one
      float2* sums = l_s + (piece & 1) * kGroups * kRows;
      sums[group * kRows + r] = make_float2(l, m);
      const int owner = last % kGroups;
      if (TS && group == owner) sige_s[(piece & 1) * kRows + r] = sig;
      __syncwarp();
      if (lane == 0) mbar_arrive(&lfull[quad]);
      if (!(ok = wait_w(&lfull[quad], piece))) break;
      ++piece;
      m = sums[owner * kRows + r].y;
      l = 0.f;
#pragma unroll
      for (int y = 0; y < kGroups; ++y) {
        const float2 s = sums[y * kRows + r];
        l += s.x * (s.y == -INFINITY || s.y == m ? 1.f : fast_exp2((s.y - m) * lscale));
      }
      const float svs = TS ? sige_s[((piece - 1) & 1) * kRows + r] : BF ? 1.f : __ldg(p.vs + (p.per_head ? pc.head : 0));
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const int64_t part = static_cast<int64_t>(2 * cta + (pc.i0 == 0)) * kRows + r;
      const int64_t qrow = (static_cast<int64_t>(pc.s.q0) + node) * p.Hq + pc.head * p.G + r % p.G;
      if (!pc.whole() && live && group == owner) p.ws_ml[part] = make_float2(fp4::merge_max(m, lscale), l);
      if (some) {
#pragma unroll 1
      for (int c = 16 * group; c < DH; c += 16 * kGroups) {
        float o[16];
        uint32_t bits[16];
        tc::tmem_ld16(tm + kOutCol + c, bits);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(bits[e]);
        if (put_back && live) {
          const int32_t* table = p.block_tables + static_cast<int64_t>(pc.b) * p.max_blocks;
          for (int k = pc.s.first + pc.i0 * kKeys; k < min(pc.s.L, pc.s.first + pc.i1 * kKeys); ++k) {
            if (k >= lo_most && k < P) {
              k = P - 1;
              continue;
            }
            if (!(seen32(k, 0u) & 1u)) continue;
            const int blk = __ldg(table + k / kBS);
            if (blk < 0 || blk >= p.num_blocks) continue;
            const uint8_t* row = p.vc + ((static_cast<int64_t>(blk) * p.Hkv + pc.head) * kBS + k % kBS) * C::kRow;
#pragma unroll 1
            for (int e = 0; e < 16; ++e) {
              const float v = code_value<FMT>(row, c + e);
              if (!(fabsf(v) <= 3.4028235e38f)) {
#pragma unroll
                for (int z = 0; z < 16; ++z) o[z] = z == e ? o[z] + v : o[z];
              }
            }
          }
        }
        if (live && pc.whole()) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + qrow * DH + c);
#pragma unroll
          for (int y = 0; y < 2; ++y)
            dst[y] = make_uint4(fp4::output2(o[8 * y], o[8 * y + 1], inv, svs), fp4::output2(o[8 * y + 2], o[8 * y + 3], inv, svs),
                                fp4::output2(o[8 * y + 4], o[8 * y + 5], inv, svs), fp4::output2(o[8 * y + 6], o[8 * y + 7], inv, svs));
        } else if (live) {
          float4* dst = reinterpret_cast<float4*>(p.ws_o + part * DH + c);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            dst[y] = make_float4(o[4 * y] * inv * svs, o[4 * y + 1] * inv * svs, o[4 * y + 2] * inv * svs, o[4 * y + 3] * inv * svs);
        }
      }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree);
    }
    if (!ok) {
      tc::tmem_st_wait();
      fail();
    }
  }

  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  // After an abort: wait (bounded) for the copies in flight; the issuers waited for their steps.
  if (*abort_flag && tid < 2)
    for (int g = max(0, issued[tid] - S); g < issued[tid]; ++g)
      mbar_wait(&full[tid * S + g % S], static_cast<uint32_t>((g / S) & 1));
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- the rows of segments that were cut: half a warp a row, or a warp.  A piece's state is (maximum, sum,
// normalised row); the rows add with weights sum 2^maximum.  Chains of loads (record, states, rows) that
// nothing but many rows at once hides.
constexpr int kMergeThreads = 256, kMergeCtas = 5;  // CTAs of an SM
constexpr int kMaxCtas = 512;

template <int DH>
__global__ void __launch_bounds__(kMergeThreads, kMergeCtas) merge_kernel(const __grid_constant__ TreeParams p, int ctas) {
  __shared__ int off[kMaxCtas + 1];
  __shared__ int4 recs[kMaxCtas];
  __shared__ int warp_sum[kMergeThreads / 32];
  pdl_wait();
  pdl_allow_next();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = kMaxCtas / kMergeThreads;
  int rows[kPer], mine = 0;
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    const int c = kPer * tid + y;
    const int4 rec = c < ctas ? __ldcg(p.ws_rec + c) : make_int4(0, 0, 0, 0);
    recs[c] = rec;
    rows[y] = rec.x;
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
  __syncthreads();
  constexpr int E = DH / 16;  // values of a lane, in runs of 4
  const int l16 = lane & 15;
  const uint32_t half = 0xFFFFu << (lane & 16);
  // Few rows take a warp each, a half of it every second piece.
  const bool wide = 2 * total <= static_cast<int>(gridDim.x) * (kMergeThreads / 16);
  const int step = wide ? 2 : 1, sub = wide ? lane >> 4 : 0;
  const int each = kMergeThreads / 16 / step;  // rows of a CTA
  for (int x = blockIdx.x * each + (tid >> 4) / step; x < total; x += gridDim.x * each) {
    const int c0 = find_seq(off, kMaxCtas, x), r = x - off[c0];
    const int4 rec = recs[c0];
    const int n = rec.y - c0 + 1;  // pieces
    auto part = [&](int y) { return static_cast<int64_t>(2 * (c0 + y) + (y == 0)) * kRows + r; };
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int y0 = 0; y0 < n; y0 += 16) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (y0 + l16 < n) ml = __ldcg(p.ws_ml + part(y0 + l16));
      float nm = ml.x;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) nm = fmaxf(nm, __shfl_xor_sync(half, nm, o));
      nm = fmaxf(nm, M);
      const float a = M == -INFINITY ? 0.f : fast_exp2((M - nm) * fp4::kMergeUnit);
      // (a piece without a maximum has a sum of 0, or a NaN, which stays)
      const float w = ml.y * (ml.x == -INFINITY ? 1.f : fast_exp2((ml.x - nm) * fp4::kMergeUnit));
      float sum = w;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(half, sum, o);
      L = L * a + sum;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= a;
      M = nm;
      const int k = min(16, n - y0);
#pragma unroll 4
      for (int y = sub; y < k; y += step) {
        const float wy = __shfl_sync(half, w, (lane & 16) + y);
        const float4* o = reinterpret_cast<const float4*>(p.ws_o + part(y0 + y) * DH) + l16;
#pragma unroll
        for (int e = 0; e < E / 4; ++e) {
          const float4 f = __ldcg(o + 16 * e);
          acc[4 * e] = fmaf(wy, f.x, acc[4 * e]);
          acc[4 * e + 1] = fmaf(wy, f.y, acc[4 * e + 1]);
          acc[4 * e + 2] = fmaf(wy, f.z, acc[4 * e + 2]);
          acc[4 * e + 3] = fmaf(wy, f.w, acc[4 * e + 3]);
        }
      }
    }
    if (wide) {
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += __shfl_xor_sync(kFull, acc[e], 16);
      if (sub) continue;
    }
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
    uint2* dst = reinterpret_cast<uint2*>(p.out + ((static_cast<int64_t>(rec.z) + r / p.G) * p.Hq + rec.w * p.G + r % p.G) * DH) + l16;
#pragma unroll
    for (int e = 0; e < E / 4; ++e)
      dst[16 * e] = make_uint2(f32x2_to_bf16x2(acc[4 * e] * inv, acc[4 * e + 1] * inv),
                               f32x2_to_bf16x2(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv));
  }
}

}  // namespace tree
}  // namespace kvq
