// kvq_fp4_prefill.cuh -- prefill attention over the microscaled 4-bit cache on
// the 5th-generation tensor cores (tcgen05, accumulators in tensor memory).
//
//   O = softmax(q K^^T / sqrt(dh)) V^,  K^ = code * block scale * sK
//
// An item of work is one or two tiles of query rows of a sequence and KV head; a CTA
// takes an item, or a share of its keys.  A row is a (query token, query head of the
// group) pair, a tile 128 of them (128 / G tokens).  The visible pages of the CTA's
// rows (the first tokens' pages, then the window's) form a list, taken in blocks of
// 8 pages = 128 keys:
//   warp 16 (producer)    copies a block's 8 K pages, then its 8 V pages (one
//     bulk copy a page: codes and scales), into a ring of 3 stages
//   warps 8-11 and 12-15 (converters of K, of V)  code * block scale as f16 (exact),
//     both token-major in the 128-byte-swizzled layout, two buffers each; K runs a
//     block ahead, as its buffer is let go of half a block before V's
//   warps 17, 18 (one per tile)  one lane each issues, for each half (64 keys) of a
//     block, S = Q K^T (M 128, N 64) and, as the softmax delivers P, O += P V
//     (A = P from tensor memory, K 64), then the half's next S at once
//   warps 0-3, 4-7 (softmax of tiles 0, 1; thread = row = TMEM lane)  64 keys
//     at a time: S from TMEM, mask, P = 2^(x - m + 7) as f16 over the S columns
//     that it came from, with the running maximum m raised lazily (and O rescaled).
//     One f16 a weight: within 2^-11, which bf16's 2^-8 in the output covers (error against 64
//     bits 0.0017 relative, with binary32 weights 0.0016 to 0.0017); a second part would double P V,
//     and the operands' share of shared memory with it
// S and P share columns: 2 tiles x (2 halves of 64 + 128 of O) fill the 512.  A
// half's next S waits for the PV that reads its P, while the softmax works on the
// other half.  The softmax takes most registers (setmaxnreg).
//
// What bounds it: an N 64 step reads 6 KB of shared memory in 48 cycles (128 bytes a
// cycle, all there are), an N 128 step 8 KB in 64: for the two tiles' block 32 x 48 +
// 16 x 64 = 2560 cycles beside the converters' loads and stores, of about 4000 measured.
// Shared memory's bandwidth is 82% taken (50 operands, 32 converters); the rest is the
// chain of a half, softmax, P V, next S.  2048 queries of 32 heads over 32768 tokens,
// 8 KV heads of 128 dims: 859 to 865 us, 1240 TFLOP/s (563 us at the measured bf16 rate).
// On the way: S in steps of N 128, tiles taking turns 1201 us; halves 1106; issue
// under elect.sync, K and V converted by a warpgroup each 927; the rest after whole
// waves split 857.  S in one 64-column buffer with two of P beside it 987.
// Equal stretches of all items' keys for every SM instead of whole items: 1107 where
// whole ones took 1106, and small calls a third slower.  Codes read 16 bytes a lane,
// free of bank conflicts: 855.
//
// Where items leave SMs idle the host splits their blocks over several CTAs; each
// leaves (m, l, O) of its rows in the workspace and the one that completes the item
// merges them.
//
// Every wait is bounded; a timeout sets KVQ_DEV_WAIT_TIMEOUT, the roles stop,
// and the CTA waits (bounded) for copies and matrix steps in flight.
#pragma once

#include "kvq_decode.cuh"
#include "kvq_fp4.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace fp4 {

constexpr int kRows = 128;   // query rows of a tile (MMA M)
constexpr int kTiles = 2;    // tiles of a CTA
constexpr int kKeys = 128;   // keys of a block
constexpr int kBlkPages = kKeys / kTok;
constexpr int kPreThreads = 640;
constexpr int kConvWarp = 8, kProdWarp = 16, kMmaWarp = 17;
// Registers of a thread at launch, of the 256 softmax, the 256 converter and the 128 other threads
// while they have their parts, and again what all had for the merge, which all take part in.
constexpr int kLaunchRegs = 96, kSoftRegs = 136, kConvRegs = 72, kIssueRegs = 64;
static_assert(256 * kSoftRegs + 256 * kConvRegs + 128 * kIssueRegs <= kPreThreads * kLaunchRegs, "registers");
constexpr uint32_t kTmemCols = 512, kTileCols = 256;  // per tile: S and P at +0, O at +128
constexpr int kPreStages = 3, kBufs = 2;
constexpr float kPreBias = 7.f;  // log2 of the factor that the weights carry
constexpr float kFarMax = 0x1p16f;  // maxima (in exponents) from which keys lose them before the scale

struct PreParams {
  const uint16_t* q;
  const int32_t* cu_q;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  int max_blocks, B, Hq, Hkv, G;
  int64_t num_blocks, total_q;
  int window, sinks;
  int tiles;   // tiles of the longest chunk
  int tpc;     // tiles of a CTA
  int groups;  // items of a sequence and KV head: tpc tiles each
  int64_t whole;   // items that one CTA each takes, the first ones
  int ns;          // shares of the keys of the items after them, at most
  int min_share;   // blocks of a share, at least
  const float* ks;
  const float* vs;
  int per_head;
  float logit_scale;  // log2(e) / sqrt(dh)
  uint32_t* ws_cnt;   // [shared item] arrivals
  float2* ws_ml;      // [share][kTiles * kRows]
  float* ws_o;        // [share][kTiles * kRows][DH]
  uint16_t* out;
  uint32_t* status;
  int withhold;       // test builds: stage of CTA 0's run that is never copied; -1
};

// Workspace: the arrival counters (kvq_decode_attn's table), then the states of the rows
// of each share, at most kShares per SM.
constexpr int kShares = 3;
struct PreWs {
  size_t ml, o, total;
};
inline PreWs pre_ws(int DH, int sms) {
  const size_t rows = static_cast<size_t>(sms) * kShares * kTiles * kRows;
  PreWs w;
  w.ml = KVQ_WS_COUNTER_BYTES;
  w.o = w.ml + round256(rows * sizeof(float2));
  w.total = w.o + round256(rows * DH * sizeof(float));
  return w;
}

template <int DH>
struct PreSmem {
  static constexpr int kStage = kBlkPages * Page<DH>::kBytes;
  static constexpr int kTile = kKeys * DH * 2;  // K or V buffer, f16
  static constexpr int q = 0;                   // kTiles x [128][DH] f16
  static constexpr int k = q + kTiles * kRows * DH * 2;
  static constexpr int v = k + kBufs * kTile;
  static constexpr int stage = v + kBufs * kTile;
  static constexpr int bars = stage + kPreStages * kStage;
  static constexpr int kBars = 2 * kPreStages + 4 * kBufs + 6 * kTiles + 2;
  static constexpr int misc = bars + kBars * 8;
  // tmem address, abort flag, V NaN flag, merge flag, page flags [stages][8], issued [stages], masks [4]
  static constexpr int total = misc + (4 + kPreStages * 9 + 4) * 4 + 1024;
  static_assert(total <= 227 * 1024, "shared memory");
};

// Byte offset of f16 element (row, col) in a 128-row tile of 128-byte-swizzled
// rows of 64 columns (wider tiles: further 64-column blocks).
KVQ_DEVI uint32_t tile_off(int row, int col) {
  const int blk = col >> 6, c16 = (col & 63) >> 3;
  return static_cast<uint32_t>(blk * (128 * 128) + (row >> 3) * 1024 + (row & 7) * 128 +
                               ((c16 ^ (row & 7)) << 4) + ((col & 7) << 1));
}

using tc::elect_one;
using tc::f32x2;
using tc::f32x2_add;
using tc::f32x2_fma;
using tc::f32x2_pack;
using tc::f32x2_unpack;
using tc::fmax3;
using tc::tmem_ld64;
using tc::tmem_st8;

// The pages that a CTA's rows see, as a list: the first tokens' pages [0, sink),
// then [first, last].
struct PageList {
  int sink, first, count;
  KVQ_DEVI int col(int i) const { return i < sink ? i : first + i - sink; }
};

// A CTA converts its nb blocks in the order K0 K1 V0 K2 V1 ... V(nb - 1): a K buffer is
// free half a block before the V buffer.  Item `it` of these, and the last K up to it.
struct PreTask {
  int block, last_k;
  bool v;
};
KVQ_DEVI PreTask pre_task(int it, int nb) {
  const bool v = it == 2 * nb - 1 || (it > 0 && (it & 1) == 0);
  const int k = min((it + 1) >> 1, nb - 1);
  return {v ? (it == 2 * nb - 1 ? nb - 1 : (it >> 1) - 1) : k, k, v};
}

template <int DH>
__global__ void __launch_bounds__(kPreThreads, 1) prefill_kernel(const __grid_constant__ PreParams p) {
  using SM = PreSmem<DH>;
  using PG = Page<DH>;
  constexpr int S = kPreStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::bars);  // [S] a stage landed
  uint64_t* empty = full + S;            // [S] a stage converted, and seen by the other converters (256 arrivals)
  uint64_t* conv_k = empty + S;          // [kBufs] K buffer filled (128)
  uint64_t* conv_v = conv_k + kBufs;     // [kBufs]
  uint64_t* done_k = conv_v + kBufs;     // [kBufs] K buffer read by both tiles (a commit each)
  uint64_t* done_v = done_k + kBufs;     // [kBufs]
  uint64_t* sfull = done_v + kBufs;      // [kTiles][2] a half of S written (commit, and the issuer's arrival)
  uint64_t* pfull = sfull + 2 * kTiles;  // [kTiles][2] the half of P written, of S read (128)
  uint64_t* pdone = pfull + 2 * kTiles;  // [kTiles][2] its PV done (commit, and the issuer's arrival)
  uint64_t* fin = pdone + 2 * kTiles;    // every matrix step done (a commit of each issuer)
  uint64_t* qready = fin + 1;            // both Q tiles written (256)
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + SM::misc);
  volatile uint32_t* tmem_slot = misc;
  volatile uint32_t* abort_flag = misc + 1;
  volatile uint32_t* vnan = misc + 2;    // a V block of the list has a NaN scale
  volatile uint32_t* merge_s = misc + 3;
  volatile uint32_t* pg_bad = misc + 4;  // [S][8]
  volatile int32_t* issued = reinterpret_cast<volatile int32_t*>(misc + 4 + S * 8);  // [S] last item
  // masked pages of block j at [j % 4]: rewritten for block j + 4, whose K waits
  // for the QKs of block j + 2, which come after the softmax of block j + 1
  volatile uint32_t* bmask = misc + 4 + S * 9;

  // A parity wait for phase k of a barrier is sound while the barrier has
  // completed k or k + 1 phases.  Each waiter takes its barriers' phases in
  // order (the converters of K wait for V's copies too, and the other way round, and the stage
  // waits for both: a waiter that skipped a phase could take the one before for its own), but for
  // the softmax's waits for pdone, where O is rescaled: S of half h
  // of block i came after the PV of half h of block i - 1, and that PV's next phase
  // needs this softmax's own later progress.

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t cta = blockIdx.x;
  const int64_t shared = cta < p.whole ? 0 : (cta - p.whole) / p.ns;  // which of the shared items
  const int64_t item = cta < p.whole ? cta : p.whole + shared;
  const int share = cta < p.whole ? 0 : static_cast<int>((cta - p.whole) % p.ns);
  const int group = p.groups - 1 - static_cast<int>(item % p.groups);  // longest first
  const int b = static_cast<int>(item / p.groups / p.Hkv), gkv = static_cast<int>(item / p.groups % p.Hkv);
  const int TQ = kRows / p.G;  // query tokens of a tile

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 256);
      issued[i] = -1;
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&conv_k[i], 128);
      mbar_init(&conv_v[i], 128);
      mbar_init(&done_k[i], kTiles);
      mbar_init(&done_v[i], kTiles);
    }
    for (int t = 0; t < 2 * kTiles; ++t) {
      mbar_init(&sfull[t], 2);
      mbar_init(&pfull[t], 128);
      mbar_init(&pdone[t], 2);
    }
    mbar_init(fin, kTiles);
    mbar_init(qready, kTiles * 128);
    *abort_flag = 0u;
    *vnan = 0u;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_allow_next();

  const int q0 = __ldg(p.cu_q + b);
  const int q1 = __ldg(p.cu_q + b + 1);
  const bool bad_q = q0 < 0 || q1 < q0 || q1 > p.total_q;  // no rows of its own
  const int n = bad_q ? 0 : q1 - q0;
  const int j0 = group * p.tpc * TQ;  // first query token of tile 0
  if (group == 0 && share == 0 && gkv == 0 && tid == 0 && (bad_q || n > p.tiles * TQ))
    flag_status(p.status, KVQ_DEV_BAD_QLEN);
  if (n == 0 || j0 >= min(n, p.tiles * TQ)) return;
  const int nc = min(n, p.tiles * TQ);  // query tokens that the grid covers
  const int j1 = min(nc, j0 + p.tpc * TQ);
  const int L = __ldg(p.seq_lens + b);
  if (L < n || L > p.max_blocks * kTok) {
    if (group == 0 && share == 0 && gkv == 0 && tid == 0) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
    if (share == 0)
      for (int i = tid; i < (j1 - j0) * p.G * DH; i += kPreThreads) {
        const int r = i / DH, d = i - r * DH;
        p.out[((static_cast<int64_t>(q0) + j0 + r / p.G) * p.Hq + gkv * p.G + r % p.G) * DH + d] = 0;
      }
    return;
  }
  const int base = L - n;  // position of query token 0
  // the list from what the first row sees to the last row's own token
  const Visible v0 = visible(p.window, p.sinks, base + j0 + 1);
  const PageList list = {v0.sink, v0.first, v0.sink + (base + j1 - 1) / kTok - v0.first + 1};
  const int nall = (list.count + kBlkPages - 1) / kBlkPages;
  // few blocks need fewer CTAs
  const int ns = cta < p.whole ? 1 : max(1, min(p.ns, nall / p.min_share));
  if (share >= ns) return;
  // this CTA's blocks [c0, c1) and tile t's [jb, je) of them
  const int c0 = static_cast<int>(static_cast<int64_t>(nall) * share / ns);
  const int c1 = static_cast<int>(static_cast<int64_t>(nall) * (share + 1) / ns);
  const int nb = c1 - c0;
  int jb[kTiles], je[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int a = j0 + t * TQ, e = min(nc, a + TQ);
    if (t >= p.tpc || a >= nc) {
      jb[t] = je[t] = c0;
    } else {
      const int lo = visible(p.window, p.sinks, base + a + 1).first;
      // (where the first row still sees all tokens, the list has no first part, but tile 1 may
      // need its first pages all the same)
      jb[t] = max(c0, p.sinks > 0 ? 0 : (lo - list.first) / kBlkPages);
      je[t] = min(c1, (list.sink + (base + e - 1) / kTok - list.first) / kBlkPages + 1);
      if (je[t] < jb[t]) je[t] = jb[t];
    }
  }

  if (warp == kMmaWarp) tc::tmem_alloc(const_cast<uint32_t*>(tmem_slot), kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&] {
    if (!*abort_flag) {
      *abort_flag = 1u;
      flag_status(p.status, KVQ_DEV_WAIT_TIMEOUT);
    }
  };
  auto wait_w = [&](uint64_t* bar, int phase) {  // warp-uniform
    return __all_sync(kFull, wait_or_abort(bar, static_cast<uint32_t>(phase & 1), abort_flag));
  };

  if (warp >= kProdWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
  if (warp == kProdWarp) {
    // ------------------------------------------------------------ producer
    // The 32 lanes look up the block ids of 4 blocks at once; lanes 0-7 copy a page each.
    int64_t my_at = -1, old_at = -1;  // byte offset of list page 8 (c0 + i - i % 4) + lane, -1: masked out
    for (int it = 0; it < 2 * nb; ++it) {
      const int s = it % S;
      const PreTask task = pre_task(it, nb);
      const int i = task.block;
      if (!task.v && (i & 3) == 0) {
        const int lp = kBlkPages * (c0 + i) + lane;
        old_at = my_at;  // V is at most two blocks behind K
        my_at = -1;
        if (lp < list.count) {
          const int col = list.col(lp);
          const int blk = col >= 0 && col < p.max_blocks
                              ? __ldg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks + col)
                              : -1;
          if (blk >= 0 && blk < p.num_blocks)
            my_at = (static_cast<int64_t>(blk) * p.Hkv + gkv) * PG::kBytes;
          else
            flag_status(p.status, KVQ_DEV_BAD_BLOCK);
        }
      }
      const bool old = task.v && (i >> 2) != (task.last_k >> 2);
      const int64_t at = __shfl_sync(kFull, old ? old_at : my_at, 8 * (i & 3) + (lane & 7));
      const bool ok = it < S || wait_w(&empty[s], it / S - 1);
      if (__any_sync(kFull, !ok || *abort_flag)) {
        if (lane == 0) fail();
        break;
      }
#ifdef KVQ_TEST_HOOKS
      if (cta == 0 && it == p.withhold) continue;  // its full barrier never completes
#endif
      const uint32_t good = __ballot_sync(kFull, lane < kBlkPages && at >= 0);
      if (lane < kBlkPages) pg_bad[s * 8 + lane] = at < 0;
      __syncwarp();
      if (lane == 0) {
        issued[s] = it;
        if (good == 0)
          mbar_arrive(&full[s]);  // nothing to copy
        else
          mbar_arrive_expect_tx(&full[s], __popc(good) * PG::kBytes);
      }
      __syncwarp();
      if (lane < kBlkPages && at >= 0)
        bulk_load(smem + SM::stage + s * SM::kStage + lane * PG::kBytes, (task.v ? p.vc : p.kc) + at,
                  PG::kBytes, &full[s]);
    }
  } else if (warp < kMmaWarp + kTiles) {
    // ------------------------------------------------------------ matrix steps of one tile
    const int t = __shfl_sync(kFull, warp, 0) - kMmaWarp;
    const uint32_t tmem_u = __shfl_sync(kFull, tmem, 0);
    if (elect_one()) {
      const uint32_t id_qk = tc::idesc_f16(kRows, kKeys / 2), id_pv = tc::idesc_f16(kRows, DH) | (1u << 16);
      const uint32_t tm = tmem_u + t * kTileCols;
      auto wait = [&](uint64_t* bar, int phase) {
        return wait_or_abort(bar, static_cast<uint32_t>(phase & 1), abort_flag);
      };
      // S of half h of block j
      auto qk = [&](int j, int h) {
        tc::tc_fence_after();
        const uint32_t a = sbase + SM::q + t * kRows * DH * 2;
        const uint32_t bk = sbase + SM::k + (j - c0) % kBufs * SM::kTile + h * 8192;
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          const uint32_t o = (k >> 2) * (128 * 128) + (k & 3) * 32;
          tc::mma_f16_ss(tm + h * 64, tc::sw128_desc(a + o), tc::sw128_desc(bk + o), id_qk, k > 0 ? 1u : 0u);
        }
        mbar_arrive(&sfull[2 * t + h]);  // hands on what conv_k's arrival showed (bmask)
        tc::mma_commit(&sfull[2 * t + h]);
      };
      bool ok = wait(qready, 0);
      for (int j = c0; j < c1 && ok; ++j) {
        const int i = j - jb[t], x = (j - c0) % kBufs, ph = (j - c0) / kBufs;
        const bool active = j >= jb[t] && j < je[t], more = active && j + 1 < je[t];
        if (!active || i == 0) {  // (later blocks' S was issued beside the block before)
          if (!(ok = wait(&conv_k[x], ph))) break;
          if (active) {
            qk(j, 0);
            qk(j, 1);
          }
          tc::mma_commit(&done_k[x]);
        }
        if (!(ok = wait(&conv_v[x], ph))) break;
        for (int h = 0; h < 2 && active && ok; ++h) {
          if (!(ok = wait(&pfull[2 * t + h], i))) break;
          tc::tc_fence_after();
          // V token-major: MN-major B, 64 dims a 128-byte row, 16 tokens = two 8-row groups
          const uint32_t bv = sbase + SM::v + x * SM::kTile + h * 8192;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_f16_ts(tm + 128, tm + h * 64 + k * 8, tc::sw128_desc(bv + k * 2048, 128 * 128, 1024),
                           id_pv, (i > 0 || h > 0 || k > 0) ? 1u : 0u);
          mbar_arrive(&pdone[2 * t + h]);  // hands on what conv_v's arrival showed (vnan)
          tc::mma_commit(&pdone[2 * t + h]);
          if (more) {  // the half's next S, over the P that this PV has read, beside the other half's softmax
            const int xn = (j + 1 - c0) % kBufs;
            if (h == 0 && !(ok = wait(&conv_k[xn], (j + 1 - c0) / kBufs))) break;
            if (!(ok = wait(&pdone[2 * t + h], i))) break;
            qk(j + 1, h);
            if (h == 1) tc::mma_commit(&done_k[xn]);
          }
        }
        if (!ok) break;
        tc::mma_commit(&done_v[x]);
      }
      if (!ok) fail();
      tc::mma_commit(fin);
      if (!mbar_wait(fin, 0u)) fail();
    }
  }
  } else if (warp >= kConvWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // ------------------------------------------------------------ converters
    const bool is_v = warp >= kConvWarp + 4;
    const int ct = tid & 127;
    for (int it = 0; it < 2 * nb; ++it) {
      const PreTask task = pre_task(it, nb);
      const int i = task.block, s = it % S, x = i % kBufs;
      bool ok = wait_w(&full[s], it / S);
      if (ok && task.v != is_v) {  // the other warpgroup's
        mbar_arrive(&empty[s]);
        continue;
      }
      if (ok && i >= kBufs) ok = wait_w(is_v ? &done_v[x] : &done_k[x], i / kBufs - 1);
      if (!ok) {
        fail();
        break;
      }
      uint32_t bm = 0;
#pragma unroll
      for (int e = 0; e < kBlkPages; ++e) bm |= (pg_bad[s * 8 + e] ? 1u : 0u) << e;
      if (ct == 0 && !is_v) bmask[(c0 + i) & 3] = bm;
      // Thread ct converts 16 dims of rows r0, r0 + 32, r0 + 64, r0 + 96 (pages p0, p0 + 2, ...,
      // all at row r0 % 16 of theirs), for each 64 dims of the head: block ct % 4 of the 64.  Eight
      // lanes' 16-byte stores (two rows, four swizzled columns each) cover all banks.
      const int r0 = ct >> 2, c4 = ct & 3, tr = r0 & 15, p0 = r0 >> 4;
      const uint8_t* src = smem + SM::stage + s * SM::kStage + p0 * PG::kBytes;
      const uint8_t* code = src + tr * PG::kRow + c4 * 8;
      const uint8_t* scale = src + PG::kScaleOff + tr * PG::kScales + c4;
      uint8_t* dst = smem + (is_v ? SM::v : SM::k) + x * SM::kTile + (r0 >> 3) * 1024 + (r0 & 7) * 128;
      uint8_t* lo = dst + (((2 * c4) ^ (r0 & 7)) << 4);
      uint8_t* hi = dst + (((2 * c4 + 1) ^ (r0 & 7)) << 4);
      // Masked pages may hold anything.  Their keys are masked later; values count as 0, like
      // those past the sequence (weights of 0 do not clear a NaN), and so do NaN blocks, which
      // the epilogue puts back where they are seen.
      uint32_t keep = 0xFu;  // bit y: row r0 + 32 y
      if (is_v && (bm || kBlkPages * (c0 + i + 1) >= list.count)) {  // (L ends in the list's last page)
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if ((bm >> (p0 + 2 * y) & 1u) || list.col(kBlkPages * (c0 + i) + p0 + 2 * y) * kTok + tr >= L) keep &= ~(1u << y);
      }
      bool nan = false;
#pragma unroll
      for (int y = 0; y < 4 * (DH / 64); ++y) {
        const int yr = y & 3, yc = y >> 2;
        const uint2 w = *reinterpret_cast<const uint2*>(code + yr * 2 * PG::kBytes + yc * 32);
        uint32_t sb = scale[yr * 2 * PG::kBytes + yc * 4];
        if (is_v) {
          const bool bad = (sb & 0x7Fu) == 0x7Fu, in = keep >> yr & 1u;
          nan |= bad && in;
          sb = bad || !in ? 0u : sb;
        }
        const uint32_t f = fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(sb * 0x101u));
        uint32_t a[4], d[4];
        e2m1x8_to_f16x2x4(w.x, a);
        e2m1x8_to_f16x2x4(w.y, d);
        *reinterpret_cast<uint4*>(lo + yr * 4096 + yc * 16384) =
            make_uint4(hmul2(a[0], f), hmul2(a[1], f), hmul2(a[2], f), hmul2(a[3], f));
        *reinterpret_cast<uint4*>(hi + yr * 4096 + yc * 16384) =
            make_uint4(hmul2(d[0], f), hmul2(d[1], f), hmul2(d[2], f), hmul2(d[3], f));
      }
      if (nan) *vnan = 1u;
      fence_proxy_async_smem();  // generic writes -> the tensor core's reads
      mbar_arrive(is_v ? &conv_v[x] : &conv_k[x]);
      mbar_arrive(&empty[s]);
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int t = warp >> 2, r = tid & 127;
    const int jr = j0 + t * TQ + r / p.G;  // query token of this row
    const bool live = t < p.tpc && r < TQ * p.G && jr < nc;
    const int pos = base + jr;
    const int lo = live && p.window > 0 && pos >= p.window ? pos + 1 - p.window : 0;
    const int64_t qrow = live ? (static_cast<int64_t>(q0) + jr) * p.Hq + gkv * p.G + r % p.G : 0;
    const uint32_t tm_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * kTileCols;
    const uint32_t tm_o = tm_s + 128;
    // the query row times a power of two 2^a, its largest value in [2^14, 2^15): f16, exact for
    // values down to 2^-17 (8 significant bits over a least step of 2^-24), off by 2^-25 at most below
    float lscale = __ldg(p.ks + (p.per_head ? gkv : 0));
    {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + qrow * DH);
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < DH / 8; ++c) {
        const uint4 w = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(bf16lo_to_f32(u[e])), fabsf(bf16hi_to_f32(u[e]))));
      }
      int a = 0;
      if (amax > 0.f) {
        a = 14 - (static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu) - 127);
        a = a > 126 ? 126 : (a < -126 ? -126 : a);
      }
      const float up = __int_as_float((a + 127) << 23);
      lscale = bounded_scale(lscale * __int_as_float((127 - a) << 23) * p.logit_scale);
#pragma unroll
      for (int c = 0; c < DH / 8; ++c) {
        const uint4 w = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = f32x2_to_f16x2(bf16lo_to_f32(u[e]) * up, bf16hi_to_f32(u[e]) * up);
        tc::sts128(sbase + SM::q + t * kRows * DH * 2 + tile_off(r, 8 * c), h[0], h[1], h[2], h[3]);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(qready);
    // m, a raw dot product; the exponents' offset 7 - m lscale (7 while every key so far is masked and
    // m is -inf: any finite value keeps 2^-inf = 0, and a NaN)
    float m = -INFINITY, l = 0.f, off = kPreBias;
    const float rise = kRescaleThreshold / lscale;
    bool far = false;  // a row of the warp has a maximum past kFarMax
    bool ok = true;
    const int nI = je[t] - jb[t];
    const bool some = __any_sync(kFull, live);
    for (int i = 0; i < 2 * nI && ok && !some; ++i) {  // no row of the warp is asked for: any P does
      if ((ok = wait_w(&sfull[2 * t + (i & 1)], i >> 1))) mbar_arrive(&pfull[2 * t + (i & 1)]);
    }
    for (int i = 0; i < nI && ok && some; ++i) {
      const int j = jb[t] + i;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (!(ok = wait_w(&sfull[2 * t + h], i))) break;
        const uint32_t bm8 = bmask[j & 3];
        tc::tc_fence_after();
        float x[64];
        tmem_ld64(tm_s + h * 64, x);
        const int lp = j * kBlkPages + h * 4;  // list page of the half's first key
        const uint32_t bm = (bm8 >> (4 * h)) & 15u;
        const int k0 = list.col(lp) * kTok;
        // the row sees all 64 keys: four consecutive pages inside its window, or of its first tokens
        const bool whole = (bm == 0u && k0 + 63 <= pos &&
                                     (lp >= list.sink ? k0 >= lo : lp + 3 < list.sink && k0 + 63 < p.sinks));
        if (!whole) {
#pragma unroll
          for (int e4 = 0; e4 < 4; ++e4) {
            const int kp0 = list.col(lp + e4) * kTok;
            auto below = [&](int end) { return (1u << min(max(end - kp0, 0), kTok)) - 1u; };  // keys before `end`
            const uint32_t seen = bm >> e4 & 1u ? 0u : below(pos + 1) & (~below(lo) | below(p.sinks));
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[16 * e4 + e] = seen >> e & 1u ? x[16 * e4 + e] : -INFINITY;
          }
        }
        // Weights against the maximum so far, which grows rarely, and the half's own maximum
        // beside them (no wait of one for the other); where it grew by over 8, O and l are
        // rescaled and the weights formed again.
        float sum, mx;
        auto weights = [&](float off) {
          const f32x2 sc2 = f32x2_pack(lscale, lscale), off2 = f32x2_pack(off, off);
          f32x2 l2[2] = {f32x2_pack(0.f, 0.f), f32x2_pack(0.f, 0.f)};
          float mx2[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t ph[8];
#pragma unroll
            for (int e2 = 0; e2 < 8; ++e2) {
              const int e = 16 * c + 2 * e2;
              float p0, p1;
              f32x2_unpack(f32x2_fma(f32x2_pack(x[e], x[e + 1]), sc2, off2), p0, p1);
              p0 = fast_exp2(p0);
              p1 = fast_exp2(p1);
              l2[e2 & 1] = f32x2_add(l2[e2 & 1], f32x2_pack(p0, p1));
              mx2[e2 & 1] = fmax3(mx2[e2 & 1], x[e], x[e + 1]);
              ph[e2] = f32x2_to_f16x2(p0, p1);
            }
            tmem_st8(tm_s + h * 64 + 8 * c, ph);
          }
          float s0, s1;
          f32x2_unpack(f32x2_add(l2[0], l2[1]), s0, s1);
          sum = s0 + s1;
          mx = fmaxf(mx2[0], mx2[1]);
        };
        weights(off);
        const bool grow = mx > m + rise;
        if (__any_sync(kFull, grow) || far) {
          // O's last writer: the PV of the half before
          if (h == 1 ? !(ok = wait_w(&pdone[2 * t], i)) : i > 0 && !(ok = wait_w(&pdone[2 * t + 1], i - 1))) break;
          tc::tc_fence_after();
          const float nm = grow ? mx : m;
          const float a = m == -INFINITY ? 0.f : fast_exp2((m - nm) * lscale);
          if (i > 0 || h > 0) {
#pragma unroll 1
            for (int c = 0; c < DH; c += 16) {
              uint32_t o[16];
              tc::tmem_ld16(tm_o + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (grow ? a : 1.f));
              tc::tmem_st16(tm_o + c, o);
            }
          }
          if (grow) l *= a;
          m = nm;
          // The offset's rounding, up to 2^-24 of the maximum's exponent, is common to all keys and
          // cancels, but from about 2^27 on it takes the weights out of f16's range.  Rows far below
          // that already subtract the maximum itself: its key's exponent is exactly 7.  (In place of
          // the offset for all rows: 918 us where this takes 861, 2048 queries over 32768 tokens.)
          const float fm = m == -INFINITY ? 0.f : m;
          off = fmaf(-fm, lscale, kPreBias);
          far = __any_sync(kFull, fabsf(fm) * lscale > kFarMax);
          if (far) {
#pragma unroll
            for (int e = 0; e < 64; ++e) x[e] -= fm;
          }
          weights(far ? kPreBias : off);
        }
        l += sum;
        tc::tmem_st_wait();
        tc::tc_fence_before();
        mbar_arrive(&pfull[2 * t + h]);
      }
    }
    if (ok && nI > 0) ok = wait_w(&pdone[2 * t], nI - 1) && wait_w(&pdone[2 * t + 1], nI - 1);
    if (!ok) {
      tc::tmem_st_wait();  // (weights of the half that was given up)
      fail();
    }
    // ---- epilogue: the row of O, normalised, or (keys shared out) as it is
    const float sv = __ldg(p.vs + (p.per_head ? gkv : 0));
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int64_t part = (cta - p.whole) * (kTiles * kRows) + t * kRows + r;
    tc::tc_fence_after();
    if (ok) {
      if (ns > 1 && live) p.ws_ml[part] = make_float2(merge_max(m, lscale), l);
#pragma unroll 1
      for (int c = 0; c < DH; c += 32) {
        float o[32];
        if (nI > 0) {
          tc::tmem_ld32(tm_o + c, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (*vnan && live) {  // put back the NaN of the blocks that this row sees
          for (int lp = c0 * kBlkPages; lp < min(list.count, c1 * kBlkPages); ++lp) {
            const int col = list.col(lp);
            const int blk = __ldg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks + col);
            if (blk < 0 || blk >= p.num_blocks) continue;
            const uint8_t* sc = p.vc + (static_cast<int64_t>(blk) * p.Hkv + gkv) * PG::kBytes + PG::kScaleOff + c / 16;
            for (int e = 0; e < kTok; ++e) {
              const int kp = col * kTok + e;
              if (!(kp <= pos && (kp >= lo || kp < p.sinks))) continue;
#pragma unroll
              for (int y = 0; y < 2; ++y)
                if ((sc[e * PG::kScales + y] & 0x7Fu) == 0x7Fu)
#pragma unroll
                  for (int z = 0; z < 16; ++z) o[16 * y + z] = NAN;
            }
          }
        }
        if (live && ns == 1) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + qrow * DH + c);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            dst[y] = make_uint4(output2(o[8 * y], o[8 * y + 1], inv, sv), output2(o[8 * y + 2], o[8 * y + 3], inv, sv),
                                output2(o[8 * y + 4], o[8 * y + 5], inv, sv), output2(o[8 * y + 6], o[8 * y + 7], inv, sv));
        } else if (live) {
          float4* dst = reinterpret_cast<float4*>(p.ws_o + part * DH + c);
#pragma unroll
          for (int y = 0; y < 8; ++y) dst[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
        }
      }
    }
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLaunchRegs));
  }

  tc::tc_fence_before();
  __syncthreads();
  // Every softmax warp has let go of its registers.  (A warp that took its own back any earlier
  // could take them from a softmax warp that waits for them at its start.)
  if (warp >= kConvWarp) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLaunchRegs));
  // After an abort: wait (bounded) for the copies in flight; the issuers waited for their steps.
  if (*abort_flag && tid == 0)
    for (int s = 0; s < S; ++s)
      if (issued[s] >= 0) mbar_wait(&full[s], static_cast<uint32_t>((issued[s] / S) & 1));
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
  if (ns == 1) return;

  // ---- the CTA that completes a tile group merges its shares: the barriers above
  // order every thread's stores before thread 0's acquire-release arrival
  const int64_t first = cta - p.whole - share;
  uint32_t* cnt = p.ws_cnt + shared;
  if (tid == 0) *merge_s = atom_add_acq_rel_gpu(cnt, 1u) + 1 == static_cast<uint32_t>(ns);
  __syncthreads();
  if (!*merge_s) return;
  if (tid == 0) *cnt = 0u;
  const float sv = __ldg(p.vs + (p.per_head ? gkv : 0));
  const int rows = kTiles * kRows;
  const int live0 = min(TQ, nc - j0) * p.G;  // live rows of tile 0, then of both
  const int live = live0 + (p.tpc > 1 ? max(0, min(TQ, nc - j0 - TQ)) * p.G : 0);
  for (int i = tid; i < live * (DH / 4); i += kPreThreads) {
    const int at = i / (DH / 4), e = i - at * (DH / 4);
    const int t = at >= live0, r = t ? at - live0 : at, row = t * kRows + r;
    const int jr = j0 + t * TQ + r / p.G;
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int y = 0; y < ns; ++y) {
      const int64_t at = (first + y) * rows + row;
      const float2 ml = __ldcg(p.ws_ml + at);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.ws_o + at * DH) + e);
      const float nm = fmaxf(M, ml.x);
      const float a = M == -INFINITY ? 1.f : fast_exp2((M - nm) * kMergeUnit);
      const float w = ml.x == -INFINITY ? 1.f : fast_exp2((ml.x - nm) * kMergeUnit);
      l = l * a + ml.y * w;
      acc.x = acc.x * a + v.x * w;
      acc.y = acc.y * a + v.y * w;
      acc.z = acc.z * a + v.z * w;
      acc.w = acc.w * a + v.w * w;
      M = nm;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const uint2 o = make_uint2(output2(acc.x, acc.y, inv, sv), output2(acc.z, acc.w, inv, sv));
    const int64_t qrow = (static_cast<int64_t>(q0) + jr) * p.Hq + gkv * p.G + r % p.G;
    *reinterpret_cast<uint2*>(p.out + qrow * DH + 4 * e) = o;
  }
}

}  // namespace fp4
}  // namespace kvq
