// kvq_pages.cu -- rows and pages of the caches moved, and the pool that pages
// are taken from: kvq_tree_commit, kvq_copy_pages, kvq_pages_*.
//
// Nothing here computes: each kernel is a chain of a few dependent loads
// (lengths, then a path or a table, then rows) and then a copy, so the work
// is laid out to have all of a warp's rows in flight behind one such chain.
//
// The pool takes the lowest free pages first.  A bit for each free page makes
// that a prefix sum over num_blocks / 32 words (200 000 pages are 25 KB, where
// their counts are 800 KB) whose result depends on nothing but the pool:
// giving pages back in any order, by atomics, leaves the same pool.
#include <algorithm>
#include <functional>

#include "../../include/kvq_step.h"
#include "kvq_common.cuh"
#include "kvq_host.h"

namespace kvq {
namespace pages {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kTok = 16;
constexpr int kMaxRowsCaches = 128;  // caches of one launch (their descriptions are kernel parameters)
constexpr int kMaxTables = 4096;     // sequences of a pool's call

struct Caches {
  kvq_rows c[kMaxRowsCaches];
};

// ------------------------------------------------------------------ commit

struct CommitParams {
  int caches, B, hkv, max_blocks, max_path, first;  // first: this launch writes new_lens
  int shares;                                       // of a cache's heads, each a warp's
  int64_t num_blocks;
  const int32_t* cu_q;
  const int32_t* tables;
  const int32_t* seq_lens;
  const int32_t* path;
  const int32_t* taken;
  int32_t* new_lens;
  uint32_t* status;
};

constexpr int kUnits = 4;  // 16-byte (4-byte) units that a lane has in flight

// Rows [i0, i0 + c) of the path in heads [head0, head1), a T a unit: all of a head's rows are read before
// the first is written.  A path rises, so rows of later chunks come from at or behind their own places.
template <typename T>
KVQ_DEVI void move_rows(const CommitParams& p, uint8_t* data, int64_t page_bytes, int part_off, int row_bytes,
                        const int32_t* path, const int32_t* table, int before, int taken, int head0, int head1) {
  const int lane = threadIdx.x & 31;
  const int u = row_bytes / static_cast<int>(sizeof(T));  // units of a row
  if (u == 0) return;
  const int most = max(1, 32 * kUnits / u);
  for (int i0 = 0; i0 < taken; i0 += most) {
    const int c = min(most, taken - i0), per_head = c * u;
    const int hb = max(1, 32 * kUnits / per_head);  // heads of a batch
    for (int h0 = head0; h0 < head1; h0 += hb) {
      const int n = min(hb, head1 - h0) * per_head;
      T val[kUnits];
      T* dst[kUnits];
#pragma unroll
      for (int y = 0; y < kUnits; ++y) {
        const int x = lane + 32 * y;
        dst[y] = nullptr;
        if (x >= n) continue;
        const int h = x / per_head, r = (x - h * per_head) / u, e = x % u, i = i0 + r;
        const int from = __ldg(path + i);
        if (from == i) continue;  // in its place already
        const int s = before + from, d = before + i;
        const int ps = __ldg(table + s / kTok), pd = __ldg(table + d / kTok);
        if (ps < 0 || ps >= p.num_blocks || pd < 0 || pd >= p.num_blocks) {
          flag_status(p.status, KVQ_DEV_BAD_BLOCK);
          continue;
        }
        const int64_t head = h0 + h;
        const uint8_t* src = data + (ps * static_cast<int64_t>(p.hkv) + head) * page_bytes + part_off + (s % kTok) * row_bytes;
        dst[y] = reinterpret_cast<T*>(data + (pd * static_cast<int64_t>(p.hkv) + head) * page_bytes + part_off +
                                      (d % kTok) * row_bytes) + e;
        val[y] = reinterpret_cast<const T*>(src)[e];
      }
      __syncwarp();
#pragma unroll
      for (int y = 0; y < kUnits; ++y)
        if (dst[y]) *dst[y] = val[y];
      __syncwarp();
    }
  }
}

// A warp takes a sequence and a share of a cache's heads: up to 2 KB of rows in flight behind one
// chain of lengths, path and table (some 4 us with the launch).  Heads are shared out until the GPU's
// warps are taken: with all of a cache's heads to a warp, 32 sequences' paths in 32 caches of 8 heads
// took 8.1 us, several chains' time at 7 warps an SM; shared out 6.4.
__global__ void __launch_bounds__(128, 8) commit_kernel(const __grid_constant__ CommitParams p,
                                                     const __grid_constant__ Caches cs) {
  pdl_wait();
  pdl_allow_next();
  const int lane = threadIdx.x & 31;
  const int per = max(1, p.caches * p.shares);
  const int64_t items = static_cast<int64_t>(p.B) * per, warps = static_cast<int64_t>(gridDim.x) * 4;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5); it < items; it += warps) {
    const int b = static_cast<int>(it / per), at = static_cast<int>(it - static_cast<int64_t>(b) * per);
    const int c = at / p.shares, share = at - c * p.shares;
    const int L = __ldg(p.seq_lens + b), q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
    const int taken = __ldg(p.taken + b);
    const int32_t* path = p.path + static_cast<int64_t>(b) * p.max_path;
    const bool bad_q = q0 < 0 || q1 < q0;
    const int n = bad_q ? 0 : q1 - q0;
    const bool bad_len = L < n || L > p.max_blocks * kTok;
    bool good = taken >= 0 && taken <= min(n, p.max_path);
    if (good && !bad_q && !bad_len) {
      bool rises = true;
      for (int i = lane; i < taken; i += 32) {
        const int node = __ldg(path + i);
        rises = rises && node >= 0 && node < n && (i == 0 || __ldg(path + i - 1) < node);
      }
      good = __all_sync(kAll, rises);
    }
    const bool moves = good && !bad_q && !bad_len;
    if (at == 0 && p.first && lane == 0) {
      p.new_lens[b] = moves ? L - n + taken : L;
      if (!moves) flag_status(p.status, bad_q ? KVQ_DEV_BAD_QLEN : bad_len ? KVQ_DEV_BAD_SEQLEN : KVQ_DEV_BAD_TREE);
    }
    if (!moves || p.caches == 0) continue;
    const kvq_rows r = cs.c[c];
    const int32_t* table = p.tables + static_cast<int64_t>(b) * p.max_blocks;
    const int64_t page = static_cast<int64_t>(kTok) * (r.row_bytes + r.sub_bytes);
    uint8_t* data = static_cast<uint8_t*>(r.data);
    const int h0 = p.hkv * share / p.shares, h1 = p.hkv * (share + 1) / p.shares;
    if (r.row_bytes % 16 == 0 && r.sub_bytes % 4 == 0)
      move_rows<uint4>(p, data, page, 0, r.row_bytes, path, table, L - n, taken, h0, h1);
    else
      move_rows<uint32_t>(p, data, page, 0, r.row_bytes, path, table, L - n, taken, h0, h1);
    move_rows<uint32_t>(p, data, page, kTok * r.row_bytes, r.sub_bytes, path, table, L - n, taken, h0, h1);
  }
}

// ------------------------------------------------------------------ copies of pages

struct CopyParams {
  int caches, hkv, n;
  int64_t num_blocks;
  const int32_t* copies;
  uint32_t* status;
};

constexpr int kCopyThreads = 256;

// A CTA a page of a cache, all its heads: one run of 16 Hkv (row + sub) bytes.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p,
                                                            const __grid_constant__ Caches cs) {
  pdl_wait();
  pdl_allow_next();
  const int64_t items = static_cast<int64_t>(p.n) * p.caches;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = static_cast<int>(it / p.caches), c = static_cast<int>(it - static_cast<int64_t>(i) * p.caches);
    const int s = __ldg(p.copies + 2 * i), d = __ldg(p.copies + 2 * i + 1);
    if (s < 0 || d < 0) continue;
    if (s >= p.num_blocks || d >= p.num_blocks) {
      if (threadIdx.x == 0) flag_status(p.status, KVQ_DEV_BAD_BLOCK);
      continue;
    }
    const kvq_rows r = cs.c[c];
    const int64_t bytes = static_cast<int64_t>(kTok) * p.hkv * (r.row_bytes + r.sub_bytes);
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(r.data) + s * bytes);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(r.data) + d * bytes);
    const int64_t n = bytes / 16;
    for (int64_t x = threadIdx.x; x < n; x += 4 * kCopyThreads) {
      uint4 v[4];
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (x + y * kCopyThreads < n) v[y] = __ldcs(src + x + y * kCopyThreads);
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (x + y * kCopyThreads < n) dst[x + y * kCopyThreads] = v[y];
    }
  }
}

// ------------------------------------------------------------------ the pool

struct PoolParams {
  int32_t* pool;
  int num_blocks;
  int32_t* tables;
  int max_blocks;
  const int32_t* old_lens;
  const int32_t* new_lens;
  int B;
  uint32_t* status;
};

KVQ_DEVI int pages_of(int len) { return len / kTok + (len % kTok != 0); }
KVQ_DEVI bool length_ok(int len, int max_blocks) { return len >= 0 && pages_of(len) <= max_blocks; }

constexpr int kPoolThreads = 1024;

// Block-wide exclusive scan; warp_sum: a word for each warp.
template <int NT>
KVQ_DEVI int64_t block_scan(int64_t v, int64_t& total, int64_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t t = __shfl_up_sync(kAll, incl, off);
    if (lane >= off) incl += t;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int64_t base = 0;
  total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    const int64_t s = warp_sum[w];
    base += w < warp ? s : 0;
    total += s;
  }
  __syncthreads();
  return base + incl - v;
}

// Page after page of the pool's free ones, lowest first, to take(rank, page) for the ranks below
// `wanted`.  One CTA: a thread counts a word's bits and a scan gives the words' ranks, then a warp takes
// a word at a time, a page a lane.  (A thread took its words' pages one after the other before: a pool
// whose free pages lie together then has a few threads at work, and 64 pages with a look-up each took 25 us.)
struct Words {
  uint32_t bits[kPoolThreads];
  int rank[kPoolThreads];
  int64_t sum[kPoolThreads / 32];
};

template <typename F>
KVQ_DEVI void take_lowest(int32_t* pool, int num_blocks, int wanted, Words& s, F&& take) {
  uint32_t* bits = reinterpret_cast<uint32_t*>(pool + KVQ_POOL_HEADER + num_blocks);
  const int words = (num_blocks + 31) / 32, lane = threadIdx.x & 31;
  int base = 0;
  for (int w0 = 0; w0 < words && base < wanted; w0 += kPoolThreads) {
    const int at = w0 + static_cast<int>(threadIdx.x);
    const uint32_t w = at < words ? bits[at] : 0u;
    int64_t total;
    const int rank = base + static_cast<int>(block_scan<kPoolThreads>(__popc(w), total, s.sum));
    s.bits[threadIdx.x] = w;
    s.rank[threadIdx.x] = rank;
    __syncthreads();
    for (int y = threadIdx.x >> 5; y < min(kPoolThreads, words - w0) && s.rank[y] < wanted; y += kPoolThreads / 32) {
      const uint32_t of = s.bits[y];
      const int mine = s.rank[y] + __popc(of & ((1u << lane) - 1u)), page = 32 * (w0 + y) + lane;
      const bool taken = (of >> lane & 1u) && mine < wanted;
      const uint32_t gone = __ballot_sync(kAll, taken);
      if (lane == 0 && gone) bits[w0 + y] = of & ~gone;
      if (taken && page < num_blocks) take(mine, page);
    }
    base += static_cast<int>(total);
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kPoolThreads) alloc_kernel(const __grid_constant__ PoolParams p) {
  __shared__ int32_t off[kMaxTables + 1];
  __shared__ Words words;
  pdl_wait();
  pdl_allow_next();
  const int free_pages = p.pool[1];
  // what each sequence wants, and where its pages' ranks begin
  constexpr int kPer = kMaxTables / kPoolThreads;
  int need[kPer];
  int64_t mine = 0;
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    const int b = kPer * static_cast<int>(threadIdx.x) + y;
    need[y] = 0;
    if (b < p.B) {
      const int a = p.old_lens[b], z = p.new_lens[b];
      if (!length_ok(a, p.max_blocks) || !length_ok(z, p.max_blocks))
        flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
      else
        need[y] = max(0, pages_of(z) - pages_of(a));
    }
    mine += need[y];
  }
  int64_t total;
  int64_t at = block_scan<kPoolThreads>(mine, total, words.sum);
  if (total > free_pages) {
    if (threadIdx.x == 0) flag_status(p.status, KVQ_DEV_NO_PAGES);
    return;
  }
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    const int b = kPer * static_cast<int>(threadIdx.x) + y;
    if (b <= p.B) off[b] = static_cast<int32_t>(at);
    at += need[y];
  }
  if (threadIdx.x == 0) off[p.B] = static_cast<int32_t>(total);
  __syncthreads();
  take_lowest(p.pool, p.num_blocks, static_cast<int>(total), words, [&](int rank, int page) {
    int lo = 0, hi = p.B - 1;  // the last b with off[b] <= rank
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= rank)
        lo = mid;
      else
        hi = mid - 1;
    }
    p.pool[KVQ_POOL_HEADER + page] = 1;
    p.tables[static_cast<int64_t>(lo) * p.max_blocks + pages_of(__ldg(p.old_lens + lo)) + (rank - off[lo])] = page;
  });
  if (threadIdx.x == 0) p.pool[1] = free_pages - static_cast<int32_t>(total);
}

// One holder less; the last one's page is free.  False where nothing held it.
KVQ_DEVI bool let_go(int32_t* pool, int num_blocks, int page) {
  int32_t* refs = pool + KVQ_POOL_HEADER;
  const int32_t old = atomicSub(refs + page, 1);
  if (old <= 0) {
    atomicAdd(refs + page, 1);
    return false;
  }
  if (old == 1) {
    atomicOr(reinterpret_cast<uint32_t*>(refs + num_blocks) + page / 32, 1u << (page % 32));
    atomicAdd(pool + 1, 1);
  }
  return true;
}

constexpr int kRowThreads = 128;

__global__ void __launch_bounds__(kRowThreads) free_kernel(const __grid_constant__ PoolParams p) {
  pdl_wait();
  pdl_allow_next();
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int a = p.old_lens[b], z = p.new_lens[b];
    if (!length_ok(a, p.max_blocks) || !length_ok(z, p.max_blocks)) {
      if (threadIdx.x == 0) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
      continue;
    }
    int32_t* row = p.tables + static_cast<int64_t>(b) * p.max_blocks;
    for (int i = pages_of(z) + threadIdx.x; i < pages_of(a); i += kRowThreads) {
      const int page = row[i];
      row[i] = -1;
      if (page < 0 || page >= p.num_blocks || !let_go(p.pool, p.num_blocks, page))
        flag_status(p.status, KVQ_DEV_BAD_BLOCK);
    }
  }
}

struct ForkParams {
  int32_t* pool;
  int num_blocks;
  const int32_t* tables;
  const int32_t* lens;
  int num_src, max_blocks;
  const int32_t* parents;
  int num_out;
  int32_t* out_tables;
  int32_t* out_lens;
  int32_t* copies;
  uint32_t* status;
};

struct ForkRow {
  int src, len;  // -1: an empty row
  int last;      // the last page, where it is not full and can be copied; -1
  bool bad_len, bad_page;
};

// What row b goes on from.  A page that nothing holds stays so until every row is written, one that is
// held is held throughout, so every CTA sees the same.
KVQ_DEVI ForkRow fork_row(const ForkParams& p, int b) {
  ForkRow r = {-1, 0, -1, false, false};
  const int s = __ldg(p.parents + b);
  if (s < 0) return r;
  const int len = s < p.num_src ? __ldg(p.lens + s) : -1;
  if (!length_ok(len, p.max_blocks)) {
    r.bad_len = true;
    return r;
  }
  r.src = s;
  r.len = len;
  if (len % kTok) {
    const int page = __ldg(p.tables + static_cast<int64_t>(s) * p.max_blocks + len / kTok);
    if (page >= 0 && page < p.num_blocks && __ldcg(p.pool + KVQ_POOL_HEADER + page) > 0)
      r.last = page;
    else
      r.bad_page = true;
  }
  return r;
}

// One cluster; 64 beams of 100 pages: 7.1 us, 6 of 5: 6.7 (launch, four loads that wait on one another, a
// scan, the barrier).  Every CTA counts the pages wanted; the first takes them while the others write the
// rows; behind the cluster's barrier it changes what the others compare with: the count of free pages,
// and the counts of those taken.  (With a CTA a row and a counter in memory that the last one of them
// finds, the fence, the atomic and the last one's reads cost 2 us more than the barrier does.)
constexpr int kForkCtas = 8;

__global__ void __cluster_dims__(kForkCtas, 1, 1) __launch_bounds__(kPoolThreads)
    fork_kernel(const __grid_constant__ ForkParams p) {
  // for each page wanted its row (12 bits), the row's count of full pages (27) and the page to be copied (24)
  constexpr uint64_t kTaken = 1ull << 63;
  __shared__ uint64_t wants_s[kMaxTables];
  __shared__ Words words;
  static_assert(sizeof(wants_s) + sizeof(Words) <= 48 * 1024 && kMaxTables <= 4096, "packing, shared memory");
  pdl_wait();
  pdl_allow_next();
  constexpr int kPer = kMaxTables / kPoolThreads;
  const int cta = blockIdx.x;
  const int free_pages = __ldcg(p.pool + 1);
  uint32_t wants = 0;
  uint64_t want[kPer];
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    const int b = y * kPoolThreads + static_cast<int>(threadIdx.x);
    want[y] = 0;
    if (b < p.num_out) {
      const ForkRow r = fork_row(p, b);
      if (r.last >= 0) {
        wants |= 1u << y;
        want[y] = static_cast<uint64_t>(r.last) | static_cast<uint64_t>(r.len / kTok) << 24 | static_cast<uint64_t>(b) << 51;
      }
    }
  }
  // the pages' order is the rows'
  int64_t all = 0;
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    if (y * kPoolThreads >= p.num_out) break;
    int64_t total;
    const int64_t at = all + block_scan<kPoolThreads>(wants >> y & 1u, total, words.sum);
    all += total;
    if (cta == 0 && (wants >> y & 1u)) wants_s[at] = want[y];
  }
  const int total = static_cast<int>(all);
  const bool enough = total <= free_pages;
  if (enough && cta == 0) {
    __syncthreads();
    take_lowest(p.pool, p.num_blocks, total, words, [&](int rank, int page) {
      const uint64_t w = wants_s[rank];
      const int64_t b = static_cast<int64_t>(w >> 51), full = static_cast<int64_t>(w >> 24 & 0x7FFFFFFu);
      p.out_tables[b * p.max_blocks + full] = page;
      p.copies[2 * b] = static_cast<int32_t>(w & 0xFFFFFFu);
      p.copies[2 * b + 1] = page;
      wants_s[rank] = kTaken | static_cast<uint64_t>(page);  // (a rank is one thread's)
    });
  }
  if (enough && cta > 0) {
    // a warp a row
    const int lane = threadIdx.x & 31;
    for (int b = (cta - 1) + (kForkCtas - 1) * static_cast<int>(threadIdx.x >> 5); b < p.num_out;
         b += (kForkCtas - 1) * (kPoolThreads / 32)) {
      const ForkRow r = fork_row(p, b);
      if (lane == 0) {
        if (r.bad_len) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
        if (r.bad_page) flag_status(p.status, KVQ_DEV_BAD_BLOCK);
        p.out_lens[b] = r.len;
        if (r.last < 0) p.copies[2 * b] = p.copies[2 * b + 1] = -1;
      }
      int32_t* out = p.out_tables + static_cast<int64_t>(b) * p.max_blocks;
      const int full = r.len / kTok;
      const int32_t* from = p.tables + static_cast<int64_t>(r.src) * p.max_blocks;
      for (int i0 = lane; i0 < p.max_blocks; i0 += 32 * kPer) {  // four entries of a lane in flight
        int page[kPer];
        bool held[kPer];
#pragma unroll
        for (int y = 0; y < kPer; ++y) page[y] = i0 + 32 * y < full ? __ldg(from + i0 + 32 * y) : -1;
#pragma unroll
        for (int y = 0; y < kPer; ++y)
          held[y] = page[y] >= 0 && page[y] < p.num_blocks && __ldcg(p.pool + KVQ_POOL_HEADER + page[y]) > 0;
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
          const int i = i0 + 32 * y;
          if (i >= p.max_blocks || (i == full && r.last >= 0)) continue;  // (the new page's)
          if (held[y])
            atomicAdd(p.pool + KVQ_POOL_HEADER + page[y], 1);
          else if (i < full)
            flag_status(p.status, KVQ_DEV_BAD_BLOCK);
          out[i] = held[y] ? page[y] : -1;
        }
      }
    }
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (cta > 0) return;
  if (!enough) {
    if (threadIdx.x == 0) flag_status(p.status, KVQ_DEV_NO_PAGES);
    return;
  }
  if (threadIdx.x == 0) p.pool[1] = free_pages - total;
  for (int k = threadIdx.x; k < total; k += kPoolThreads)
    if (wants_s[k] & kTaken) p.pool[KVQ_POOL_HEADER + static_cast<int>(wants_s[k] & 0xFFFFFFu)] = 1;
}

__global__ void __launch_bounds__(256) init_kernel(int32_t* pool, const int num_blocks) {
  pdl_wait();
  pdl_allow_next();
  const int words = (num_blocks + 31) / 32, n = KVQ_POOL_HEADER + num_blocks + words;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
    int32_t v = 0;
    if (i == 1) v = num_blocks;
    if (i >= KVQ_POOL_HEADER + num_blocks) {
      const int left = num_blocks - 32 * (i - KVQ_POOL_HEADER - num_blocks);
      v = left >= 32 ? -1 : static_cast<int32_t>((1u << left) - 1u);
    }
    pool[i] = v;
  }
}

static int done(cudaError_t e) {
  if (e != cudaSuccess) return KVQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether na words at a and nb at b share one (none at a NULL).
static bool share(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x && y && na > 0 && nb > 0 && x < y + 4 * static_cast<uint64_t>(nb) && y < x + 4 * static_cast<uint64_t>(na);
}

static int check_rows(const kvq_rows* caches, int num_caches, int64_t num_blocks, int num_kv_heads, int block_size) {
  if (num_caches < 0 || num_blocks <= 0 || num_kv_heads <= 0) return KVQ_ERR_ARG;
  if (num_caches > 0 && !caches) return KVQ_ERR_NULL;
  if (block_size != kTok || num_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  for (int i = 0; i < num_caches; ++i) {
    const kvq_rows& r = caches[i];
    if (!r.data) return KVQ_ERR_NULL;
    if (r.row_bytes <= 0 || r.row_bytes > 512 || r.row_bytes % 4 || r.sub_bytes < 0 || r.sub_bytes > 512 || r.sub_bytes % 4)
      return KVQ_ERR_SHAPE;
    if (!aligned16(r.data)) return KVQ_ERR_ALIGN;
    if (num_blocks > INT64_MAX / (static_cast<int64_t>(kTok) * 1024 * num_kv_heads)) return KVQ_ERR_SHAPE;
  }
  return KVQ_OK;
}

// Whether a cache is listed twice: its rows would be moved twice.  Lists mostly rise; others are sorted.
constexpr int kMaxCommitCaches = 1024;
static bool listed_twice(const kvq_rows* caches, int n) {
  bool rises = true;
  for (int i = 1; i < n; ++i) rises = rises && std::less<const void*>()(caches[i - 1].data, caches[i].data);
  if (rises) return false;
  const void* at[kMaxCommitCaches];
  for (int i = 0; i < n; ++i) at[i] = caches[i].data;
  std::sort(at, at + n, std::less<const void*>());
  return std::adjacent_find(at, at + n) != at + n;
}

static int check_pool(const int32_t* pool, int64_t num_blocks, int max_blocks, int n) {
  if (num_blocks <= 0 || max_blocks <= 0 || n < 0) return KVQ_ERR_ARG;
  if (!pool) return KVQ_ERR_NULL;
  if (num_blocks > (1 << 24) || n > kMaxTables || max_blocks > INT32_MAX / kTok) return KVQ_ERR_UNSUPPORTED;
  return aligned4(pool) ? KVQ_OK : KVQ_ERR_ALIGN;
}

static int pool_call(void (*kernel)(PoolParams), bool rows, int32_t* pool, int64_t num_blocks, int32_t* tables,
                     int max_blocks, const int32_t* old_lens, const int32_t* new_lens, int B, uint32_t* status,
                     kvq_stream_t stream) {
  const int st = check_pool(pool, num_blocks, max_blocks, B);
  if (st != KVQ_OK) return st;
  if (B > 0 && (!tables || !old_lens || !new_lens)) return KVQ_ERR_NULL;
  if (!aligned4(tables) || !aligned4(old_lens) || !aligned4(new_lens)) return KVQ_ERR_ALIGN;
  if (B == 0) return KVQ_OK;
  PoolParams p = {pool, static_cast<int>(num_blocks), tables, max_blocks, old_lens, new_lens, B, status};
  return done(launch_pdl(kernel, dim3(rows ? B : 1), dim3(rows ? kRowThreads : kPoolThreads), 0,
                         reinterpret_cast<cudaStream_t>(stream), p));
}

}  // namespace pages
}  // namespace kvq

using namespace kvq;
using namespace kvq::pages;

extern "C" int kvq_tree_commit(const kvq_rows* caches, int num_caches, int64_t num_blocks,
                               int num_kv_heads, int block_size, const int32_t* cu_q_lens,
                               const int32_t* block_tables, int max_blocks_per_seq,
                               const int32_t* seq_lens, int num_seqs, const int32_t* accepted,
                               int max_path, const int32_t* num_accepted, int32_t* new_lens,
                               uint32_t* dev_status, kvq_stream_t stream) {
  const int st = check_rows(caches, num_caches, num_blocks, num_kv_heads, block_size);
  if (st != KVQ_OK) return st;
  if (num_seqs < 0 || max_path < 0 || max_blocks_per_seq <= 0) return KVQ_ERR_ARG;
  if (num_seqs > 0 && (!cu_q_lens || !block_tables || !seq_lens || !num_accepted || !new_lens || (max_path > 0 && !accepted)))
    return KVQ_ERR_NULL;
  if (num_seqs > 65535 || max_path > 4096 || max_blocks_per_seq > INT32_MAX / kTok || num_caches > kMaxCommitCaches)
    return KVQ_ERR_UNSUPPORTED;
  if (listed_twice(caches, num_caches)) return KVQ_ERR_ARG;
  if (!aligned4(cu_q_lens) || !aligned4(block_tables) || !aligned4(seq_lens) || !aligned4(accepted) ||
      !aligned4(num_accepted) || !aligned4(new_lens))
    return KVQ_ERR_ALIGN;
  // (written while other warps, and later launches, still read their sequence's lengths and path)
  const int64_t B = num_seqs;
  if (share(new_lens, B, seq_lens, B) || share(new_lens, B, num_accepted, B) || share(new_lens, B, cu_q_lens, B + 1) ||
      share(new_lens, B, accepted, B * max_path) || share(new_lens, B, block_tables, B * max_blocks_per_seq))
    return KVQ_ERR_ARG;
  if (num_seqs == 0) return KVQ_OK;
  const int sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  CommitParams p = {0, num_seqs, num_kv_heads, max_blocks_per_seq, max_path, 1, 1, num_blocks, cu_q_lens, block_tables,
                    seq_lens, accepted, num_accepted, new_lens, dev_status};
  int at = 0;
  do {
    Caches cs = {};
    p.caches = num_caches - at < kMaxRowsCaches ? num_caches - at : kMaxRowsCaches;
    for (int i = 0; i < p.caches; ++i) cs.c[i] = caches[at + i];
    const int64_t each = static_cast<int64_t>(num_seqs) * (p.caches > 0 ? p.caches : 1), most = static_cast<int64_t>(sms) * 32 / each;
    p.shares = most < 1 ? 1 : most < num_kv_heads ? static_cast<int>(most) : num_kv_heads;
    const int64_t warps = each * p.shares;
    const int64_t ctas = (warps + 3) / 4, cap = static_cast<int64_t>(sms) * 64;
    const int r = done(launch_pdl(commit_kernel, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(128), 0,
                                  reinterpret_cast<cudaStream_t>(stream), p, cs));
    if (r != KVQ_OK) return r;
    at += p.caches;
    p.first = 0;
  } while (at < num_caches);
  return KVQ_OK;
}

extern "C" int kvq_copy_pages(const kvq_rows* caches, int num_caches, int64_t num_blocks,
                              int num_kv_heads, int block_size, const int32_t* copies,
                              int num_copies, uint32_t* dev_status, kvq_stream_t stream) {
  const int st = check_rows(caches, num_caches, num_blocks, num_kv_heads, block_size);
  if (st != KVQ_OK) return st;
  if (num_copies < 0) return KVQ_ERR_ARG;
  if (num_copies > 0 && !copies) return KVQ_ERR_NULL;
  if (num_copies > (1 << 20)) return KVQ_ERR_UNSUPPORTED;
  if (!aligned4(copies)) return KVQ_ERR_ALIGN;
  const int sms = num_copies > 0 && num_caches > 0 ? device_sm_count() : 1;
  if (sms <= 0) return KVQ_ERR_CUDA;
  for (int at = 0; at < num_caches && num_copies > 0; at += kMaxRowsCaches) {
    Caches cs = {};
    CopyParams p = {num_caches - at < kMaxRowsCaches ? num_caches - at : kMaxRowsCaches, num_kv_heads, num_copies,
                    num_blocks, copies, dev_status};
    for (int i = 0; i < p.caches; ++i) cs.c[i] = caches[at + i];
    const int64_t items = static_cast<int64_t>(num_copies) * p.caches, cap = static_cast<int64_t>(sms) * 64;
    const int r = done(launch_pdl(copy_kernel, dim3(static_cast<unsigned>(items < cap ? items : cap)), dim3(kCopyThreads), 0,
                                  reinterpret_cast<cudaStream_t>(stream), p, cs));
    if (r != KVQ_OK) return r;
  }
  return KVQ_OK;
}

extern "C" int kvq_pages_init(int32_t* pool, int64_t num_blocks, kvq_stream_t stream) {
  const int st = check_pool(pool, num_blocks, 1, 0);
  if (st != KVQ_OK) return st;
  const int64_t ctas = (KVQ_POOL_WORDS(num_blocks) + 255) / 256;
  return done(launch_pdl(init_kernel, dim3(static_cast<unsigned>(ctas < 1024 ? ctas : 1024)), dim3(256), 0,
                         reinterpret_cast<cudaStream_t>(stream), pool, static_cast<int>(num_blocks)));
}

extern "C" int kvq_pages_alloc(int32_t* pool, int64_t num_blocks, int32_t* block_tables,
                               int max_blocks_per_seq, const int32_t* old_lens,
                               const int32_t* new_lens, int num_seqs, uint32_t* dev_status,
                               kvq_stream_t stream) {
  return pool_call(alloc_kernel, false, pool, num_blocks, block_tables, max_blocks_per_seq, old_lens, new_lens, num_seqs,
                   dev_status, stream);
}

extern "C" int kvq_pages_free(int32_t* pool, int64_t num_blocks, int32_t* block_tables,
                              int max_blocks_per_seq, const int32_t* old_lens,
                              const int32_t* new_lens, int num_seqs, uint32_t* dev_status,
                              kvq_stream_t stream) {
  return pool_call(free_kernel, true, pool, num_blocks, block_tables, max_blocks_per_seq, old_lens, new_lens, num_seqs,
                   dev_status, stream);
}

extern "C" int kvq_pages_fork(int32_t* pool, int64_t num_blocks, const int32_t* tables,
                              const int32_t* lens, int num_src, int max_blocks_per_seq,
                              const int32_t* parents, int num_out, int32_t* out_tables,
                              int32_t* out_lens, int32_t* copies, uint32_t* dev_status,
                              kvq_stream_t stream) {
  int st = check_pool(pool, num_blocks, max_blocks_per_seq, num_out);
  if (st == KVQ_OK) st = check_pool(pool, num_blocks, max_blocks_per_seq, num_src);
  if (st != KVQ_OK) return st;
  if ((num_src > 0 && (!tables || !lens)) || (num_out > 0 && (!parents || !out_tables || !out_lens || !copies)))
    return KVQ_ERR_NULL;
  if (!aligned4(tables) || !aligned4(lens) || !aligned4(parents) || !aligned4(out_tables) || !aligned4(out_lens) ||
      !aligned4(copies))
    return KVQ_ERR_ALIGN;
  // (rows are written while others are still read, from the pool too)
  const int64_t columns = max_blocks_per_seq, words = KVQ_POOL_WORDS(num_blocks);
  const struct {
    const int32_t* p;
    int64_t n;
  } in[4] = {{tables, num_src * columns}, {lens, num_src}, {parents, num_out}, {pool, words}},
    out[3] = {{out_tables, num_out * columns}, {out_lens, num_out}, {copies, 2 * static_cast<int64_t>(num_out)}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& x : in)
      if (share(out[i].p, out[i].n, x.p, x.n)) return KVQ_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (share(out[i].p, out[i].n, out[j].p, out[j].n)) return KVQ_ERR_ARG;
  }
  if (num_out == 0) return KVQ_OK;
  ForkParams p = {pool, static_cast<int>(num_blocks), tables, lens, num_src, max_blocks_per_seq, parents, num_out,
                  out_tables, out_lens, copies, dev_status};
  return done(launch_pdl(fork_kernel, dim3(kForkCtas), dim3(kPoolThreads), 0,
                         reinterpret_cast<cudaStream_t>(stream), p));
}
