// kvq_tree.cu -- entry point and launches of the attention over drafted trees.
#include <atomic>

#include "kvq_tree.cuh"

namespace kvq {
namespace tree {

template <int FMT, int DH, bool TS>
static int launch_tree(const TreeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, int sms, cudaStream_t s) {
  using SM = TreeSmem<FMT, DH, TS>;
  static DeviceOnce once;
  if (!once.run(current_device(), [] {
        return cudaFuncSetAttribute(tree_kernel<FMT, DH, TS>, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::total) ==
               cudaSuccess;
      }))
    return KVQ_ERR_CUDA;
  if (launch_pdl(tree_kernel<FMT, DH, TS>, dim3(ctas), dim3(kTreeThreads), SM::total, s, p, tk, tv) != cudaSuccess)
    return KVQ_ERR_CUDA;
  if (launch_pdl(merge_kernel<DH>, dim3(sms * kMergeCtas), dim3(kMergeThreads), 0, s, p, ctas) != cudaSuccess) return KVQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

template <int FMT, bool TS>
static int launch_tree_dh(const TreeParams& p, int dh, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, int sms,
                          cudaStream_t s) {
  return dh == 128 ? launch_tree<FMT, 128, TS>(p, tk, tv, ctas, sms, s) : launch_tree<FMT, 64, TS>(p, tk, tv, ctas, sms, s);
}

static int ctas_of(int sms) { return std::min(sms, kMaxCtas); }

}  // namespace tree
}  // namespace kvq

using namespace kvq;

#ifdef KVQ_TEST_HOOKS
static std::atomic<int> g_late{-1};
extern "C" __attribute__((visibility("default"))) void kvq_test_late_warp(int warp) { g_late.store(warp); }
#endif

extern "C" size_t kvq_tree_workspace_size(int num_q_heads, int num_kv_heads, int head_dim, int num_sms) {
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > 8) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return 0;
  return tree::tree_ws(head_dim, tree::ctas_of(num_sms)).total;
}

extern "C" int kvq_tree_attn(const void* q, const int32_t* cu_q_lens, int64_t num_q_tokens,
                             const int32_t* parents, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, int max_blocks_per_seq,
                             const int32_t* seq_lens, int num_seqs, int num_q_heads,
                             int num_kv_heads, int head_dim, int64_t num_blocks, int block_size,
                             const float* q_scale, int q_scale_len, const float* k_scale,
                             int k_scale_len, const float* v_scale, int v_scale_len,
                             int scale_granularity, int fmt, int sliding_window, unsigned flags,
                             void* workspace, size_t workspace_bytes, void* out,
                             uint32_t* dev_status, kvq_stream_t stream) {
  if (fmt < KVQ_FMT_BF16 || fmt > KVQ_FMT_E5M2) return KVQ_ERR_ARG;
  if (scale_granularity < KVQ_SCALE_PER_TENSOR || scale_granularity > KVQ_SCALE_PER_TOKEN_HEAD) return KVQ_ERR_ARG;
  if (flags & ~KVQ_Q_FP8) return KVQ_ERR_ARG;
  const bool q_fp8 = (flags & KVQ_Q_FP8) != 0;
  if (q_fp8 && fmt == KVQ_FMT_BF16) return KVQ_ERR_UNSUPPORTED;
  if (q_fp8 && !q_scale) return KVQ_ERR_NULL;
  if (num_q_tokens < 0 || num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || sliding_window < 0)
    return KVQ_ERR_ARG;
  if (!cu_q_lens || !k_cache || !v_cache || !block_tables || !seq_lens || !workspace || (num_q_tokens > 0 && (!q || !out)))
    return KVQ_ERR_NULL;
  if (head_dim != 64 && head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (block_size != kBS) return KVQ_ERR_UNSUPPORTED;
  if (num_q_heads % num_kv_heads) return KVQ_ERR_SHAPE;
  const int G = num_q_heads / num_kv_heads;
  if (G > 8 || num_kv_heads > 256 || num_seqs > 4096) return KVQ_ERR_UNSUPPORTED;
  if (num_q_tokens > (int64_t(1) << 30) || static_cast<int64_t>(max_blocks_per_seq) * kBS >= (int64_t(1) << 30))
    return KVQ_ERR_UNSUPPORTED;
  const int64_t tiles = num_q_tokens * G <= tree::kRows ? 1 : 16;
  // (the sum of all costs: a tile has at most max_blocks_per_seq / 4 + 1 blocks)
  if (num_seqs * tiles * num_kv_heads * (max_blocks_per_seq / 4 + 2 + tree::kSegCost) >= (int64_t(1) << 31))
    return KVQ_ERR_UNSUPPORTED;
  if (num_blocks > ((int64_t(1) << 31) - 1) / (static_cast<int64_t>(num_kv_heads) * kBS)) return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(seq_lens) |
        reinterpret_cast<uintptr_t>(cu_q_lens) | reinterpret_cast<uintptr_t>(parents)) & 3u))
    return KVQ_ERR_ALIGN;
  const bool ts = scale_granularity == KVQ_SCALE_PER_TOKEN_HEAD && fmt != KVQ_FMT_BF16;
  if (fmt != KVQ_FMT_BF16) {
    if (!k_scale || !v_scale) return KVQ_ERR_NULL;
    const int64_t want = ts ? num_blocks * num_kv_heads * kBS : scale_granularity == KVQ_SCALE_PER_HEAD ? num_kv_heads : 1;
    if (k_scale_len != want || v_scale_len != want) return KVQ_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & (ts ? 15u : 3u)) return KVQ_ERR_ALIGN;
  }
  if (q_scale) {
    const bool ok = scale_granularity == KVQ_SCALE_PER_TOKEN_HEAD
                        ? q_scale_len == 1 || q_scale_len == num_q_heads
                        : q_scale_len == (scale_granularity == KVQ_SCALE_PER_HEAD ? num_q_heads : 1);
    if (!ok) return KVQ_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(q_scale) & 3u) return KVQ_ERR_ALIGN;
  }
  if (num_q_tokens == 0) return KVQ_OK;
  const int sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const int ctas = tree::ctas_of(sms);
  const tree::TreeWs wl = tree::tree_ws(head_dim, ctas);
  if (workspace_bytes < wl.total) return KVQ_ERR_WORKSPACE;

  tree::TreeParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.cu_q = cu_q_lens;
  p.parents = parents;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.vc = static_cast<const uint8_t*>(v_cache);
  p.max_blocks = max_blocks_per_seq;
  p.B = num_seqs;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.G = G;
  p.num_blocks = num_blocks;
  p.total_q = num_q_tokens;
  p.window = sliding_window;
  p.qs = q_fp8 ? q_scale : nullptr;
  p.q_per_head = q_scale && q_scale_len == num_q_heads && num_q_heads > 1;
  p.ks = fmt == KVQ_FMT_BF16 ? nullptr : k_scale;
  p.vs = fmt == KVQ_FMT_BF16 ? nullptr : v_scale;
  p.per_head = scale_granularity == KVQ_SCALE_PER_HEAD;
  p.logit_scale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(head_dim)));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.ws_rec = reinterpret_cast<int4*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(ws + wl.ml);
  p.ws_o = reinterpret_cast<float*>(ws + wl.o);
  p.out = static_cast<uint16_t*>(out);
  p.status = dev_status;
#ifdef KVQ_TEST_HOOKS
  p.withhold = test_withheld();
  p.late = g_late.load();
#else
  p.withhold = p.late = -1;
#endif
  const uint64_t rows = static_cast<uint64_t>(num_blocks) * num_kv_heads * kBS;
  CUtensorMap tk, tv;
  if (!make_cache_map(&tk, k_cache, fmt, head_dim, rows) || !make_cache_map(&tv, v_cache, fmt, head_dim, rows))
    return KVQ_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (fmt == KVQ_FMT_BF16) return tree::launch_tree_dh<KVQ_FMT_BF16, false>(p, head_dim, tk, tv, ctas, sms, s);
  if (fmt == KVQ_FMT_E4M3)
    return ts ? tree::launch_tree_dh<KVQ_FMT_E4M3, true>(p, head_dim, tk, tv, ctas, sms, s)
              : tree::launch_tree_dh<KVQ_FMT_E4M3, false>(p, head_dim, tk, tv, ctas, sms, s);
  return ts ? tree::launch_tree_dh<KVQ_FMT_E5M2, true>(p, head_dim, tk, tv, ctas, sms, s)
            : tree::launch_tree_dh<KVQ_FMT_E5M2, false>(p, head_dim, tk, tv, ctas, sms, s);
}
