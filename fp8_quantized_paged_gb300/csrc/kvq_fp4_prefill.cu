// kvq_fp4_prefill.cu -- entry point and launch of the 4-bit cache's prefill.
#include "kvq_fp4_prefill.cuh"
#include "kvq_fp4_host.h"

namespace kvq {
namespace fp4 {

// Least key blocks of a share where SMs would idle, by the tiles of an item: the merge of 256 rows
// takes about 15 us, of a few rows 3.  One sequence, 8 KV heads, 4 queries over 1024 tokens (8
// blocks): shares of 2 blocks 11.4 us, of 4 14.2, none 17.6; over 4096 13.5, 14.6, 31.2.  64 queries
// (two tiles) over 1024: shares of 2 32.4, of 4 35.4, none 27.4; over 2048 39.0, 35.9, 41.4.
constexpr int kMinShare[2] = {2, 5};
// And where they would after the last whole wave.  Ragged chunks under a window (10 blocks, 220
// items): whole 41.5 us, the rest in two 47.2.  2048 queries over 32768 tokens (256 blocks, 256
// items): whole 919 us, the rest in four 858.  In between, one sequence and 8 KV heads, whole / with
// a least share of 12 / 24 blocks: 160 items of 32 blocks 114 / 111 / 114 us, of 48 171 / 142 / 171, of
// 64 227 / 169 / 192, of 128 453 / 296 / 312; 200 items of 48 180 / 154 / 181, of 96 349 / 267 / 267; 256
// items of 64 242 / 265 / 241, of 96 354 / 364 / 379, of 128 467 / 462 / 463.
constexpr int kMinTail = 24;
constexpr int kOverhead = 6;  // a share's start, end and merge, in blocks

template <int DH>
static int launch_prefill(const PreParams& p, int64_t ctas, cudaStream_t s) {
  static DeviceOnce once;
  if (!once.run(current_device(), [] {
        return cudaFuncSetAttribute(prefill_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    PreSmem<DH>::total) == cudaSuccess;
      }))
    return KVQ_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(ctas)), block(kPreThreads);
  if (launch_pdl(prefill_kernel<DH>, grid, block, PreSmem<DH>::total, s, p) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace fp4
}  // namespace kvq

using namespace kvq;

extern "C" int kvq_fp4_prefill_attn(const void* q, const int32_t* cu_q_lens, int64_t num_q_tokens,
                                    int max_q_len, const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, int max_blocks_per_seq,
                                    const int32_t* seq_lens, int num_seqs, int num_q_heads,
                                    int num_kv_heads, int head_dim, int64_t num_blocks,
                                    int block_size, const float* k_scale, int k_scale_len,
                                    const float* v_scale, int v_scale_len, int scale_granularity,
                                    int sliding_window, int num_sinks, void* workspace,
                                    size_t workspace_bytes, void* out, uint32_t* dev_status,
                                    kvq_stream_t stream) {
  const int st = fp4::check_attn(num_q_tokens != 0, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens,
                                 num_seqs, num_q_heads, num_kv_heads, head_dim, num_blocks,
                                 block_size, k_scale, k_scale_len, v_scale, v_scale_len,
                                 scale_granularity, sliding_window, num_sinks, workspace, out);
  if (st != KVQ_OK) return st;
  if (!cu_q_lens) return KVQ_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(cu_q_lens) & 3u) return KVQ_ERR_ALIGN;
  if (num_q_tokens < 0 || max_q_len < 0) return KVQ_ERR_ARG;
  if (num_seqs > 65535) return KVQ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_blocks_per_seq) * fp4::kTok >= (int64_t(1) << 30))
    return KVQ_ERR_UNSUPPORTED;
  if (num_q_tokens > (int64_t(1) << 30)) return KVQ_ERR_UNSUPPORTED;
  const int G = num_q_heads / num_kv_heads, TQ = fp4::kRows / G;
  const int64_t tiles = (std::min<int64_t>(max_q_len, num_q_tokens) + TQ - 1) / TQ;
  // Two tiles a CTA share each converted block.
  const int tpc = tiles > 1 ? fp4::kTiles : 1;
  // (with a bound of 0 there are no tiles: the CTAs only look for chunks past it)
  const int64_t groups = std::max<int64_t>(1, (tiles + tpc - 1) / tpc), items = groups * num_kv_heads * num_seqs;
  if (items >= (int64_t(1) << 31) - 65536) return KVQ_ERR_UNSUPPORTED;  // (the grid)
  if (num_q_tokens == 0) return KVQ_OK;
  const int sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const fp4::PreWs wl = fp4::pre_ws(head_dim, sms);
  if (workspace_bytes < wl.total) return KVQ_ERR_WORKSPACE;

  fp4::PreParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.cu_q = cu_q_lens;
  p.kc = static_cast<const uint8_t*>(k_cache);
  p.vc = static_cast<const uint8_t*>(v_cache);
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.max_blocks = max_blocks_per_seq;
  p.B = num_seqs;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.G = G;
  p.num_blocks = num_blocks;
  p.total_q = num_q_tokens;
  p.window = sliding_window;
  p.sinks = num_sinks;
  p.tiles = static_cast<int>(tiles);
  p.tpc = tpc;
  p.groups = static_cast<int>(groups);
  int64_t pages = max_blocks_per_seq;
  if (sliding_window > 0)
    pages = std::min<int64_t>(pages, (static_cast<int64_t>(sliding_window) + static_cast<int64_t>(tpc) * TQ) / fp4::kTok +
                                         2 + (static_cast<int64_t>(num_sinks) + fp4::kTok - 1) / fp4::kTok);
  const int64_t blocks = (pages + fp4::kBlkPages - 1) / fp4::kBlkPages;
  // Items are whole while they fill waves of a CTA per SM; the rest, where it would leave SMs
  // idle, shares its keys out.  A single, partial wave takes what SMs there are; after whole
  // waves the split is the one that ends first (a split's rounds times a share's length).
  p.whole = items;
  p.ns = 1;
  p.min_share = fp4::kMinTail;
  const int64_t rest = items % sms;
  if (items < sms) {
    p.ns = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms / items, blocks / fp4::kMinShare[tpc - 1])));
    p.min_share = fp4::kMinShare[tpc - 1];
  } else {
    double best = static_cast<double>(blocks + fp4::kOverhead);
    for (int64_t n = 2; rest > 0 && rest * n <= static_cast<int64_t>(fp4::kShares) * sms && n * fp4::kMinTail <= blocks; ++n) {
      const double t = static_cast<double>((rest * n + sms - 1) / sms) * (static_cast<double>(blocks) / n + fp4::kOverhead);
      if (t < best) {
        best = t;
        p.ns = static_cast<int>(n);
      }
    }
  }
  if (p.ns > 1) p.whole = items - rest;
  const int64_t ctas = p.whole + (items - p.whole) * p.ns;
  p.ks = k_scale;
  p.vs = v_scale;
  p.per_head = scale_granularity == KVQ_SCALE_PER_HEAD;
  p.logit_scale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(head_dim)));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.ws_cnt = reinterpret_cast<uint32_t*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(ws + wl.ml);
  p.ws_o = reinterpret_cast<float*>(ws + wl.o);
  p.out = static_cast<uint16_t*>(out);
  p.status = dev_status;
#ifdef KVQ_TEST_HOOKS
  p.withhold = test_withheld();
#else
  p.withhold = -1;
#endif
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return head_dim == 128 ? fp4::launch_prefill<128>(p, ctas, s) : fp4::launch_prefill<64>(p, ctas, s);
}
