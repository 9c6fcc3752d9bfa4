// kvq_fp4_decode.cu -- entry point and launch of the 4-bit cache's decode.
#include "kvq_fp4_decode.cuh"
#include "kvq_fp4_host.h"
#include "kvq_fp4_prefill.cuh"

namespace kvq {
namespace fp4 {

// Segments of at most this many pages, with an SM each, go whole to one CTA, without a plan.
constexpr int kSegPages = 128;
// Most pieces of a segment that units of several heads may leave.  One sequence of 32768 tokens,
// 8 KV heads: one head a unit (19 pieces) 19.1 us, two 24.5, eight (152 pieces) 70.8.
constexpr int kMaxPieces = 10;
constexpr int kMaxSmem = 227 * 1024 - 1024;  // the static part and the system's

template <int DH>
static int launch_decode(DecParams p, bool fix, int grid, cudaStream_t s) {
  static DeviceOnce once;
  if (!once.run(current_device(), [] {
        auto configure = [](auto kernel) {
          return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kMaxSmem) == cudaSuccess &&
                 cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                      cudaSharedmemCarveoutMaxShared) == cudaSuccess;
        };
        return configure(decode_kernel<DH, true>) && configure(decode_kernel<DH, false>);
      }))
    return KVQ_ERR_CUDA;
  const int rings = kDecWarps / p.HG;
  const int fixed = dec_smem<DH>(0, p.HG, p.G, p.B, fix).total + 32;  // (all but the slots, and their rounding)
  const int slot = 2 * p.HG * Page<DH>::kBytes + 24;
  p.depth = std::min(kMaxDepth, (kMaxSmem - fixed) / slot / rings);
  if (p.depth < kStepUnits) return KVQ_ERR_UNSUPPORTED;  // (a step holds so many slots; not reached)
  const size_t smem = dec_smem<DH>(p.depth * rings, p.HG, p.G, p.B, fix).total;
  const cudaError_t e =
      fix ? launch_pdl(decode_kernel<DH, true>, dim3(grid), dim3(kDecThreads), smem, s, p)
          : launch_pdl(decode_kernel<DH, false>, dim3(grid), dim3(kDecThreads), smem, s, p);
  if (e != cudaSuccess) return KVQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace fp4
}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_fp4_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                         int head_dim, int num_sms) {
  if (num_seqs <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads)
    return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return 0;
  return std::max(fp4::dec_ws(num_seqs, num_q_heads / num_kv_heads, num_kv_heads, head_dim,
                              num_sms).total,
                  fp4::pre_ws(head_dim, num_sms).total);
}

extern "C" int kvq_fp4_decode_attn(const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int max_blocks_per_seq,
                                   const int32_t* seq_lens, int num_seqs, int num_q_heads,
                                   int num_kv_heads, int head_dim, int64_t num_blocks,
                                   int block_size, const float* k_scale, int k_scale_len,
                                   const float* v_scale, int v_scale_len, int scale_granularity,
                                   int sliding_window, int num_sinks, void* workspace,
                                   size_t workspace_bytes, void* out, uint32_t* dev_status,
                                   kvq_stream_t stream) {
  const int st = fp4::check_attn(true, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens,
                                 num_seqs, num_q_heads, num_kv_heads, head_dim, num_blocks,
                                 block_size, k_scale, k_scale_len, v_scale, v_scale_len,
                                 scale_granularity, sliding_window, num_sinks, workspace, out);
  if (st != KVQ_OK) return st;
  if (num_seqs > kMaxSeqs || num_seqs * num_kv_heads > kMaxSegments) return KVQ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_seqs) * (static_cast<int64_t>(max_blocks_per_seq) + fp4::kPc) *
          num_kv_heads >= (int64_t(1) << 31) ||
      static_cast<int64_t>(max_blocks_per_seq) * fp4::kTok >= (int64_t(1) << 31))
    return KVQ_ERR_UNSUPPORTED;
  const int G = num_q_heads / num_kv_heads, sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const int P = sms;
  const fp4::DecWs wl = fp4::dec_ws(num_seqs, G, num_kv_heads, head_dim, P);
  if (workspace_bytes < wl.total) return KVQ_ERR_WORKSPACE;

  // the most pages that one segment can have, from what the host knows
  int64_t pages = max_blocks_per_seq;
  if (sliding_window > 0)
    pages = std::min<int64_t>(pages, (static_cast<int64_t>(sliding_window) + fp4::kTok - 1) / fp4::kTok + 1 +
                                         (static_cast<int64_t>(num_sinks) + fp4::kTok - 1) / fp4::kTok);
  // One sequence, or short ones with an SM for each KV head: a number of CTAs for each, one head
  // a unit.  Else the units are split at equal cost, with as many heads a unit as leave a segment
  // kMaxPieces pieces or fewer (32 sequences of 2049 tokens / 128 of mixed lengths: one head a unit
  // 38.3 / 119 us, two 32.0 / 79.1, four 31.2 / 66.9, eight 30.7 / 62.9).
  const int segs = num_seqs * num_kv_heads;
  const bool fix = segs <= P && (num_seqs == 1 || pages <= fp4::kSegPages);
  int HG = 1, cps = 1;
  if (fix) {
    if (num_seqs == 1)
      cps = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(P / segs, pages / fp4::kMinUnits)));
  } else {
    for (int h = fp4::kMaxHeads; h > 1; h /= 2)
      if (num_kv_heads % h == 0 && segs / h * fp4::kMaxPieces >= P) {
        HG = h;
        break;
      }
  }
  const int64_t units = static_cast<int64_t>(segs / HG) * pages;
  const int64_t ctas = fix ? static_cast<int64_t>(segs) * cps
                           : std::min<int64_t>(P, (units * HG + fp4::kDecWarps - 1) / fp4::kDecWarps);

  fp4::DecParams p;
  p.q = static_cast<const uint16_t*>(q);
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
  p.window = sliding_window;
  p.sinks = num_sinks;
  p.ks = k_scale;
  p.vs = v_scale;
  p.per_head = scale_granularity == KVQ_SCALE_PER_HEAD;
  p.logit_scale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(head_dim)));
  p.HG = HG;
  p.NG = num_kv_heads / HG;
  p.P = P;
  p.cps = cps;
  p.depth = 0;
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
  const int grid = static_cast<int>(ctas);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return head_dim == 128 ? fp4::launch_decode<128>(p, fix, grid, s)
                         : fp4::launch_decode<64>(p, fix, grid, s);
}
