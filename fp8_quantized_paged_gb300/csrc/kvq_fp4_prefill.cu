// kvq_fp4_prefill.cu -- prefill attention over the microscaled 4-bit cache: a
// plain kernel.
//
// One CTA per (query token, KV head).  Its four warps take the visible pages
// in turn; a page's 16 tokens go two lanes a token for the logits, and the
// head dims are spread over the lanes for the weighted sum of V.  Online
// softmax in binary32, the warps' states merged at the end.
#include <algorithm>
#include <cmath>

#include "kvq_fp4.cuh"
#include "kvq_fp4_host.h"

namespace kvq {
namespace fp4 {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMaxG = 8;  // query heads per KV head
constexpr int kWarps = 4;

struct AttnParams {
  const uint16_t* q;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* cu_q;  // NULL: one query per sequence
  int max_blocks, B, Hq, Hkv, G;
  int64_t num_blocks, total_q;
  int max_q;
  int window, sinks;
  const float* ks;
  const float* vs;
  int per_head;
  float logit_scale;  // log2(e) / sqrt(dh)
  uint16_t* out;
  uint32_t* status;
};

template <int DH>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(const AttnParams p) {
  using P = Page<DH>;
  constexpr int D = DH / 32;  // dims of V a lane sums
  __shared__ float qs[kMaxG][DH];
  __shared__ float sm[kWarps][kMaxG], sl[kWarps][kMaxG];
  __shared__ float so[kWarps][kMaxG][DH];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_allow_next();
  pdl_wait();
  const int g = blockIdx.y, b = blockIdx.z, j = blockIdx.x;
  const int q0 = p.cu_q ? __ldg(p.cu_q + b) : b;
  int n = p.cu_q ? __ldg(p.cu_q + b + 1) - q0 : 1;
  if (j == 0 && g == 0 && tid == 0 && n > p.max_q) flag_status(p.status, KVQ_DEV_BAD_QLEN);
  if (j >= n || q0 < 0 || q0 + j >= p.total_q) return;
  const int64_t orow = (static_cast<int64_t>(q0 + j) * p.Hq + g * p.G) * DH;
  int L = __ldg(p.seq_lens + b);
  if (L < (p.cu_q ? n : 0) || L > p.max_blocks * kTok) {
    if (j == 0 && g == 0 && tid == 0) flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
    L = n = 0;
  }
  L = L > 0 ? L - n + j + 1 : 0;  // what this query sees ends with its own token
  const Visible vis = visible(p.window, p.sinks, L);
  for (int i = tid; i < p.G * DH; i += kWarps * 32)
    qs[i / DH][i % DH] = __uint_as_float(static_cast<uint32_t>(p.q[orow + i]) << 16);
  __syncthreads();
  const float ls = __ldg(p.ks + (p.per_head ? g : 0)) * p.logit_scale;
  float m[kMaxG], l[kMaxG], o[kMaxG][D];
  for (int h = 0; h < kMaxG; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    for (int d = 0; d < D; ++d) o[h][d] = 0.f;
  }
  for (int i = warp; i < vis.count; i += kWarps) {
    const int col = i < vis.sink ? i : vis.first + i - vis.sink;
    const int blk = __ldg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks + col);
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) flag_status(p.status, KVQ_DEV_BAD_BLOCK);
      continue;
    }
    const int64_t page = (static_cast<int64_t>(blk) * p.Hkv + g) * P::kBytes;
    const int tok = lane & 15, half = lane >> 4;
    const int t = col * kTok + tok;
    const bool seen = t < L && (t >= vis.lo || t < p.sinks);
    float x[kMaxG];
    for (int h = 0; h < kMaxG; ++h) x[h] = 0.f;
    for (int c = half * (P::kScales / 2); c < (half + 1) * (P::kScales / 2); ++c) {
      const float sb = e4m3_to_f32(__ldg(p.kc + page + P::kScaleOff + tok * P::kScales + c));
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.kc + page + tok * P::kRow + c * 8));
      for (int e = 0; e < 2; ++e) {
        uint32_t f[4];
        e2m1x8_to_f16x2x4(e ? w.y : w.x, f);
        for (int y = 0; y < 4; ++y)
          for (int h = 0; h < p.G; ++h) {
            const float* qv = &qs[h][c * 16 + e * 8 + y * 2];
            x[h] += qv[0] * (f16lo_to_f32(f[y]) * sb) + qv[1] * (f16hi_to_f32(f[y]) * sb);
          }
      }
    }
    for (int h = 0; h < p.G; ++h) {
      float v = (x[h] + __shfl_xor_sync(kAll, x[h], 16)) * ls;
      if (!seen) v = -INFINITY;
      float mx = v;
      for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, off));
      const float nm = fmaxf(m[h], mx);
      const float a = nm == -INFINITY ? 1.f : exp2f(m[h] - nm);
      const float pr = v == -INFINITY ? 0.f : exp2f(v - nm);
      m[h] = nm;
      l[h] = l[h] * a + (half == 0 ? pr : 0.f);
      for (int d = 0; d < D; ++d) o[h][d] *= a;
      x[h] = pr;
    }
    for (int r = 0; r < kTok; ++r) {
      const int tt = col * kTok + r;
      if (!(tt < L && (tt >= vis.lo || tt < p.sinks))) continue;  // the same on every lane
      const float sb = e4m3_to_f32(__ldg(p.vc + page + P::kScaleOff + r * P::kScales + lane * D / 16));
      uint32_t w = 0;
      for (int d = 0; d < D / 2; ++d)
        w |= static_cast<uint32_t>(__ldg(p.vc + page + r * P::kRow + lane * (D / 2) + d)) << (8 * d);
      uint32_t f[4];
      e2m1x8_to_f16x2x4(w, f);
      for (int h = 0; h < p.G; ++h) {
        const float pr = __shfl_sync(kAll, x[h], r);
        for (int d = 0; d < D; d += 2) {
          o[h][d] += pr * (f16lo_to_f32(f[d / 2]) * sb);
          o[h][d + 1] += pr * (f16hi_to_f32(f[d / 2]) * sb);
        }
      }
    }
  }
  for (int h = 0; h < p.G; ++h) {
    for (int off = 1; off < 32; off <<= 1) l[h] += __shfl_xor_sync(kAll, l[h], off);
    if (lane == 0) {
      sm[warp][h] = m[h];
      sl[warp][h] = l[h];
    }
    for (int d = 0; d < D; ++d) so[warp][h][lane * D + d] = o[h][d];
  }
  __syncthreads();
  const float sv = __ldg(p.vs + (p.per_head ? g : 0));
  for (int i = tid; i < p.G * DH; i += kWarps * 32) {
    const int h = i / DH, d = i % DH;
    float M = -INFINITY, den = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][h]);
    for (int w = 0; w < kWarps; ++w) {
      const float a = sm[w][h] == -INFINITY ? 0.f : exp2f(sm[w][h] - M);
      den += a * sl[w][h];
      acc += a * so[w][h][d];
    }
    const float r = den > 0.f ? acc * (sv / den) : acc * 0.f;
    p.out[orow + i] = static_cast<uint16_t>(f32x2_to_bf16x2(r, 0.f) & 0xFFFFu);
  }
}

static int launch_attn(const AttnParams& p, int dh, cudaStream_t s) {
  const dim3 grid(p.max_q, p.Hkv, p.B), block(kWarps * 32);
  const cudaError_t e = dh == 128 ? launch_pdl(attn_kernel<128>, grid, block, 0, s, p)
                                  : launch_pdl(attn_kernel<64>, grid, block, 0, s, p);
  if (e != cudaSuccess) return KVQ_ERR_CUDA;
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
  const int st = fp4::check_attn(q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens,
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
  if (num_q_tokens >= (int64_t(1) << 31)) return KVQ_ERR_UNSUPPORTED;
  const size_t need = kvq_fp4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, 0);
  if (need == 0) return KVQ_ERR_CUDA;
  if (workspace_bytes < need) return KVQ_ERR_WORKSPACE;
  if (num_q_tokens == 0 || max_q_len == 0) return KVQ_OK;
  const fp4::AttnParams p = {
      static_cast<const uint16_t*>(q), static_cast<const uint8_t*>(k_cache),
      static_cast<const uint8_t*>(v_cache), block_tables, seq_lens, cu_q_lens, max_blocks_per_seq,
      num_seqs, num_q_heads, num_kv_heads, num_q_heads / num_kv_heads, num_blocks, num_q_tokens,
      max_q_len, sliding_window, num_sinks, k_scale, v_scale,
      scale_granularity == KVQ_SCALE_PER_HEAD,
      static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(head_dim))),
      static_cast<uint16_t*>(out), dev_status};
  return fp4::launch_attn(p, head_dim, reinterpret_cast<cudaStream_t>(stream));
}
