// kvq_fp4_write.cu -- quantize-and-scatter into the microscaled 4-bit cache,
// and the gather back to bf16.
//
// Both are HBM streams.  A thread owns one block of 16 consecutive dims of
// one (token, KV head) row, the unit that shares a scale: the write loads two
// 16-byte words per tensor and stores 8 bytes of codes and one of scale, the
// read the reverse, so a row's lanes move whole contiguous runs.
#include <algorithm>

#include "kvq_fp4.cuh"
#include "kvq_fp4_host.h"

namespace kvq {
namespace fp4 {

struct WriteParams {
  const uint16_t* k;
  const uint16_t* v;
  int64_t token_stride;
  const int64_t* slots;
  int64_t num_tokens;
  int hkv;
  uint8_t* kc;
  uint8_t* vc;
  int64_t capacity;  // num_blocks * 16
  const float* ks;
  const float* vs;
  int per_head;
  uint32_t* status;
};

// x / d for bf16 x as the IEEE binary32 quotient: for d in [2^-80, 2^80] from
// r = RN(1/d) and one fused residual correction (Markstein's iteration, exact
// for every bf16 significand over every binary32 one), else by division.  The
// numerator is first clamped to +-2^20 d rounded toward zero, far past what
// the codes and scales hold, so that no intermediate overflows.
struct Divider {
  float d, r;
  uint32_t L2;  // bf16x2 (L, L), L the clamp
  bool fast;
};

KVQ_DEVI Divider divider(float d) {
  Divider v;
  v.d = d;
  v.fast = d >= 0x1p-80f && d <= 0x1p80f;
  v.r = __frcp_rn(d);
  uint16_t L;
  asm("cvt.rz.bf16.f32 %0, %1;" : "=h"(L) : "f"(v.fast ? d * 1048576.f : 0.f));
  v.L2 = static_cast<uint32_t>(L) * 0x10001u;
  return v;
}

// The two bf16 of a word over v.d, v.fast.
KVQ_DEVI float2 quotient2(uint32_t w, const Divider& v) {
  uint32_t c;  // sign(x) min(|x|, L)
  asm("min.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(w), "r"(v.L2));
  const float2 x = make_float2(bf16lo_to_f32(c), bf16hi_to_f32(c));
  const float2 r2 = make_float2(v.r, v.r), nd2 = make_float2(-v.d, -v.d);
  const float2 q0 = __fmul2_rn(x, r2);
  const float2 e = __ffma2_rn(q0, nd2, x);
  return __ffma2_rn(e, r2, q0);
}

// One block: 16 bf16 (a, b) -> 8 bytes of codes and the scale byte.
// s: the head's scale; six: the divider of 6 s.
KVQ_DEVI uint2 quantize_block(const uint4& a, const uint4& b, float s, const Divider& six,
                              uint32_t& scale) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  // magnitudes order like their bits: finite < infinity (0x7F80) < NaN
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
  const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  if (m > 0x7F80u) {  // a NaN: the scale code NaN, codes of 0
    scale = 0x7Fu;
    return make_uint2(0u, 0u);
  }
  const uint32_t amax = min(m, 0x7F7Fu);
  const float top = six.fast ? quotient2(amax, six).x : __fdiv_rn(bf16lo_to_f32(amax), six.d);
  scale = f32x2_to_fp8x2<KVQ_FMT_E4M3>(top, 0.f) & 0xFFu;
  const float r = __fmul_rn(e4m3_to_f32(scale), s);
  if (!(r > 0.f)) return make_uint2(0u, 0u);
  const Divider div = divider(r);
  float q[16];
  if (div.fast) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = quotient2(w[i], div);
      q[2 * i] = v.x;
      q[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[2 * i] = __fdiv_rn(bf16lo_to_f32(w[i]), r);
      q[2 * i + 1] = __fdiv_rn(bf16hi_to_f32(w[i]), r);
    }
  }
  uint2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float e[8] = {q[8 * h], q[8 * h + 1], q[8 * h + 2], q[8 * h + 3],
                        q[8 * h + 4], q[8 * h + 5], q[8 * h + 6], q[8 * h + 7]};
    // The residual form loses the sign of a zero quotient: all signs are taken from the inputs,
    // bits 15 and 31 of word i to bits 8 i + 3 and 8 i + 7.
    const uint32_t lo = prmt(w[4 * h], w[4 * h + 1], 0x7531u), hi = prmt(w[4 * h + 2], w[4 * h + 3], 0x7531u);
    const uint32_t even = prmt(lo, hi, 0x6420u), odd = prmt(lo, hi, 0x7531u);
    (h ? o.y : o.x) = f32x8_to_e2m1x8(e) | ((even >> 4) & 0x08080808u) | (odd & 0x80808080u);
  }
  return o;
}

// Blocks of 256 threads per SM: at 5 (51 registers) the conversion spills.
// 32768 tokens of 8 heads of 128: 3 blocks 35.8 us, 4 34.9, 5 51.2.
constexpr int kWriteCtas = 4;

// K and V are two rows of the grid.  The grid's thread count is a multiple of
// the Hkv * DH / 16 blocks of a token (token_row_shape), so a thread keeps its
// block and its head's scale and strides over the tokens; the next token's loads
// are issued before the current one is converted.
template <int DH>
__global__ void __launch_bounds__(256, kWriteCtas) write_kernel(const WriteParams p) {
  using P = Page<DH>;
  constexpr int CH = DH / 16;
  pdl_wait();  // the inputs may come from the kernel before this one
  pdl_allow_next();
  const bool is_v = blockIdx.y != 0;
  const uint16_t* in = is_v ? p.v : p.k;
  uint8_t* cache = is_v ? p.vc : p.kc;
  const int row_units = p.hkv * CH;
  const int64_t gtid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int rem = static_cast<int>(gtid % row_units);
  const int h = rem / CH, c = rem % CH;
  const int64_t tstride = static_cast<int64_t>(gridDim.x) * blockDim.x / row_units;
  int64_t t = gtid / row_units;
  if (t >= p.num_tokens) return;
  const float s = __ldg((is_v ? p.vs : p.ks) + (p.per_head ? h : 0));
  const Divider six = divider(__fmul_rn(6.f, s));
  uint4 x[2];
  int64_t slot;
  auto load = [&](int64_t tt, uint4 (&xx)[2], int64_t& sl) {
    const uint4* src = reinterpret_cast<const uint4*>(in + tt * p.token_stride + rem * 16);
    xx[0] = __ldcs(src);
    xx[1] = __ldcs(src + 1);
    sl = __ldg(p.slots + tt);
  };
  load(t, x, slot);
  while (true) {
    const int64_t tn = t + tstride;
    uint4 xn[2];
    int64_t sn = -1;
    if (tn < p.num_tokens) load(tn, xn, sn);
    if (slot >= p.capacity) {
      if (rem == 0) flag_status(p.status, KVQ_DEV_BAD_SLOT);
    } else if (slot >= 0) {  // a negative slot is a padding token
      uint8_t* page = cache + ((slot >> 4) * p.hkv + h) * P::kBytes;
      const int row = static_cast<int>(slot & 15);
      uint32_t sb;
      *reinterpret_cast<uint2*>(page + row * P::kRow + c * 8) = quantize_block(x[0], x[1], s, six, sb);
      page[P::kScaleOff + row * P::kScales + c] = static_cast<uint8_t>(sb);
    }
    if (tn >= p.num_tokens) break;
    t = tn;
    x[0] = xn[0];
    x[1] = xn[1];
    slot = sn;
  }
}

struct ReadParams {
  const uint8_t* kc;
  const uint8_t* vc;
  int64_t num_blocks;
  int hkv;
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* starts;
  const int32_t* cu;
  int num_seqs;
  int64_t num_rows;
  const float* ks;
  const float* vs;
  int per_head;
  uint16_t* ko;
  uint16_t* vo;
  int64_t out_stride;
  uint32_t* status;
  int warp_rows;  // output rows that a warp takes
};

// 16 values of one block: (code * block scale) exact in f16 and binary32, one
// binary32 product with s, then bf16.
KVQ_DEVI void read_block(uint2 w, uint32_t sb8, float s, uint16_t* dst) {
  const float sb = e4m3_to_f32(sb8);
  uint32_t o[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f[4];
    e2m1x8_to_f16x2x4(h ? w.y : w.x, f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[4 * h + i] = f32x2_to_bf16x2(__fmul_rn(__fmul_rn(f16lo_to_f32(f[i]), sb), s),
                                     __fmul_rn(__fmul_rn(f16hi_to_f32(f[i]), sb), s));
  }
  uint4* d = reinterpret_cast<uint4*>(dst);
  __stcs(d, make_uint4(o[0], o[1], o[2], o[3]));
  __stcs(d + 1, make_uint4(o[4], o[5], o[6], o[7]));
}

// A warp takes p.warp_rows output rows at a time: a lane looks up one row's
// sequence and page, then the lanes go through the rows' blocks in order, so
// that the stores run on and kReadDeep blocks of K and of V are in flight a lane.
constexpr int kReadDeep = 4;
constexpr int kMaxReadRows = 8;

template <int DH>
__global__ void __launch_bounds__(256) read_kernel(const ReadParams p) {
  using P = Page<DH>;
  constexpr int CH = DH / 16;
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  pdl_wait();
  pdl_allow_next();
  const int lane = threadIdx.x & 31;
  const int units = p.hkv * CH;  // blocks of a row
  const int64_t rows = min(p.num_rows, static_cast<int64_t>(__ldg(p.cu + p.num_seqs)));
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5)) * p.warp_rows;
  if (r0 < rows) {
    const int n = static_cast<int>(min(static_cast<int64_t>(p.warp_rows), rows - r0));
    // the first row's sequence, the last b with cu[b] <= r0, by all lanes: 32 probes a step
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
      const int below = __popc(__ballot_sync(kAll, at <= hi && __ldg(p.cu + at) <= r0));
      lo += below * step;
      hi = min(hi, lo + step - 1);
    }
    int my_blk = -1, my_tok = 0;
    if (lane < n) {
      const int64_t r = r0 + lane;
      while (lo < p.num_seqs - 1 && __ldg(p.cu + lo + 1) <= r) ++lo;
      const int64_t pos = r - __ldg(p.cu + lo) + (p.starts ? __ldg(p.starts + lo) : 0);
      if (pos < 0 || pos >= static_cast<int64_t>(p.max_blocks) * kTok) {
        flag_status(p.status, KVQ_DEV_BAD_SEQLEN);
      } else {
        my_tok = static_cast<int>(pos % kTok);
        my_blk = __ldg(p.block_tables + static_cast<int64_t>(lo) * p.max_blocks + pos / kTok);
        if (my_blk < 0 || my_blk >= p.num_blocks) {
          flag_status(p.status, KVQ_DEV_BAD_BLOCK);
          my_blk = -1;
        }
      }
    }
    __syncwarp();
    const int total = n * units;
    for (int i0 = 0; i0 < total; i0 += 32 * kReadDeep) {
      uint2 wk[kReadDeep], wv[kReadDeep];
      uint32_t sk[kReadDeep], sv[kReadDeep];
      int row[kReadDeep], rem[kReadDeep];
#pragma unroll
      for (int y = 0; y < kReadDeep; ++y) {
        const int i = i0 + 32 * y + lane;
        row[y] = i < total ? i / units : -1;
        rem[y] = i - row[y] * units;
        const int from = row[y] < 0 ? 0 : row[y];
        const int blk = __shfl_sync(kAll, my_blk, from), tok = __shfl_sync(kAll, my_tok, from);
        wk[y] = wv[y] = make_uint2(0u, 0u);
        sk[y] = sv[y] = 0u;
        if (row[y] >= 0 && blk >= 0) {
          const int h = rem[y] / CH, c = rem[y] % CH;
          const int64_t page = (static_cast<int64_t>(blk) * p.hkv + h) * P::kBytes;
          const int64_t code = page + tok * P::kRow + c * 8, sc = page + P::kScaleOff + tok * P::kScales + c;
          wk[y] = __ldg(reinterpret_cast<const uint2*>(p.kc + code));
          wv[y] = __ldg(reinterpret_cast<const uint2*>(p.vc + code));
          sk[y] = __ldg(p.kc + sc);
          sv[y] = __ldg(p.vc + sc);
        }
      }
#pragma unroll
      for (int y = 0; y < kReadDeep; ++y) {
        if (row[y] < 0) continue;
        const int h = p.per_head ? rem[y] / CH : 0;
        const int64_t dst = (r0 + row[y]) * p.out_stride + rem[y] * 16;
        read_block(wk[y], sk[y], __ldg(p.ks + h), p.ko + dst);
        read_block(wv[y], sv[y], __ldg(p.vs + h), p.vo + dst);
      }
    }
  }
}

}  // namespace fp4
}  // namespace kvq

using namespace kvq;

extern "C" int kvq_fp4_write(const void* k, const void* v, int64_t token_stride,
                             const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads,
                             int head_dim, void* k_cache, void* v_cache, int64_t num_blocks,
                             int block_size, const float* k_scale, int k_scale_len,
                             const float* v_scale, int v_scale_len, int scale_granularity,
                             uint32_t* dev_status, kvq_stream_t stream) {
  if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0) return KVQ_ERR_ARG;
  const int sc = fp4::check_scales(k_scale, k_scale_len, v_scale, v_scale_len, scale_granularity,
                                   num_kv_heads);
  if (sc != KVQ_OK) return sc;
  if (!k_cache || !v_cache) return KVQ_ERR_NULL;
  if (num_tokens > 0 && (!k || !v || !slot_mapping)) return KVQ_ERR_NULL;
  const int cc = fp4::check_caches(num_blocks, block_size, num_kv_heads, head_dim);
  if (cc != KVQ_OK) return cc;
  if (token_stride < static_cast<int64_t>(num_kv_heads) * head_dim) return KVQ_ERR_SHAPE;
  if (token_stride % 8 != 0) return KVQ_ERR_ALIGN;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return KVQ_ERR_ALIGN;
  if (num_tokens > 0 && token_stride > (INT64_MAX / 16) / num_tokens)
    return KVQ_ERR_SHAPE;
  if (num_tokens == 0) return KVQ_OK;
  if (device_sm_count() <= 0) return KVQ_ERR_CUDA;
  fp4::WriteParams p;
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.token_stride = token_stride;
  p.slots = slot_mapping;
  p.num_tokens = num_tokens;
  p.hkv = num_kv_heads;
  p.kc = static_cast<uint8_t*>(k_cache);
  p.vc = static_cast<uint8_t*>(v_cache);
  p.capacity = num_blocks * block_size;
  p.ks = k_scale;
  p.vs = v_scale;
  p.per_head = scale_granularity == KVQ_SCALE_PER_HEAD;
  p.status = dev_status;
  int grid = 0, block = 0;
  token_row_shape(num_tokens, num_kv_heads * (head_dim / 16), fp4::kWriteCtas, grid, block);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = head_dim == 128
                            ? launch_pdl(fp4::write_kernel<128>, dim3(grid, 2), dim3(block), 0, s, p)
                            : launch_pdl(fp4::write_kernel<64>, dim3(grid, 2), dim3(block), 0, s, p);
  if (e != cudaSuccess) return KVQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

extern "C" int kvq_fp4_read(const void* k_cache, const void* v_cache, int64_t num_blocks,
                            int block_size, int num_kv_heads, int head_dim,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* starts, const int32_t* cu_lens, int num_seqs,
                            int64_t num_rows, const float* k_scale, int k_scale_len,
                            const float* v_scale, int v_scale_len, int scale_granularity,
                            void* k_out, void* v_out, int64_t out_stride, uint32_t* dev_status,
                            kvq_stream_t stream) {
  if (num_rows < 0 || num_kv_heads <= 0 || num_blocks <= 0 || num_seqs <= 0 ||
      max_blocks_per_seq <= 0)
    return KVQ_ERR_ARG;
  const int sc = fp4::check_scales(k_scale, k_scale_len, v_scale, v_scale_len, scale_granularity,
                                   num_kv_heads);
  if (sc != KVQ_OK) return sc;
  if (!k_cache || !v_cache || !block_tables || !cu_lens) return KVQ_ERR_NULL;
  if (num_rows > 0 && (!k_out || !v_out)) return KVQ_ERR_NULL;
  const int cc = fp4::check_caches(num_blocks, block_size, num_kv_heads, head_dim);
  if (cc != KVQ_OK) return cc;
  if (out_stride < static_cast<int64_t>(num_kv_heads) * head_dim) return KVQ_ERR_SHAPE;
  if (out_stride % 8 != 0) return KVQ_ERR_ALIGN;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out) ||
      ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(starts) |
        reinterpret_cast<uintptr_t>(cu_lens)) & 3u))
    return KVQ_ERR_ALIGN;
  if (num_rows > 0 && out_stride > (INT64_MAX / 16) / num_rows)
    return KVQ_ERR_SHAPE;
  if (num_rows == 0) return KVQ_OK;
  if (device_sm_count() <= 0) return KVQ_ERR_CUDA;
  fp4::ReadParams p;
  p.kc = static_cast<const uint8_t*>(k_cache);
  p.vc = static_cast<const uint8_t*>(v_cache);
  p.num_blocks = num_blocks;
  p.hkv = num_kv_heads;
  p.block_tables = block_tables;
  p.max_blocks = max_blocks_per_seq;
  p.starts = starts;
  p.cu = cu_lens;
  p.num_seqs = num_seqs;
  p.num_rows = num_rows;
  p.ks = k_scale;
  p.vs = v_scale;
  p.per_head = scale_granularity == KVQ_SCALE_PER_HEAD;
  p.ko = static_cast<uint16_t*>(k_out);
  p.vo = static_cast<uint16_t*>(v_out);
  p.out_stride = out_stride;
  p.status = dev_status;
  // Rows of a warp, for rows of 64 blocks (more of them where a row has fewer).  Few rows go one
  // to a warp, for the shortest chain of loads.  One sequence of 8 heads of 128, graph replay over
  // tensors past L2, one / two / four a warp: 32 rows 2.7 / 3.4 / 5.2 us, 1023 3.4 / 4.0 / 5.8, 2049
  // 4.7 / 4.4 / 6.1, 32768 35.2 / 35.5 / 34.6, 65535 65.5 / 61.4 / 62.0, 262144 242 / 215 / 222; 64
  // sequences of 512 to 8192 tokens, new inputs every time, 180 / 165 / 160.
  const int units = num_kv_heads * (head_dim / 16);
  const int base = num_rows < 1024 ? 1 : (num_rows < 65536 ? 2 : 4);
  p.warp_rows = std::min(fp4::kMaxReadRows, base * std::max(1, 64 / units));
  const int64_t need = (num_rows + 8 * p.warp_rows - 1) / (8 * p.warp_rows);
  if (need > 0x7FFFFFFF) return KVQ_ERR_UNSUPPORTED;
  const int grid = static_cast<int>(need), block = 256;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = head_dim == 128
                            ? launch_pdl(fp4::read_kernel<128>, dim3(grid), dim3(block), 0, s, p)
                            : launch_pdl(fp4::read_kernel<64>, dim3(grid), dim3(block), 0, s, p);
  if (e != cudaSuccess) return KVQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
