// kvq_rope.cu -- norm, rotation and quantize-and-scatter in one pass.
//
// Per head row x of q and k, in binary32: y = x rsqrt(mean x^2 + eps) w, then
// (y_a, y_b) turned by the angle of their pair; q leaves as bf16, k and v as
// the cache's codes (cast_fp8(x / s), kvq_quant.cuh) in the row of the token's
// slot.  What it saves against a norm, a rotation and a write of their own is
// the rows' way to memory and back between them.
//
// A stream: (2 Hq + 2 Hkv) dh bf16 values in or out and 2 Hkv dh codes out a
// token.  DH / 16 lanes share a row, 16 dims a lane in two runs of 8: the two
// halves of its pairs, so that a pair's dims meet in one lane.  A warp takes a
// token (or a share of its rows, where the tokens are few), so its angles are
// formed once for all of the token's rows, each by one lane, and handed
// round: their turns are a 64-bit integer product modulo 2^64, exact at any
// position, of which the upper 32 bits go to sincospif.
//
// At full rate the stream leaves an SM some 9000 issue slots for 1000 rows,
// so instructions count as much as bytes: a step's rows are all of q, of k or
// of v, and what each needs is all it runs.
#include "../../include/kvq_step.h"
#include "kvq_host.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace rope {

constexpr uint32_t kAll = 0xFFFFFFFFu;
// 28 warps an SM of 72 registers each, and a step's rows on their way while one is worked on.  32768
// tokens of 32 + 2 * 8 rows of 128 (738 MB): 133 us.  When the squares were no loop, and spilled: 136; then
// with 32 warps 141, with two steps' rows on their way 156 to 168.
constexpr int kThreads = 128;
constexpr int kCtasPerSM = 7;
constexpr int kAngles = 1;  // what forming a token's angles takes, in steps

struct RopeParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride, out_stride;
  int64_t tokens;
  int hq, hkv;
  const int32_t* pos;
  int axes;
  const unsigned long long* turns;
  const uint8_t* axis;
  int pairs;  // a multiple of 8
  int interleaved;
  const uint16_t* wq;
  const uint16_t* wk;
  float eps;
  const int64_t* slots;
  void* kc;
  void* vc;
  int64_t capacity;  // num_blocks * 16
  float* ks;         // scales, or (TS) scale caches
  float* vs;
  int per_head;
  uint16_t* out;
  uint32_t* status;
  int split;  // warps that share a token's rows
};

KVQ_DEVI void unpack8(const uint4& a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(w[i]);
    x[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}

KVQ_DEVI uint4 pack8(const float (&x)[8]) {
  return make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                    f32x2_to_bf16x2(x[6], x[7]));
}

// Eight binary32 values -> eight codes of cast_fp8(x / s).  The quotient is the IEEE one: as in
// quantize2, but x has 24 significant bits where a bf16 has 8, so q0 = RN(x r) may be off by two
// units; one correction takes it within one, and from there Markstein's second is exact.
template <int FMT>
KVQ_DEVI uint2 quantize8(const float (&x)[8], const HeadScale& h) {
  uint32_t o[4];
  const float L = __uint_as_float(h.L2 & 0xFFFF0000u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 q;
    if (h.fast) {
      float2 c;
      asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(c.x) : "f"(x[2 * i]), "f"(L));
      asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(c.y) : "f"(x[2 * i + 1]), "f"(L));
      q = __fmul2_rn(c, h.r2);
      q = __ffma2_rn(__ffma2_rn(q, h.ns2, c), h.r2, q);
      q = __ffma2_rn(__ffma2_rn(q, h.ns2, c), h.r2, q);
    } else {
      q = make_float2(__fdiv_rn(x[2 * i], h.s), __fdiv_rn(x[2 * i + 1], h.s));
    }
    const uint32_t signs = ((__float_as_uint(x[2 * i]) >> 24) & 0x80u) | ((__float_as_uint(x[2 * i + 1]) >> 16) & 0x8000u);
    o[i] = f32x2_to_fp8x2<FMT>(q.x, q.y) | signs;
  }
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

template <int FMT, int DH, bool TS>
__global__ void __launch_bounds__(kThreads, kCtasPerSM) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int CH = DH / 16;      // lanes of a row
  constexpr int RW = 32 / CH;      // rows of a warp
  constexpr int NA = 8 / RW;       // angles that a lane forms, of the eight that it uses
  constexpr bool BF = FMT == KVQ_FMT_BF16;
  pdl_wait();
  pdl_allow_next();
  const int lane = threadIdx.x & 31, g = lane / CH, l = lane % CH;
  const uint32_t row_mask = (CH == 8 ? 0xFFu : 0xFu) << (lane & ~(CH - 1));
  const int pc = p.pairs >> 3;
  const bool turned = l < pc;
  // the lane's runs of 8 dims: both halves of its pairs, or (interleaved, or past the pairs) neighbours
  const bool apart = !p.interleaved && turned;
  const int d0 = 8 * (apart ? l : 2 * l), d1 = 8 * (apart ? l + pc : 2 * l + 1);
  const int sq = (p.hq + RW - 1) / RW, sk = (p.hkv + RW - 1) / RW, steps = sq + 2 * sk;
  unsigned long long turns[NA];
  uint32_t axes[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int at = 8 * l + NA * g + i;
    turns[i] = turned ? __ldg(p.turns + at) : 0ull;
    const uint32_t a = turned && p.axis ? __ldg(p.axis + at) : 0u;
    axes[i] = a < static_cast<uint32_t>(p.axes) ? a : 0u;
  }
  const int64_t items = p.tokens * p.split;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += warps) {
    const int64_t t = it / p.split;
    const int first = static_cast<int>(it - t * p.split);
    auto load = [&](int s, uint4& a, uint4& b) {
      const uint16_t* src;
      if (s < sq) {
        if (s * RW + g >= p.hq) return;
        src = p.q + t * p.q_stride + (s * RW + g) * DH;
      } else if (s < sq + sk) {
        if ((s - sq) * RW + g >= p.hkv) return;
        src = p.k + t * p.k_stride + ((s - sq) * RW + g) * DH;
      } else {
        if (s >= steps || (s - sq - sk) * RW + g >= p.hkv) return;
        src = p.v + t * p.v_stride + ((s - sq - sk) * RW + g) * DH;
      }
      // (not as constant data: q_out may be q)
      a = __ldcg(reinterpret_cast<const uint4*>(src + d0));
      b = __ldcg(reinterpret_cast<const uint4*>(src + d1));
    };
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    load(first, a, b);
    const int64_t slot = __ldg(p.slots + t);
    float cs[8], sn[8];
    {
      float c[NA], n[NA];
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        const int64_t at = __ldg(p.pos + static_cast<int64_t>(axes[i]) * p.tokens + t);
        const unsigned long long turn = static_cast<unsigned long long>(at) * turns[i];
        // the upper 32 bits, 2^32 to a turn: the nearest quarter turn, and what is left of it, at most an
        // eighth of a turn, which binary32 holds within 2^-27 half turns (sincospif takes half turns)
        const uint32_t a = static_cast<uint32_t>(turn >> 32), quarter = (a + 0x20000000u) >> 30;
        float sine, cosine;
        sincospif(static_cast<float>(static_cast<int32_t>(a - (quarter << 30))) * 0x1p-31f, &sine, &cosine);
        c[i] = __uint_as_float(__float_as_uint(quarter & 1u ? sine : cosine) ^ ((quarter + 1u & 2u) << 30));
        n[i] = __uint_as_float(__float_as_uint(quarter & 1u ? cosine : sine) ^ ((quarter & 2u) << 30));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = __shfl_sync(kAll, c[i % NA], i / NA * CH + l);
        sn[i] = __shfl_sync(kAll, n[i % NA], i / NA * CH + l);
      }
    }
    if (slot >= p.capacity && first == 0 && lane == 0) flag_status(p.status, KVQ_DEV_BAD_SLOT);
    const bool kept = slot >= 0 && slot < p.capacity;
    // The rows' norm and turn: x, y are the lane's two runs.
    auto norm_and_turn = [&](float (&x)[8], float (&y)[8], const uint16_t* w) {
      if (w) {
        // Squares leave binary32 where values pass 2^63, or lie below 2^-63 beside an eps that is as small:
        // such rows are multiplied by a power of two, and summed once more.  (A loop that ordinary rows go
        // through once: with the second sum written out after the first, 48 bytes spilled, 12.6 us where
        // 4100 tokens of 16 + 2 * 16 rows of 64 in bf16 take 11.5.)
        float mean, eps = p.eps;
#pragma unroll 1
        for (int again = 0;; ++again) {
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(x[2 * i], x[2 * i + 1]), sum);
            sum = __ffma2_rn(make_float2(y[2 * i], y[2 * i + 1]), make_float2(y[2 * i], y[2 * i + 1]), sum);
          }
          float sq2 = sum.x + sum.y;
#pragma unroll
          for (int off = 1; off < CH; off <<= 1) sq2 += __shfl_xor_sync(kAll, sq2, off);
          mean = sq2 * (1.f / DH) + eps;
          if (__builtin_expect(again || !__any_sync(kAll, !(mean > 0x1p-90f && mean < 0x1p120f)), 1)) break;
          const float by = mean <= 0x1p-90f ? 0x1p100f : mean < 0x1p120f ? 1.f : 0x1p-70f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] *= by;
            y[i] *= by;
          }
          eps *= by;
          eps *= by;
        }
        const float f = rsqrtf(mean);
        float u[8], v[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(w + d0)), u);
        unpack8(__ldg(reinterpret_cast<const uint4*>(w + d1)), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= f * u[i];
          y[i] *= f * v[i];
        }
      }
      if (!turned) return;
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
          x[2 * i] = x0 * cs[i] - x1 * sn[i];
          x[2 * i + 1] = x0 * sn[i] + x1 * cs[i];
          y[2 * i] = y0 * cs[4 + i] - y1 * sn[4 + i];
          y[2 * i + 1] = y0 * sn[4 + i] + y1 * cs[4 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x2 = make_float2(x[2 * i], x[2 * i + 1]), y2 = make_float2(y[2 * i], y[2 * i + 1]);
          const float2 c2 = make_float2(cs[2 * i], cs[2 * i + 1]), s2 = make_float2(sn[2 * i], sn[2 * i + 1]);
          const float2 n2 = make_float2(-s2.x, -s2.y);
          const float2 u = __ffma2_rn(x2, c2, __fmul2_rn(y2, n2)), v = __ffma2_rn(y2, c2, __fmul2_rn(x2, s2));
          x[2 * i] = u.x;
          x[2 * i + 1] = u.y;
          y[2 * i] = v.x;
          y[2 * i + 1] = v.y;
        }
      }
    };
    auto step = [&](int s, const uint4& a, const uint4& b) {
      if (s < sq) {
        float x[8], y[8];
        unpack8(a, x);
        unpack8(b, y);
        norm_and_turn(x, y, p.wq);
        const int row = s * RW + g;
        if (row >= p.hq) return;
        uint16_t* dst = p.out + t * p.out_stride + row * DH;
        __stcs(reinterpret_cast<uint4*>(dst + d0), pack8(x));
        __stcs(reinterpret_cast<uint4*>(dst + d1), pack8(y));
        return;
      }
      const bool is_v = s >= sq + sk;
      const int h = (s - sq - (is_v ? sk : 0)) * RW + g;
      const bool live = h < p.hkv && kept;
      const int64_t at = ((slot >> 4) * p.hkv + h) * 16 + (slot & 15);
      uint2 lo = {}, hi = {};  // codes
      float* scale = is_v ? p.vs : p.ks;
      if (is_v) {
        if constexpr (BF) {
          if (!live) return;
          uint16_t* dst = static_cast<uint16_t*>(p.vc) + at * DH;
          *reinterpret_cast<uint4*>(dst + d0) = a;
          *reinterpret_cast<uint4*>(dst + d1) = b;
          return;
        } else {
          float f = 0.f;
          if (TS)  // every lane of the row takes part, whatever its slot
            f = scale_of_amax<FMT>(row_amax<CH>(a, b, row_mask));
          if (!live) return;
          if (!TS) f = __ldg(scale + (p.per_head ? h : 0));
          const uint4 o = quantize16<FMT>(a, b, head_scale(f));
          lo = make_uint2(o.x, o.y);
          hi = make_uint2(o.z, o.w);
          if (TS && l == 0) scale[at] = f;
        }
      } else {
        float x[8], y[8];
        unpack8(a, x);
        unpack8(b, y);
        norm_and_turn(x, y, p.wk);
        if constexpr (BF) {
          if (!live) return;
          uint16_t* dst = static_cast<uint16_t*>(p.kc) + at * DH;
          *reinterpret_cast<uint4*>(dst + d0) = pack8(x);
          *reinterpret_cast<uint4*>(dst + d1) = pack8(y);
          return;
        } else {
          float f = 0.f;
          if (TS) {
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu, v = __float_as_uint(y[i]) & 0x7FFFFFFFu;
              m = max(m, max(u < 0x7F800000u ? u : 0u, v < 0x7F800000u ? v : 0u));
            }
#pragma unroll
            for (int off = 1; off < CH; off <<= 1) m = max(m, __shfl_xor_sync(row_mask, m, off));
            f = scale_of_amax<FMT>(__uint_as_float(m));
          }
          if (!live) return;
          if (!TS) f = __ldg(scale + (p.per_head ? h : 0));
          const HeadScale hs = head_scale(f);
          lo = quantize8<FMT>(x, hs);
          hi = quantize8<FMT>(y, hs);
          if (TS && l == 0) scale[at] = f;
        }
      }
      uint8_t* dst = static_cast<uint8_t*>(is_v ? p.vc : p.kc) + at * DH;
      *reinterpret_cast<uint2*>(dst + d0) = lo;
      *reinterpret_cast<uint2*>(dst + d1) = hi;
    };
    for (int s = first; s < steps; s += p.split) {
      const uint4 ha = a, hb = b;
      load(s + p.split, a, b);
      step(s, ha, hb);
      __syncwarp();
    }
  }
}

template <int FMT, int DH, bool TS>
static cudaError_t launch_rope(RopeParams& p, cudaStream_t s) {
  const int rw = 32 / (DH / 16), steps = (p.hq + rw - 1) / rw + 2 * ((p.hkv + rw - 1) / rw);
  const int64_t warps = static_cast<int64_t>(device_sm_count()) * kCtasPerSM * (kThreads / 32);
  // A token's steps are shared by as many warps as make the longest warp's work least, a share's
  // angles counted as kAngles steps.
  int64_t split = 1, least = INT64_MAX;
  for (int n = 1; n <= steps && n <= 64; ++n) {
    const int64_t work = (p.tokens * n + warps - 1) / warps * ((steps + n - 1) / n + kAngles);
    if (work < least) {
      least = work;
      split = n;
    }
  }
  p.split = static_cast<int>(split);
  const int64_t need = (p.tokens * split + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * kCtasPerSM;
  const dim3 grid(static_cast<unsigned>(need < cap ? need : cap));
  return launch_pdl(rope_kernel<FMT, DH, TS>, grid, dim3(kThreads), 0, s, p);
}

template <int FMT, bool TS>
static cudaError_t launch_rope_dh(RopeParams& p, int dh, cudaStream_t s) {
  return dh == 128 ? launch_rope<FMT, 128, TS>(p, s) : launch_rope<FMT, 64, TS>(p, s);
}

}  // namespace rope
}  // namespace kvq

using namespace kvq;

extern "C" int kvq_rope_write(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, int64_t num_tokens, int num_q_heads,
                              int num_kv_heads, int head_dim, const int32_t* positions, int num_axes,
                              const int64_t* turns, const uint8_t* axis, int num_pairs,
                              int interleaved, const void* q_weight, const void* k_weight, float eps,
                              const int64_t* slot_mapping, void* k_cache, void* v_cache,
                              int64_t num_blocks, int block_size, float* k_scale, int k_scale_len,
                              float* v_scale, int v_scale_len, int scale_granularity, int fmt,
                              void* q_out, int64_t q_out_stride, uint32_t* dev_status,
                              kvq_stream_t stream) {
  if (fmt < KVQ_FMT_BF16 || fmt > KVQ_FMT_E5M2) return KVQ_ERR_ARG;
  if (scale_granularity < KVQ_SCALE_PER_TENSOR || scale_granularity > KVQ_SCALE_PER_TOKEN_HEAD) return KVQ_ERR_ARG;
  const bool ts = scale_granularity == KVQ_SCALE_PER_TOKEN_HEAD;
  if (ts && fmt == KVQ_FMT_BF16) return KVQ_ERR_UNSUPPORTED;
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 || num_axes <= 0 || num_pairs < 0 ||
      !(eps >= 0.f))
    return KVQ_ERR_ARG;
  if (!k_cache || !v_cache || (num_pairs > 0 && !turns)) return KVQ_ERR_NULL;
  if (num_tokens > 0 && (!q || !k || !v || !q_out || !slot_mapping || !positions)) return KVQ_ERR_NULL;
  if (head_dim != 64 && head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (block_size != 16 || num_axes > 16) return KVQ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_q_heads) + num_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  if (num_pairs % 8 || num_pairs > head_dim / 2) return KVQ_ERR_SHAPE;
  const int64_t nq = static_cast<int64_t>(num_q_heads) * head_dim, nk = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_stride < nq || q_out_stride < nq || k_stride < nk || v_stride < nk) return KVQ_ERR_SHAPE;
  if (q == q_out && q_stride != q_out_stride) return KVQ_ERR_SHAPE;
  if ((q_stride | q_out_stride | k_stride | v_stride) % 8) return KVQ_ERR_ALIGN;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(q_weight) || !aligned16(k_weight) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) ||
      (reinterpret_cast<uintptr_t>(turns) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u) ||
      ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & (ts ? 15u : 3u)))
    return KVQ_ERR_ALIGN;
  if (num_blocks > (INT64_MAX / 16) / nk) return KVQ_ERR_SHAPE;
  if (fmt != KVQ_FMT_BF16) {
    if (!k_scale || !v_scale) return KVQ_ERR_NULL;
    const int64_t want = ts ? num_blocks * num_kv_heads * 16 : scale_granularity == KVQ_SCALE_PER_HEAD ? num_kv_heads : 1;
    if (k_scale_len != want || v_scale_len != want) return KVQ_ERR_SHAPE;
  }
  if (num_tokens == 0) return KVQ_OK;
  if (device_sm_count() <= 0) return KVQ_ERR_CUDA;
  rope::RopeParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.out_stride = q_out_stride;
  p.tokens = num_tokens;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.pos = positions;
  p.axes = num_axes;
  p.turns = reinterpret_cast<const unsigned long long*>(turns);
  p.axis = axis;
  p.pairs = num_pairs;
  p.interleaved = interleaved != 0;
  p.wq = static_cast<const uint16_t*>(q_weight);
  p.wk = static_cast<const uint16_t*>(k_weight);
  p.eps = eps;
  p.slots = slot_mapping;
  p.kc = k_cache;
  p.vc = v_cache;
  p.capacity = num_blocks * block_size;
  p.ks = k_scale;
  p.vs = v_scale;
  p.per_head = scale_granularity == KVQ_SCALE_PER_HEAD;
  p.out = static_cast<uint16_t*>(q_out);
  p.status = dev_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (fmt == KVQ_FMT_BF16)
    e = rope::launch_rope_dh<KVQ_FMT_BF16, false>(p, head_dim, s);
  else if (fmt == KVQ_FMT_E4M3)
    e = ts ? rope::launch_rope_dh<KVQ_FMT_E4M3, true>(p, head_dim, s) : rope::launch_rope_dh<KVQ_FMT_E4M3, false>(p, head_dim, s);
  else
    e = ts ? rope::launch_rope_dh<KVQ_FMT_E5M2, true>(p, head_dim, s) : rope::launch_rope_dh<KVQ_FMT_E5M2, false>(p, head_dim, s);
  if (e != cudaSuccess) return KVQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
