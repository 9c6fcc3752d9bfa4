// kvq_quant.cuh -- the quantizing division of the FP8 writes: x / s rounded to
// binary32, then to FP8, and the scales of rows that bring their own.
#pragma once

#include "kvq_common.cuh"

namespace kvq {

// Per-head constants of the quantizing division x / s.  For s in
// [2^-80, 2^80] the quotient comes from the reciprocal r = RN(1/s) and one
// fused residual correction (Markstein's iteration): q0 = RN(x r),
// e = RN(x - q0 s), q = RN(q0 + e r) -- the IEEE binary32 quotient for every
// bf16 significand and every binary32 scale significand (checked
// exhaustively), on the packed f32x2 pipes two elements at a time.  Inputs
// first go through a bf16x2 clamp to +-L, L = 2^20 s rounded toward zero
// (L >= 2^19 s): every |x| > L saturates the FP8 format and so does L itself,
// infinities turn into +-L and NaN stays NaN, so q0, e and q stay finite.
// The one sign the residual form can lose is that of a zero quotient from
// x = -0; the FP8 sign bit is therefore OR-ed in from the bf16 sign bit
// (equal to the quotient's sign everywhere else).  Quotients too small for
// the residual to stay normal encode to a signed FP8 zero either way.
struct HeadScale {
  float2 r2, ns2;  // (r, r), (-s, -s)
  uint32_t L2;  // bf16x2 (L, L)
  float s;
  bool fast;
};

KVQ_DEVI HeadScale head_scale(float s) {
  HeadScale h;
  h.s = s;
  h.fast = s >= 0x1p-80f && s <= 0x1p80f;
  const float r = __frcp_rn(s);
  h.r2 = make_float2(r, r);
  h.ns2 = make_float2(-s, -s);
  uint16_t L;
  asm("cvt.rz.bf16.f32 %0, %1;" : "=h"(L) : "f"(h.fast ? s * 1048576.f : 0.f));
  h.L2 = static_cast<uint32_t>(L) * 0x10001u;
  return h;
}

// sign(x) * min(|x|, L) on both halves (L positive), NaN propagated.
KVQ_DEVI uint32_t bf16x2_clamp(uint32_t w, uint32_t L2) {
  uint32_t d;
  asm("min.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(L2));
  return d;
}

// Two bf16 (one word) -> two FP8 codes (low byte = low element).
template <int FMT>
KVQ_DEVI uint32_t quantize2(uint32_t w, const HeadScale& h) {
  float2 q;
  if (h.fast) {
    const uint32_t c = bf16x2_clamp(w, h.L2);
    const float2 x = make_float2(bf16lo_to_f32(c), bf16hi_to_f32(c));
    const float2 q0 = __fmul2_rn(x, h.r2);
    const float2 e = __ffma2_rn(q0, h.ns2, x);
    q = __ffma2_rn(e, h.r2, q0);
  } else {
    q = make_float2(__fdiv_rn(bf16lo_to_f32(w), h.s), __fdiv_rn(bf16hi_to_f32(w), h.s));
  }
  return f32x2_to_fp8x2<FMT>(q.x, q.y);
}

// Sixteen bf16 values (two uint4) -> sixteen FP8 codes: binary32 quotient
// x / s, then the saturating RNE conversion to FP8; signs from the inputs.
template <int FMT>
KVQ_DEVI uint4 quantize16(const uint4& a, const uint4& b, const HeadScale& h) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t codes = prmt(quantize2<FMT>(w[2 * i], h), quantize2<FMT>(w[2 * i + 1], h), 0x5410u);
    const uint32_t signs = prmt(w[2 * i], w[2 * i + 1], 0x7531u);
    o[i] = codes | (signs & 0x80808080u);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Scale of one (token, KV head) row held by CH consecutive lanes (aligned to
// CH in the warp; mask = those lanes): the largest finite magnitude of the
// row over the format's largest finite value (binary32 division), or 1 when
// that is 0.
template <int CH>
KVQ_DEVI float row_amax(const uint4& a, const uint4& b, uint32_t mask) {
  uint32_t am = mag_of_key16(max_key16(kMagKey0, a, b));
#pragma unroll
  for (int off = 1; off < CH; off <<= 1) am = max(am, __shfl_xor_sync(mask, am, off));
  return __uint_as_float(am);
}

template <int FMT>
KVQ_DEVI float scale_of_amax(float amax) {
  const float q = __fdiv_rn(amax, FMT == KVQ_FMT_E4M3 ? 448.f : 57344.f);
  return q > 0.f ? q : 1.f;
}

// The K and V row scales' division constants: one half of the row's lanes
// derives K's, the other half V's (a correctly rounded division and
// reciprocal each), and the halves swap them.
template <int FMT, int CH>
KVQ_DEVI void row_scales(const uint4 (&k)[2], const uint4 (&v)[2], uint32_t mask, HeadScale& hk,
                         HeadScale& hv) {
  const float ak = row_amax<CH>(k[0], k[1], mask), av = row_amax<CH>(v[0], v[1], mask);
  const bool k_half = (threadIdx.x & (CH / 2)) == 0;
  const HeadScale h = head_scale(scale_of_amax<FMT>(k_half ? ak : av));
  HeadScale o;
  o.s = __shfl_xor_sync(mask, h.s, CH / 2);
  const float r = __shfl_xor_sync(mask, h.r2.x, CH / 2);
  o.L2 = __shfl_xor_sync(mask, h.L2, CH / 2);
  o.fast = o.s >= 0x1p-80f && o.s <= 0x1p80f;
  o.r2 = make_float2(r, r);
  o.ns2 = make_float2(-o.s, -o.s);
  hk = k_half ? h : o;
  hv = k_half ? o : h;
}

}  // namespace kvq
