// kvq_fp4.cuh -- device helpers of the microscaled 4-bit cache (NVFP4: E2M1
// codes, one E4M3 scale per 16 consecutive dims; layout in kvq_fp4.h).
#pragma once

#include "../../include/kvq_fp4.h"
#include "kvq_common.cuh"

namespace kvq {
namespace fp4 {

constexpr int kTok = 16;  // tokens of a page (block_size)

// One KV head's page of one tensor: 16 code rows, then 16 scale rows.
template <int DH>
struct Page {
  static constexpr int kRow = DH / 2;        // code bytes of a token
  static constexpr int kScales = DH / 16;    // scale bytes of a token
  static constexpr int kScaleOff = kTok * kRow;
  static constexpr int kBytes = KVQ_FP4_PAGE_BYTES(DH);
  static_assert(kBytes == kScaleOff + kTok * kScales && kBytes % 16 == 0, "page layout");
};

// ------------------------------------------------------------------ conversions

// Eight E2M1 codes of one word -> f16x2 pairs (byte i -> h[i], the low four
// bits in the low half).  Exact.
KVQ_DEVI void e2m1x8_to_f16x2x4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight binary32 values -> eight E2M1 codes of one word (value 0 in the low
// four bits), round to nearest even, saturating to +-6.
KVQ_DEVI uint32_t f32x8_to_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// One E4M3 byte as binary32 (NaN for 0x7F).
KVQ_DEVI float e4m3_to_f32(uint32_t byte) {
  return f16lo_to_f32(fp8x2_to_f16x2<KVQ_FMT_E4M3>(static_cast<uint16_t>(byte)));
}

KVQ_DEVI uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// ------------------------------------------------------------------ logits

// The attentions keep a row's running maximum as a raw dot product of scaled f16 queries and
// code * block scale, below 2^34, and its scale ls (to base-2 exponents) beside it: above 0, so
// that it times -inf stays -inf, and finite.
KVQ_DEVI float bounded_scale(float ls) { return fminf(fmaxf(ls, 0x1p-120f), 0x1p126f); }

// An output from its weighted sum o, inv = 1 / l (0 where l is), and the values' scale: in this order
// no intermediate leaves binary32's normal range before the output does.
KVQ_DEVI uint32_t output2(float o0, float o1, float inv, float sv) {
  return f32x2_to_bf16x2(o0 * inv * sv, o1 * inv * sv);
}

// States are merged on the maximum's exponent in units of 2^40: finite for every logit that a
// binary32 scale below 2^24 gives (and bf16 queries), where the exponent itself passes binary32.
constexpr float kMergeUnit = 0x1p40f;
KVQ_DEVI float merge_max(float m, float ls) { return m == -INFINITY ? m : m * (ls * (1.f / kMergeUnit)); }

// ------------------------------------------------------------------ visible pages

// The pages that hold a visible token of a sequence of L tokens seen from its
// last one: the first `sink` pages [0, sink), then [first, ceil(L / 16)).
struct Visible {
  int lo;     // first token of the window
  int sink;   // pages of the first tokens that lie before the window's first page
  int first;  // the window's first page
  int count;  // sink + the window's pages
};

KVQ_DEVI Visible visible(int window, int sinks, int L) {
  Visible v;
  v.lo = (window > 0 && L > window) ? L - window : 0;
  v.first = v.lo / kTok;
  const int s = sinks < v.lo ? sinks : v.lo;  // sinks inside the window add nothing
  const int sp = (s + kTok - 1) / kTok;
  v.sink = sp < v.first ? sp : v.first;
  v.count = L > 0 ? v.sink + (L + kTok - 1) / kTok - v.first : 0;
  return v;
}

}  // namespace fp4
}  // namespace kvq
