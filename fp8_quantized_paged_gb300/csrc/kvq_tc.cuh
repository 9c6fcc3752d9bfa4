// kvq_tc.cuh -- inline-PTX wrappers for the 5th-generation tensor cores
// (tcgen05: MMAs with accumulators in tensor memory) shared by the prefill
// and decode kernels.  sm_103a only.
//
// Shared-memory operands use the 128-byte swizzle: a tile is a stack of
// 128-byte rows, 8-row groups of 1024 bytes, and 16-byte chunk c of row r
// sits at chunk c ^ (r % 8) -- the layout a TMA box of 128-byte rows with
// CU_TENSOR_MAP_SWIZZLE_128B writes into a 1024-byte aligned destination.
#pragma once

#include "kvq_common.cuh"

namespace kvq {
namespace tc {

// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading
// and stride byte offsets (both multiples of 16), the Blackwell descriptor
// version bit (46) and the swizzle mode (2 = 128 B, bits 61-63).
//   K-major operand: the stride byte offset steps to the next 8-row group
//   (1024 for a dense tile); the leading byte offset is not used.
//   MN-major operand: the stride byte offset steps to the next 8 rows along
//   K, the leading byte offset to the next 128-byte span along M or N.
KVQ_DEVI uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// K-major, dense 8-row groups.
KVQ_DEVI uint64_t sw128_desc(uint32_t saddr) { return sw128_desc(saddr, 16, 1024); }

// The 64-byte swizzle of 64-byte rows: 8-row groups of 512 bytes, 16-byte chunk c of row r at
// c ^ (r / 2 % 4); swizzle mode 4.
KVQ_DEVI uint64_t sw64_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(512 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(4) << 61);
}

// Instruction descriptor of kind::f16: f32 accumulator, f16 A and B, both
// K-major unless transposed (bit 15 A, bit 16 B = MN-major), N and M.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// The same with bf16 A and B.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N) {
  return idesc_f16(M, N) | (1u << 7) | (1u << 10);
}

// 8-bit operand types of kind::f8f6f4.
constexpr uint32_t kTcE4M3 = 0, kTcE5M2 = 1;

KVQ_DEVI constexpr uint32_t tc_type(int fmt) { return fmt == KVQ_FMT_E5M2 ? kTcE5M2 : kTcE4M3; }

// Instruction descriptor of kind::f8f6f4: f32 accumulator, A and B types,
// transposes (MN-major) of A and B, N and M.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, uint32_t a_type, uint32_t b_type,
                                                bool a_mn, bool b_mn) {
  return (1u << 4) | (a_type << 7) | (b_type << 10) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

KVQ_DEVI void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A from tensor memory (M rows in the 128 lanes, K along the columns, two
// f16 per 32-bit column, the lower half the even k), B from shared memory.
KVQ_DEVI void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

KVQ_DEVI void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with 8-bit operands: four of A's values to a 32-bit column, the lowest byte the first k.
KVQ_DEVI void mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive once on bar when every tcgen05 operation this thread issued before
// has completed.
KVQ_DEVI void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               ::"r"(smem_u32(bar)) : "memory");
}

KVQ_DEVI void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
KVQ_DEVI void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Tensor-memory allocation by one whole warp: the address lands in *slot.
KVQ_DEVI void tmem_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
               ::"r"(smem_u32(slot)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

KVQ_DEVI void tmem_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
               : "memory");
}

// 16 (32) consecutive TMEM columns of this thread's lane (warp-collective).  The
// load and its wait are one asm statement, so that no use of the registers
// can be scheduled before the data has arrived.
KVQ_DEVI void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Store 4 consecutive columns of this thread's lane (no wait: several stores
// may be in flight; tmem_st_wait() completes them).
KVQ_DEVI void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
               ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

KVQ_DEVI void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
KVQ_DEVI void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Store 16 consecutive columns of this thread's lane and wait for it.
KVQ_DEVI void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n\t"
      "tcgen05.wait::st.sync.aligned;"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15])
      : "memory");
}

KVQ_DEVI void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

KVQ_DEVI void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
        "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
        "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
        "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])),
        "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])),
        "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])),
        "r"(__float_as_uint(v[17])), "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])),
        "r"(__float_as_uint(v[20])), "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])),
        "r"(__float_as_uint(v[23])), "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])),
        "r"(__float_as_uint(v[26])), "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])),
        "r"(__float_as_uint(v[29])), "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
      : "memory");
  tmem_st_wait();
}

KVQ_DEVI void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

KVQ_DEVI void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

KVQ_DEVI void sts8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

KVQ_DEVI uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}

// 64 consecutive TMEM columns of this thread's lane (warp-collective); the load and
// its wait are one statement, so that nothing uses the registers early.
KVQ_DEVI void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]),
        "=f"(v[1]),
        "=f"(v[2]),
        "=f"(v[3]),
        "=f"(v[4]),
        "=f"(v[5]),
        "=f"(v[6]),
        "=f"(v[7]),
        "=f"(v[8]),
        "=f"(v[9]),
        "=f"(v[10]),
        "=f"(v[11]),
        "=f"(v[12]),
        "=f"(v[13]),
        "=f"(v[14]),
        "=f"(v[15]),
        "=f"(v[16]),
        "=f"(v[17]),
        "=f"(v[18]),
        "=f"(v[19]),
        "=f"(v[20]),
        "=f"(v[21]),
        "=f"(v[22]),
        "=f"(v[23]),
        "=f"(v[24]),
        "=f"(v[25]),
        "=f"(v[26]),
        "=f"(v[27]),
        "=f"(v[28]),
        "=f"(v[29]),
        "=f"(v[30]),
        "=f"(v[31]),
        "=f"(v[32]),
        "=f"(v[33]),
        "=f"(v[34]),
        "=f"(v[35]),
        "=f"(v[36]),
        "=f"(v[37]),
        "=f"(v[38]),
        "=f"(v[39]),
        "=f"(v[40]),
        "=f"(v[41]),
        "=f"(v[42]),
        "=f"(v[43]),
        "=f"(v[44]),
        "=f"(v[45]),
        "=f"(v[46]),
        "=f"(v[47]),
        "=f"(v[48]),
        "=f"(v[49]),
        "=f"(v[50]),
        "=f"(v[51]),
        "=f"(v[52]),
        "=f"(v[53]),
        "=f"(v[54]),
        "=f"(v[55]),
        "=f"(v[56]),
        "=f"(v[57]),
        "=f"(v[58]),
        "=f"(v[59]),
        "=f"(v[60]),
        "=f"(v[61]),
        "=f"(v[62]),
        "=f"(v[63])
      : "r"(taddr)
      : "memory");
}

// Two binary32 values in a register pair: one instruction for both.
using f32x2 = unsigned long long;
KVQ_DEVI f32x2 f32x2_pack(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
KVQ_DEVI void f32x2_unpack(f32x2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
KVQ_DEVI f32x2 f32x2_fma(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
KVQ_DEVI f32x2 f32x2_add(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
KVQ_DEVI float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 8 consecutive columns of this thread's lane (no wait).
KVQ_DEVI void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// True in one lane of the (whole) warp.  Matrix instructions that the compiler sees issued
// under elect.sync cost 12 cycles each to issue, under lane == 0 they cost 52.
KVQ_DEVI bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

}  // namespace tc
}  // namespace kvq
