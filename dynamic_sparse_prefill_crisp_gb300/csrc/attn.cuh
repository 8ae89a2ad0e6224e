// Device building blocks of the prefill attention kernels (csrc/attention.cu,
// csrc/packed.cu): what follows a wait that ran out, the products of a 64-key
// sub-block, and the softmax arithmetic of 32 scores of a row.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace crisp {

constexpr float kOverflowSum = 0x1p64f;  // chunk row sum past which a row is redone

__device__ __forceinline__ void fail(int* abort, DevStatus* st, uint32_t where) {
  *reinterpret_cast<volatile int*>(abort) = 1;
  report_error(st, CRISP_ERR_TIMEOUT, where);
}

// p = 2^(s*c - m) for 32 scores of this thread's row: a packed FMA and a
// packed add per element pair, one MUFU per element. pk: bf16 pairs (even key
// low); sum += the fp32 sum of the 32 values.
__device__ __forceinline__ void p_exp32(const uint32_t (&sv)[32], float c, float neg_m, uint32_t (&pk)[16],
                                        float& sum) {
  float sa0 = 0.f, sa1 = 0.f, sb0 = 0.f, sb1 = 0.f;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    float x0, x1, x2, x3;
    ptx::ffma2(x0, x1, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]), c, c, neg_m, neg_m);
    ptx::ffma2(x2, x3, __uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3]), c, c, neg_m, neg_m);
    const float p0 = ptx::ex2_approx(x0), p1 = ptx::ex2_approx(x1), p2 = ptx::ex2_approx(x2), p3 = ptx::ex2_approx(x3);
    ptx::fadd2_acc(sa0, sa1, p0, p1);
    ptx::fadd2_acc(sb0, sb1, p2, p3);
    pk[e / 2] = ptx::pack_bf16x2(p0, p1);
    pk[e / 2 + 1] = ptx::pack_bf16x2(p2, p3);
  }
  sum += (sa0 + sa1) + (sb0 + sb1);
}

// S = Q K^T over 128 features as eight K = 16 products in one asm block:
// step kk reads A (Q) and B (K) at descriptor start addresses advanced by
// 2 (kk % 4) + (kk / 4) * a_half (resp. b_half) 16-byte units; the first
// step overwrites D. One predicate pair serves all eight.
template <uint32_t kAHalf, uint32_t kBHalf>
__device__ __forceinline__ void umma_qk_x8(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred f, t;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 f, %3, %3;\n\t"
      "setp.eq.b32 t, %3, %3;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, %4;\n\tadd.s64 b, %2, %5;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, %4 + 2;\n\tadd.s64 b, %2, %5 + 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, %4 + 4;\n\tadd.s64 b, %2, %5 + 4;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, %4 + 6;\n\tadd.s64 b, %2, %5 + 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}\n" ::"r"(d),
      "l"(da), "l"(db), "r"(idesc), "n"(kAHalf), "n"(kBHalf)
      : "memory");
}

// O += P V over 64 keys as four K = 16 products in one asm block: step kk
// reads P from TMEM column pa + 32 (kk / 2) + 8 (kk % 2) and V 16 keys
// (128 16-byte units) further on; the first step accumulates iff acc0.
__device__ __forceinline__ void umma_pv_x4(uint32_t d, uint32_t pa, uint64_t dv, uint32_t idesc, uint32_t acc0) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b32 ta;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, %3, %3;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.u32 ta, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], b, %3, t;\n\t"
      "add.u32 ta, %1, 32;\n\tadd.s64 b, %2, 256;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], b, %3, t;\n\t"
      "add.u32 ta, %1, 40;\n\tadd.s64 b, %2, 384;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], b, %3, t;\n\t}\n" ::"r"(d),
      "r"(pa), "l"(dv), "r"(idesc), "r"(acc0)
      : "memory");
}

// Largest of 32 raw scores.
__device__ __forceinline__ float max32(const uint32_t (&sv)[32]) {
  float ma = ptx::fmax3(__uint_as_float(sv[0]), __uint_as_float(sv[1]), __uint_as_float(sv[2]));
  float mb = ptx::fmax3(__uint_as_float(sv[3]), __uint_as_float(sv[4]), __uint_as_float(sv[5]));
#pragma unroll
  for (int e = 6; e + 3 < 32; e += 4) {
    ma = ptx::fmax3(ma, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
    mb = ptx::fmax3(mb, __uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3]));
  }
  return ptx::fmax3(ptx::fmax3(ma, mb, __uint_as_float(sv[30])), __uint_as_float(sv[31]), -INFINITY);
}

}  // namespace crisp
