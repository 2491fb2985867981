// The 4-bit cache (PA_INT4): page layout and conversions shared by the slot
// write, the read-back and the attention kernels.
//
// A page holds K (or V) of one 16-token block and one kv head, 10 D bytes in
// a row: 8 D bytes of codes, then an f16 scale s and zero z per token and
// group of 32 head dims.  Code c stands for (c s + z) x the tensor's scale.
// The order of the codes follows the fragments of the matrix instructions,
// so that a lane of the decode kernel loads its codes in one piece:
//   K  token t's D/2 bytes at t D/2; in them 4 runs of D/8 bytes, run c holding
//      a 32-bit word (8 codes, lowest nibble first) of dims 32 g + 8 c .. + 7
//      for every group g;
//      parameters of token t at 8 D + t D/8: the D/32 scales, then the zeros
//   V  tokens 2 p + 8 h and 2 p + 8 h + 1 share 32-bit words, the even token in
//      the low half: D/8 bytes at h 4 D + e D/2 + p D/8 hold dims e D/8 ..
//      + D/8 - 1 of both, four dims a word;
//      parameters of group g at 8 D + 64 g + 16 p: scales of tokens 2 p, 2 p + 1,
//      2 p + 8, 2 p + 9, then their zeros
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "pa_internal.h"

namespace pa {

template <int D>
struct I4Page {
  static constexpr int kGroups = D / 32;
  static constexpr int kCodeBytes = kBlockSize * D / 2;
  static constexpr int kBytes = kInt4PageBytesPerDim * D;
  static constexpr int kRun = D / 8;  // bytes of a run of K or V codes
  // K: word of dims 32 g + 8 c .. + 7 of token t; scale of group g (the zero
  // is kGroups f16 further)
  __host__ __device__ static constexpr int k_word(int t, int g, int c) {
    return t * (D / 2) + c * kRun + g * 4;
  }
  __host__ __device__ static constexpr int k_scale(int t, int g) {
    return kCodeBytes + t * kRun + g * 2;
  }
  // V: the 16 bits of dims d .. d + 3 (d % 4 == 0) of token t; scale of group g
  // (the zero is 4 f16 further)
  __host__ __device__ static constexpr int v_half(int t, int d) {
    return (t >> 3) * (4 * D) + (d / kRun) * (D / 2) + ((t & 7) >> 1) * kRun + ((d % kRun) >> 2) * 4 +
           (t & 1) * 2;
  }
  __host__ __device__ static constexpr int v_scale(int t, int g) {
    return kCodeBytes + g * 64 + ((t & 7) >> 1) * 16 + (t >> 3) * 4 + (t & 1) * 2;
  }
  static_assert(kCodeBytes + kBlockSize * kRun == kBytes, "codes and parameters fill the page");
};

// A constant the compiler keeps in a register (an instruction takes one constant,
// so a masked OR of two would become two instructions).
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  asm volatile("mov.u32 %0, %0;\n" : "+r"(x));
  return x;
}
struct I4Magic {
  uint32_t k1024, k64;  // 1024.0 and 64.0 in both halves
  __device__ __forceinline__ I4Magic() : k1024(opaque(0x64006400u)), k64(opaque(0x54005400u)) {}
};
// Two values c s + z in f16 from the nibbles 0 (ODD = 0) or 1 of both halves of w,
// rounded once.  The code in the low mantissa bits of 1024.0 (or from bit 4 on in
// those of 64.0) makes 1024 + c (64 + c), and the subtraction is exact: a masked
// OR, a subtraction and an FMA, without a shift.
template <int ODD>
__device__ __forceinline__ uint32_t int4_values(uint32_t w, uint32_t s, uint32_t z, const I4Magic& m) {
  uint32_t x, r;
  if constexpr (ODD) {
    asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;\n" : "=r"(x) : "r"(w), "r"(m.k64));
    asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(x) : "r"(x), "r"(0x54005400u));
  } else {
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;\n" : "=r"(x) : "r"(w), "r"(m.k1024));
    asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(x) : "r"(x), "r"(0x64006400u));
  }
  asm("fma.rn.f16x2 %0, %1, %2, %3;\n" : "=r"(r) : "r"(x), "r"(s), "r"(z));
  return r;
}

}  // namespace pa
