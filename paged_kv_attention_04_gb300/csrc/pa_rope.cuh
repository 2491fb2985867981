// Position rotation of q and k rows, and what the rotating writes share.
//
// A thread takes 16 numbers of a row, the two groups of 8 that hold 8 whole
// pairs: (8 j .., n/2 + 8 j ..) where a pair is (x_i, x_(i + n/2)), (16 j .., 16 j + 8 ..)
// where it is (x_2i, x_(2i+1)).  Either way its cosines are row[8 j ..] of the
// table and its sines row[n/2 + 8 j ..].  Products are rounded one by one
// (no FMA), so the result is that of the formula in float32 and does not
// depend on which kernel turned it.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

struct RopeParams {
  const int64_t* positions;
  const float* cos_sin;
  long long max_position;
  int size;   // n
  int pairs;  // PA_ROPE_PAIRS
};

inline RopeParams rope_params(const pa_rope* r) {
  return RopeParams{r->positions, r->cos_sin, r->max_position, r->rope_size, r->style == PA_ROPE_PAIRS};
}

// The table row of token t, null where its position is out of range (flagged).
__device__ __forceinline__ const float* rope_row(const RopeParams& r, int t, bool flag, int32_t* status) {
  const int64_t pos = __ldg(r.positions + t);
  if (pos < 0 || pos >= r.max_position) {
    if (flag) flag_error(status, PA_DEV_POSITION);
    return nullptr;
  }
  return r.cos_sin + pos * r.size;
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// 16 bytes that are read once: not kept in L1, where the table's rows are.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 w;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p));
  return w;
}

// 8 numbers as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = load_once(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void get(float (&x)[8]) const { Chunk<__nv_bfloat16>::unpack(w, x); }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    w = make_uint4(r[0], r[1], r[2], r[3]);
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    const uint4 u = load_once(p), v = load_once(p + 4);
    a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
    b = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// Offsets of thread j's two groups in a row, rotated over its first n numbers
// (j < n / 16) or not (the groups after them).
__device__ __forceinline__ void rope_groups(int j, int n, bool pairs, int& oa, int& ob) {
  if (j * 16 < n && !pairs) {
    oa = 8 * j;
    ob = n / 2 + 8 * j;
  } else {
    oa = 16 * j;
    ob = oa + 8;
  }
}

// Two numbers (word i of a group).
__device__ __forceinline__ float2 get2(const Eight<__nv_bfloat16>& e, int i) {
  const uint32_t w = i == 0 ? e.w.x : i == 1 ? e.w.y : i == 2 ? e.w.z : e.w.w;
  return make_float2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ void set2(Eight<__nv_bfloat16>& e, int i, float x, float y) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(w) : "f"(y), "f"(x));
  (i == 0 ? e.w.x : i == 1 ? e.w.y : i == 2 ? e.w.z : e.w.w) = w;
}
__device__ __forceinline__ float2 get2(const Eight<float>& e, int i) {
  return i == 0 ? make_float2(e.a.x, e.a.y) : i == 1 ? make_float2(e.a.z, e.a.w)
       : i == 2 ? make_float2(e.b.x, e.b.y) : make_float2(e.b.z, e.b.w);
}
__device__ __forceinline__ void set2(Eight<float>& e, int i, float x, float y) {
  float4& f = i < 2 ? e.a : e.b;
  if (i & 1) f.z = x, f.w = y;
  else f.x = x, f.y = y;
}

// Rotate thread j's groups by the table row, two pairs at a time (few registers).
template <typename T>
__device__ __forceinline__ void rope_turn(Eight<T>& ea, Eight<T>& eb, const float* row, int j, int n,
                                          bool pairs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 c = __ldg(reinterpret_cast<const float2*>(row + 8 * j) + i);
    const float2 s = __ldg(reinterpret_cast<const float2*>(row + n / 2 + 8 * j) + i);
    if (pairs) {
      // words 2 i, 2 i + 1 of the 16 numbers
      Eight<T>& e = i < 2 ? ea : eb;
      float2 x = get2(e, 2 * (i & 1)), y = get2(e, 2 * (i & 1) + 1);
      turn(x.x, x.y, c.x, s.x);
      turn(y.x, y.y, c.y, s.y);
      set2(e, 2 * (i & 1), x.x, x.y);
      set2(e, 2 * (i & 1) + 1, y.x, y.y);
    } else {
      float2 a = get2(ea, i), b = get2(eb, i);
      turn(a.x, b.x, c.x, s.x);
      turn(a.y, b.y, c.y, s.y);
      set2(ea, i, a.x, a.y);
      set2(eb, i, b.x, b.y);
    }
  }
}

}  // namespace pa
