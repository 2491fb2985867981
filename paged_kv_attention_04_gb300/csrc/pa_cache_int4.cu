// Slot write into and read-back from a 4-bit cache (page layout: pa_int4.cuh).
//
// Write, for a group x of 32 head dims of a token: y = x / tensor scale,
// saturated at +-PA_INT4_LIMIT; z = f16(min y), s = f16((max y - min y) / 15);
// code = (y - z) / s rounded and clamped to 0 .. 15.  All of it in float32
// with IEEE division, so the codes are those of the definition.  The limit
// keeps z - 16 s, which the attention kernels form in f16, and c s + z finite:
// |z| + 16 s <= 16384 (1 + 32 / 15) < 65504.
//
// A thread holds 8 dims of a token's K and the same of V (one 16-byte chunk of
// each), four lanes a group: minimum and maximum by two shuffles each.  Both
// kernels move 2 D + 10 D / 16 bytes per token, head and tensor.
#include "pa_device.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 256;

// min / max that return NaN if either operand is one
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct Quantised {
  uint32_t codes;  // 8 codes, lowest nibble first
  __half s, z;     // of the group (the same in its four lanes)
};

// 8 values of a group held by four adjacent lanes (whole warp).
__device__ __forceinline__ Quantised quantise8(const uint4& w, float scale) {
  float y[8];
  Chunk<__nv_bfloat16>::unpack(w, y);
  if (scale != 1.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(y[i], scale);
  }
  constexpr float kLimit = PA_INT4_LIMIT;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = min_nan(max_nan(y[i], -kLimit), kLimit);
  float lo = y[0], hi = y[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, y[i]);
    hi = max_nan(hi, y[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  Quantised q;
  q.s = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
  q.z = __float2half_rn(lo);
  const float s = __half2float(q.s), z = __half2float(q.z);
  q.codes = 0;
  if (s > 0.f) {  // not for a group of equal values, nor for one with a NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = __float2int_rn(__fdiv_rn(y[i] - z, s));
      q.codes |= static_cast<uint32_t>(min(max(c, 0), 15)) << (4 * i);
    }
  }
  return q;
}

// bf16 pair of (c s + z) x scale for nibbles i and i + 1 of `codes`
__device__ __forceinline__ uint32_t dequantise2(uint32_t codes, int i, float s, float z, float scale) {
  const float a = fmaf(static_cast<float>((codes >> (4 * i)) & 15u), s, z) * scale;
  const float b = fmaf(static_cast<float>((codes >> (4 * i + 4)) & 15u), s, z) * scale;
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, __half s, __half z, float scale) {
  const float sf = __half2float(s), zf = __half2float(z);
  return make_uint4(dequantise2(codes, 0, sf, zf, scale), dequantise2(codes, 2, sf, zf, scale),
                    dequantise2(codes, 4, sf, zf, scale), dequantise2(codes, 6, sf, zf, scale));
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_write_int4_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v, const int64_t* __restrict__ slots,
    int num_tokens, unsigned char* __restrict__ k_cache, unsigned char* __restrict__ v_cache,
    int num_kv_heads, long long num_slots, float k_scale, float v_scale, int32_t* status) {
  using Pg = I4Page<D>;
  launch_dependents();  // a following plan kernel may start; it waits for this grid
  const int row_chunks = num_kv_heads * (D / 8);
  const long long total = static_cast<long long>(num_tokens) * row_chunks;
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  // whole warps run the loop (the group's lanes exchange values)
  for (long long i0 = blockIdx.x * static_cast<long long>(kThreads) + (threadIdx.x & ~31u); i0 < total;
       i0 += stride) {
    const long long i = i0 + (threadIdx.x & 31);
    const long long t = i / row_chunks;
    const int c = static_cast<int>(i - t * row_chunks);
    int64_t s = i < total ? __ldg(slots + t) : -1;
    if (s >= num_slots) {
      if (c == 0) flag_error(status, PA_DEV_SLOT_RANGE);
      s = -1;
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const Quantised qk = quantise8(s >= 0 ? __ldg(k + i) : zero, k_scale);
    const Quantised qv = quantise8(s >= 0 ? __ldg(v + i) : zero, v_scale);
    if (s < 0) continue;
    const int head = c / (D / 8), d = (c - head * (D / 8)) * 8;
    const int row = static_cast<int>(s % kBlockSize), g = d / 32;
    const long long page = ((s / kBlockSize) * num_kv_heads + head) * Pg::kBytes;
    unsigned char* kp = k_cache + page;
    unsigned char* vp = v_cache + page;
    *reinterpret_cast<uint32_t*>(kp + Pg::k_word(row, g, (d % 32) / 8)) = qk.codes;
    *reinterpret_cast<uint16_t*>(vp + Pg::v_half(row, d)) = static_cast<uint16_t>(qv.codes);
    *reinterpret_cast<uint16_t*>(vp + Pg::v_half(row, d + 4)) = static_cast<uint16_t>(qv.codes >> 16);
    if (d % 32 == 0) {
      __half* kq = reinterpret_cast<__half*>(kp + Pg::k_scale(row, g));
      kq[0] = qk.s;
      kq[Pg::kGroups] = qk.z;
      __half* vq = reinterpret_cast<__half*>(vp + Pg::v_scale(row, g));
      vq[0] = qv.s;
      vq[4] = qv.z;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_int4_kernel(
    const unsigned char* __restrict__ k_cache, const unsigned char* __restrict__ v_cache,
    const int64_t* __restrict__ slots, int num_tokens, uint4* __restrict__ k, uint4* __restrict__ v,
    int num_kv_heads, long long num_slots, float k_scale, float v_scale, int32_t* status) {
  using Pg = I4Page<D>;
  const int row_chunks = num_kv_heads * (D / 8);
  const long long total = static_cast<long long>(num_tokens) * row_chunks;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long t = i / row_chunks;
    const int c = static_cast<int>(i - t * row_chunks);
    const int64_t s = __ldg(slots + t);
    if (s < 0) continue;
    if (s >= num_slots) {
      if (c == 0) flag_error(status, PA_DEV_SLOT_RANGE);
      continue;
    }
    const int head = c / (D / 8), d = (c - head * (D / 8)) * 8;
    const int row = static_cast<int>(s % kBlockSize), g = d / 32;
    const long long page = ((s / kBlockSize) * num_kv_heads + head) * Pg::kBytes;
    const unsigned char* kp = k_cache + page;
    const unsigned char* vp = v_cache + page;
    const uint32_t kw = __ldg(reinterpret_cast<const uint32_t*>(kp + Pg::k_word(row, g, (d % 32) / 8)));
    const uint32_t v0 = __ldg(reinterpret_cast<const uint16_t*>(vp + Pg::v_half(row, d)));
    const uint32_t v1 = __ldg(reinterpret_cast<const uint16_t*>(vp + Pg::v_half(row, d + 4)));
    const __half* kq = reinterpret_cast<const __half*>(kp + Pg::k_scale(row, g));
    const __half* vq = reinterpret_cast<const __half*>(vp + Pg::v_scale(row, g));
    k[i] = dequantise8(kw, kq[0], kq[Pg::kGroups], k_scale);
    v[i] = dequantise8(v0 | (v1 << 16), vq[0], vq[4], v_scale);
  }
}

unsigned grid_for(int num_tokens, int num_kv_heads, int head_size) {
  const long long total = static_cast<long long>(num_tokens) * num_kv_heads * (head_size / 8);
  const long long blocks = (total + kThreads - 1) / kThreads;
  return static_cast<unsigned>(blocks > 65535LL * 64 ? 65535LL * 64 : blocks);
}

}  // namespace

cudaError_t launch_cache_write_int4(const void* k, const void* v, const int64_t* slot_mapping,
                                    int num_tokens, void* k_cache, void* v_cache, int num_kv_heads,
                                    int head_size, long long num_slots, float k_scale,
                                    float v_scale, int32_t* status, cudaStream_t stream) {
  auto go = [&](auto kernel) {
    kernel<<<grid_for(num_tokens, num_kv_heads, head_size), kThreads, 0, stream>>>(
        static_cast<const uint4*>(k), static_cast<const uint4*>(v), slot_mapping, num_tokens,
        static_cast<unsigned char*>(k_cache), static_cast<unsigned char*>(v_cache), num_kv_heads,
        num_slots, k_scale, v_scale, status);
    return cudaGetLastError();
  };
  return head_size == 64 ? go(cache_write_int4_kernel<64>) : go(cache_write_int4_kernel<128>);
}

cudaError_t launch_cache_read_int4(const void* k_cache, const void* v_cache,
                                   const int64_t* slot_mapping, int num_tokens, void* k, void* v,
                                   int num_kv_heads, int head_size, long long num_slots,
                                   float k_scale, float v_scale, int32_t* status,
                                   cudaStream_t stream) {
  auto go = [&](auto kernel) {
    kernel<<<grid_for(num_tokens, num_kv_heads, head_size), kThreads, 0, stream>>>(
        static_cast<const unsigned char*>(k_cache), static_cast<const unsigned char*>(v_cache),
        slot_mapping, num_tokens, static_cast<uint4*>(k), static_cast<uint4*>(v), num_kv_heads,
        num_slots, k_scale, v_scale, status);
    return cudaGetLastError();
  };
  return head_size == 64 ? go(cache_read_int4_kernel<64>) : go(cache_read_int4_kernel<128>);
}

}  // namespace pa
