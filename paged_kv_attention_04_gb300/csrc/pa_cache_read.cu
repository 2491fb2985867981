// Read-back of cache slots: the reverse of the slot write for caches of rows.
//
// Slot s names one contiguous row of Hkv*D elements, so a bf16 or fp32
// read-back is a row copy in 16-byte chunks, as the write is.  From an FP8
// cache a thread turns 8 codes into 8 bf16 values, code x scale rounded once.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {
// Two E4M3 codes (low byte first) -> bf16 pair of code x scale.  A code is
// exact in f16 and in float32; the product rounds in float32, then to bf16.
__device__ __forceinline__ uint32_t dequantize2_e4m3(uint32_t codes16, float scale) {
  uint32_t h, r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(static_cast<uint16_t>(codes16)));
  float lo, hi;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}\n"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi * scale), "f"(lo * scale));
  return r;
}
__device__ __forceinline__ uint4 dequantize8_e4m3(const uint2& c, float scale) {
  return make_uint4(dequantize2_e4m3(c.x & 0xffffu, scale), dequantize2_e4m3(c.x >> 16, scale),
                    dequantize2_e4m3(c.y & 0xffffu, scale), dequantize2_e4m3(c.y >> 16, scale));
}

// One thread a 16-byte chunk of the output rows of K and V.
template <bool F8>
__global__ void __launch_bounds__(256) cache_read_kernel(
    const void* __restrict__ k_cache, const void* __restrict__ v_cache,
    const int64_t* __restrict__ slots, int num_tokens, uint4* __restrict__ k, uint4* __restrict__ v,
    int row_chunks, long long num_slots, float k_scale, float v_scale, int32_t* status) {
  const long long total = static_cast<long long>(num_tokens) * row_chunks;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long t = i / row_chunks;
    const int c = static_cast<int>(i - t * row_chunks);
    const int64_t s = __ldg(slots + t);
    if (s < 0) continue;
    if (s >= num_slots) {
      if (c == 0) flag_error(status, PA_DEV_SLOT_RANGE);
      continue;
    }
    const long long src = s * row_chunks + c;
    if constexpr (F8) {
      k[i] = dequantize8_e4m3(__ldg(static_cast<const uint2*>(k_cache) + src), k_scale);
      v[i] = dequantize8_e4m3(__ldg(static_cast<const uint2*>(v_cache) + src), v_scale);
    } else {
      k[i] = __ldg(static_cast<const uint4*>(k_cache) + src);
      v[i] = __ldg(static_cast<const uint4*>(v_cache) + src);
    }
  }
}

template <bool F8>
cudaError_t launch(const void* k_cache, const void* v_cache, const int64_t* slot_mapping,
                   int num_tokens, void* k, void* v, int row_bytes, long long num_slots,
                   float k_scale, float v_scale, int32_t* status, cudaStream_t stream) {
  const int row_chunks = row_bytes / 16;
  const long long total = static_cast<long long>(num_tokens) * row_chunks;
  const int threads = 256;
  long long blocks = (total + threads - 1) / threads;
  if (blocks > 65535LL * 64) blocks = 65535LL * 64;
  cache_read_kernel<F8><<<static_cast<unsigned>(blocks), threads, 0, stream>>>(
      k_cache, v_cache, slot_mapping, num_tokens, static_cast<uint4*>(k), static_cast<uint4*>(v),
      row_chunks, num_slots, k_scale, v_scale, status);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_cache_read(const void* k_cache, const void* v_cache, const int64_t* slot_mapping,
                              int num_tokens, void* k, void* v, int row_bytes, long long num_slots,
                              int32_t* status, cudaStream_t stream) {
  return launch<false>(k_cache, v_cache, slot_mapping, num_tokens, k, v, row_bytes, num_slots, 1.f,
                       1.f, status, stream);
}

cudaError_t launch_cache_read_fp8(const void* k_cache, const void* v_cache,
                                  const int64_t* slot_mapping, int num_tokens, void* k, void* v,
                                  int row_bytes, long long num_slots, float k_scale, float v_scale,
                                  int32_t* status, cudaStream_t stream) {
  return launch<true>(k_cache, v_cache, slot_mapping, num_tokens, k, v, row_bytes, num_slots,
                      k_scale, v_scale, status, stream);
}

}  // namespace pa
