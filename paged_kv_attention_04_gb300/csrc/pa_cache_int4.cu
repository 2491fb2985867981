// Slot write into and read-back from a 4-bit cache (page layout: pa_int4.cuh).
//
// Write, for a group x of 32 head dims of a token: y = x / tensor scale,
// saturated at +-PA_INT4_LIMIT; z = f16(min y), s = f16((max y - min y) / 15);
// code = (y - z) / s rounded and clamped to 0 .. 15.  All of it in float32
// with IEEE division, so the codes are those of the definition.  The limit
// keeps c s + z, which the attention kernels form in f16, finite whatever the
// rounding of s and z: |z| + 15 s <= 3 x 16384 (1 + 2^-10) < 65504.
//
// Both kernels move 2 D + 10 D / 16 bytes per token, head and tensor and are bound
// by HBM if a value costs few instructions:
//   write  minimum and maximum on packed bf16 pairs; codes by one FMA each,
//          t = d r + 1.5 2^23 with d = y - z and r = 1/s, whose low bits are the code.
//          The residual d - c s decides: below s/2 by more than the rounding of r and
//          of a division can move it, c is what IEEE division rounds to; a group
//          with a value nearer a tie takes the division itself, as do groups that
//          saturate, hold a NaN or need clamped codes;
//   read   a masked nibble is an f16 subnormal, c 2^-24 or c 2^-20; widened to float32
//          it enters fma(c 2^-24, s 2^24, z), the same value.
// Measured, 8 heads of 128: 32768 tokens written in 60 us (2.9 TB/s, bound by
// instruction issue), read in 34 us, 131072 read in 132 us (5.3 TB/s).
// A warp takes a pair of tokens (2 i, 2 i + 1 of the call) of one head (two heads at
// D = 64), a lane 8 dims; a CTA's 8 warps take 16 tokens, so the V words and sectors
// that two and four tokens of a block share are touched at about the same time.
#include <cmath>

#include "pa_device.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"
#include "pa_rope.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 16;  // of a CTA
constexpr unsigned kCtas = 8 * 152;     // a full GPU of CTAs

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {  // bf16 pairs
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// x / tensor scale in float32; a power of two divides by an exact multiplication
struct TensorScale {
  float scale, inv;  // inv = 1 / scale
  bool exact;        // scale is a power of two, and so is inv
  __device__ __forceinline__ float divide(float x) const {
    return exact ? x * inv : __fdiv_rn(x, scale);
  }
};

struct Quantised {
  uint32_t codes;  // 8 codes, lowest nibble first
  uint32_t sz;     // s and z (high half) of the group, f16
};

// 8 values of a group held by four adjacent lanes (whole warp).
__device__ __forceinline__ Quantised quantise8(const uint4& w, const TensorScale& ts) {
  uint32_t mn = min2_nan(min2_nan(w.x, w.y), min2_nan(w.z, w.w));
  uint32_t mx = max2_nan(max2_nan(w.x, w.y), max2_nan(w.z, w.w));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = min2_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = max2_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  mn = min2_nan(mn, mn >> 16);  // (the high half of the shifted word is +0: unused)
  mx = max2_nan(mx, mx >> 16);
  constexpr float kLimit = PA_INT4_LIMIT;
  constexpr float kRound = 12582912.f;  // 1.5 2^23: added, leaves the nearest integer in the low bits
  float lo = ts.divide(bf16_lo(mn)), hi = ts.divide(bf16_lo(mx));  // division keeps order
  float x[8];
  Chunk<__nv_bfloat16>::unpack(w, x);
  const bool plain = lo >= -kLimit && hi <= kLimit;  // false for NaN
  const bool nan = lo != lo;
  lo = fminf(fmaxf(lo, -kLimit), kLimit);
  hi = fminf(fmaxf(hi, -kLimit), kLimit);
  const __half sh = __float2half_rn(__fdiv_rn(hi - lo, 15.f)), zh = __float2half_rn(lo);
  const float s = __half2float(sh), z = __half2float(zh);
  Quantised q;
  q.sz = nan ? 0x7fff7fffu
             : static_cast<uint32_t>(__half_as_ushort(sh)) | (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
  q.codes = 0;
  if (nan || s == 0.f) return q;
  const float r = __frcp_rn(s);
  bool exact = plain && (lo - z) * r > -0.499f && (hi - z) * r < 15.499f;  // no code to clamp
  if (exact) {
    float worst = 0.f;
    // the sum of the constant's bits at every nibble
    uint32_t codes = 0u - (0x4b400000u + (0x4b400000u << 4) + (0x4b400000u << 8));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = ts.exact ? fmaf(x[i], ts.inv, -z) : __fdiv_rn(x[i], ts.scale) - z;
      const float t = fmaf(d, r, kRound);
      worst = fmaxf(worst, fabsf(fmaf(kRound - t, s, d)));
      codes += __float_as_uint(t) << (4 * i);
    }
    // r is off by 2^-24 of itself and so is a division: 15 x 2^-23 of s together
    const float near = s * (0.5f - 0x1p-18f);
    exact = worst < near;
    if (!exact) {
      // exact ties go to the even code; anything else that near takes the division
      exact = true;
      codes = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = ts.exact ? fmaf(x[i], ts.inv, -z) : __fdiv_rn(x[i], ts.scale) - z;
        const float t = fmaf(d, r, kRound);
        const float e = fmaf(kRound - t, s, d);
        uint32_t c = __float_as_uint(t) & 15u;
        if (fabsf(e) == 0.5f * s) c = (c & 1) ? (e > 0.f ? c + 1 : c - 1) : c;
        else if (fabsf(e) >= near) exact = false;
        codes |= c << (4 * i);
      }
    }
    q.codes = codes;
  }
  if (!exact) {
    q.codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = fminf(fmaxf(ts.divide(x[i]), -kLimit), kLimit);
      const int c = __float2int_rn(__fdiv_rn(y - z, s));
      q.codes |= static_cast<uint32_t>(min(max(c, 0), 15)) << (4 * i);
    }
  }
  return q;
}

// Two floats -> packed bf16 pair
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (c s + z) x scale of 8 codes, rounded to bf16
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, float s, float z, float scale) {
  const uint32_t high = codes >> 8;
  const uint32_t pairs[4] = {codes & 0x000f000fu, codes & 0x00f000f0u, high & 0x000f000fu,
                             high & 0x00f000f0u};  // nibbles n and n + 4
  const float s24 = s * 16777216.f, s20 = s * 1048576.f;
  float v[8];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&pairs[n]));
    const float sn = (n & 1) ? s20 : s24;
    v[n] = fmaf(c.x, sn, z);
    v[n + 4] = fmaf(c.y, sn, z);
  }
  if (scale != 1.f) {
#pragma unroll
    for (int n = 0; n < 8; ++n) v[n] *= scale;
  }
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                    pack_bf16(v[6], v[7]));
}

// Where a lane works: 8 dims from d of one token of the warp's pair and of one of
// its heads.
template <int D>
struct Place {
  static constexpr int kLanes = D / 8;             // of a row
  static constexpr int kHeads = 32 / (2 * kLanes); // of a warp
  int lane, d, head0;
  long long token;
  __device__ __forceinline__ Place() {
    lane = threadIdx.x & 31;
    d = (lane % kLanes) * 8;
    token = blockIdx.x * static_cast<long long>(kTokens) + (threadIdx.x >> 5) * 2 + (lane / kLanes) % 2;
    head0 = blockIdx.y * kHeads + lane / (2 * kLanes);
  }
};

// What the rotating write adds: the rotation, and token strides of k and v (in 16-byte words).
struct Turned {
  RopeParams rope;
  long long k_stride, v_stride;
};

// 8 dims from d of a row of k, rotated by the table row: each lane loads the
// group that holds the partners of its own too.
__device__ __forceinline__ uint4 load_turned(const uint4* row, int d, const float* table,
                                             const RopeParams& r) {
  Eight<__nv_bfloat16> own, other;
  own.w = __ldg(row + d / 8);
  if (d >= r.size) return own.w;
  const int half = r.size / 2;
  if (r.pairs) {
    // (the group's four pairs: the lower or upper half of the 16 numbers of thread d / 16)
    float x[8], c[8], s[8];
    own.get(x);
    load8(table + (d / 16) * 8, c);
    load8(table + half + (d / 16) * 8, s);
    const bool up = (d / 8) & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], up ? c[4 + i] : c[i], up ? s[4 + i] : s[i]);
    own.set(x);
    return own.w;
  }
  const bool up = d >= half;
  other.w = __ldg(row + (up ? d - half : d + half) / 8);
  const int j = (up ? d - half : d) / 8;
  if (up) {
    rope_turn(other, own, table, j, r.size, false);
  } else {
    rope_turn(own, other, table, j, r.size, false);
  }
  return own.w;
}

// TURN: k is rotated as it is read.
template <int D, bool TURN>
__global__ void __launch_bounds__(kThreads) cache_write_int4_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v, const int64_t* __restrict__ slots,
    int num_tokens, unsigned char* __restrict__ k_cache, unsigned char* __restrict__ v_cache,
    int num_kv_heads, long long num_slots, TensorScale ks, TensorScale vs, int32_t* status,
    const Turned turned) {
  using Pg = I4Page<D>;
  using Pl = Place<D>;
  launch_dependents();  // a following plan kernel may start; it waits for this grid
  const Pl at;
  int64_t s = at.token < num_tokens ? __ldg(slots + at.token) : -1;
  const float* table = nullptr;
  if constexpr (TURN) {
    if (at.token < num_tokens) table = rope_row(turned.rope, static_cast<int>(at.token), at.d == 0, status);
    if (!table) s = -1;
  }
  if (s >= num_slots) {
    if (at.d == 0) flag_error(status, PA_DEV_SLOT_RANGE);
    s = -1;
  }
  // the pair fills whole V words if it sits in an even slot and the next
  const int64_t other = __shfl_xor_sync(0xffffffffu, s, Pl::kLanes);
  const bool odd = (at.lane / Pl::kLanes) % 2;
  const bool joined = s >= 0 && (s & 1) == odd && other == s + (odd ? -1 : 1);
  const int row = static_cast<int>(s & (kBlockSize - 1)), g = at.d / 32;
  const int step = gridDim.y * Pl::kHeads;
  const uint4* kr = k + at.token * (TURN ? turned.k_stride : num_kv_heads * Pl::kLanes) + (TURN ? 0 : at.d / 8);
  const uint4* vr = v + at.token * (TURN ? turned.v_stride : num_kv_heads * Pl::kLanes) + at.d / 8;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load = [&](int head, uint4& kw, uint4& vw) {
    const bool ok = s >= 0 && head < num_kv_heads;
    if constexpr (TURN) kw = ok ? load_turned(kr + head * Pl::kLanes, at.d, table, turned.rope) : zero;
    else kw = ok ? __ldg(kr + head * Pl::kLanes) : zero;
    vw = ok ? __ldg(vr + head * Pl::kLanes) : zero;
  };
  uint4 kw, vw, kw1, vw1;  // this head's values, the next one's
  load(at.head0, kw, vw);
  for (int h0 = 0; h0 < num_kv_heads; h0 += step, kw = kw1, vw = vw1) {  // whole warps
    const int head = h0 + at.head0;
    const bool ok = s >= 0 && head < num_kv_heads;
    load(head + step, kw1, vw1);
    const Quantised qk = quantise8(kw, ks);
    const Quantised qv = quantise8(vw, vs);
    const uint32_t other_codes = __shfl_xor_sync(0xffffffffu, qv.codes, Pl::kLanes);
    const uint32_t other_sz = __shfl_xor_sync(0xffffffffu, qv.sz, Pl::kLanes);
    if (!ok) continue;
    const long long page = ((s / kBlockSize) * num_kv_heads + head) * Pg::kBytes;
    unsigned char* kp = k_cache + page;
    unsigned char* vp = v_cache + page;
    *reinterpret_cast<uint32_t*>(kp + Pg::k_word(row, g, (at.d % 32) / 8)) = qk.codes;
    if (at.d % 32 == 0) {
      uint16_t* kq = reinterpret_cast<uint16_t*>(kp + Pg::k_scale(row, g));
      kq[0] = static_cast<uint16_t>(qk.sz);
      kq[Pg::kGroups] = static_cast<uint16_t>(qk.sz >> 16);
    }
    if (joined) {
      // the even token's lane writes the word of dims d .. d + 3 and the scales,
      // the odd token's the word of d + 4 .. d + 7 and the zeros
      const int t = row & ~1;
      *reinterpret_cast<uint32_t*>(vp + Pg::v_half(t, at.d + (odd ? 4 : 0))) =
          odd ? __byte_perm(other_codes, qv.codes, 0x7632) : __byte_perm(qv.codes, other_codes, 0x5410);
      if (at.d % 32 == 0)
        *reinterpret_cast<uint32_t*>(vp + Pg::v_scale(t, g) + (odd ? 8 : 0)) =
            odd ? __byte_perm(other_sz, qv.sz, 0x7632) : __byte_perm(qv.sz, other_sz, 0x5410);
    } else {
      *reinterpret_cast<uint16_t*>(vp + Pg::v_half(row, at.d)) = static_cast<uint16_t>(qv.codes);
      *reinterpret_cast<uint16_t*>(vp + Pg::v_half(row, at.d + 4)) = static_cast<uint16_t>(qv.codes >> 16);
      if (at.d % 32 == 0) {
        uint16_t* vq = reinterpret_cast<uint16_t*>(vp + Pg::v_scale(row, g));
        vq[0] = static_cast<uint16_t>(qv.sz);
        vq[4] = static_cast<uint16_t>(qv.sz >> 16);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_int4_kernel(
    const unsigned char* __restrict__ k_cache, const unsigned char* __restrict__ v_cache,
    const int64_t* __restrict__ slots, int num_tokens, uint4* __restrict__ k, uint4* __restrict__ v,
    int num_kv_heads, long long num_slots, float k_scale, float v_scale, int32_t* status) {
  using Pg = I4Page<D>;
  using Pl = Place<D>;
  const Pl at;
  if (at.token >= num_tokens) return;
  const int64_t s = __ldg(slots + at.token);
  if (s < 0) return;
  if (s >= num_slots) {
    if (at.d == 0) flag_error(status, PA_DEV_SLOT_RANGE);
    return;
  }
  const int row = static_cast<int>(s & (kBlockSize - 1)), g = at.d / 32;
  const uint32_t half = (row & 1) ? 0x7632u : 0x5410u;  // the token's half of two V words
#pragma unroll 1
  for (int head = at.head0; head < num_kv_heads; head += gridDim.y * Pl::kHeads) {
    const long long page = ((s / kBlockSize) * num_kv_heads + head) * Pg::kBytes;
    const unsigned char* kp = k_cache + page;
    const unsigned char* vp = v_cache + page;
    const uint32_t kw = __ldg(reinterpret_cast<const uint32_t*>(kp + Pg::k_word(row, g, (at.d % 32) / 8)));
    const uint2 vw = __ldg(reinterpret_cast<const uint2*>(vp + Pg::v_half(row & ~1, at.d)));
    const __half* kq = reinterpret_cast<const __half*>(kp + Pg::k_scale(row, g));
    const __half* vq = reinterpret_cast<const __half*>(vp + Pg::v_scale(row, g));
    const __half k_s = __ldg(kq), k_z = __ldg(kq + Pg::kGroups), v_s = __ldg(vq), v_z = __ldg(vq + 4);
    const long long dst = (at.token * num_kv_heads + head) * Pl::kLanes + at.d / 8;
    k[dst] = dequantise8(kw, __half2float(k_s), __half2float(k_z), k_scale);
    v[dst] = dequantise8(__byte_perm(vw.x, vw.y, half), __half2float(v_s), __half2float(v_z), v_scale);
  }
}

TensorScale tensor_scale(float scale) {
  int e;
  const float inv = 1.f / scale;
  // (a subnormal scale's inverse is infinite: divided)
  return TensorScale{scale, inv, std::frexp(scale, &e) == 0.5f && std::isfinite(inv) && inv >= 0x1p-126f};
}

// CTAs of 16 tokens, their heads dealt out over more CTAs only as far as that
// fills the GPU: a CTA with all heads reads and writes whole rows (131072 tokens
// of 8 heads read: 132 us; one head a CTA took half as long again, 207 us).
dim3 grid_for(int num_tokens, int num_kv_heads, int head_size) {
  const unsigned x = static_cast<unsigned>((num_tokens + kTokens - 1) / kTokens);
  const unsigned heads = head_size == 64 ? 2 : 1;  // a warp's
  const unsigned most = (static_cast<unsigned>(num_kv_heads) + heads - 1) / heads;
  const unsigned want = (kCtas + x - 1) / x;
  const unsigned y = want < most ? want : most;
  return dim3(x, y < 65535u ? y : 65535u);
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
        num_slots, tensor_scale(k_scale), tensor_scale(v_scale), status, Turned{});
    return cudaGetLastError();
  };
  return head_size == 64 ? go(cache_write_int4_kernel<64, false>) : go(cache_write_int4_kernel<128, false>);
}

cudaError_t launch_rope_write_int4(const RopeWriteArgs& a, const pa_layout& L, cudaStream_t stream) {
  const Turned turned{rope_params(a.rope), a.k_stride / 8, a.v_stride / 8};
  auto go = [&](auto kernel) {
    kernel<<<grid_for(a.num_tokens, L.num_kv_heads, L.head_size), kThreads, 0, stream>>>(
        static_cast<const uint4*>(a.k), static_cast<const uint4*>(a.v), a.slots, a.num_tokens,
        static_cast<unsigned char*>(a.k_cache), static_cast<unsigned char*>(a.v_cache),
        L.num_kv_heads, static_cast<long long>(L.num_blocks) * kBlockSize, tensor_scale(L.k_scale),
        tensor_scale(L.v_scale), a.status, turned);
    return cudaGetLastError();
  };
  return L.head_size == 64 ? go(cache_write_int4_kernel<64, true>) : go(cache_write_int4_kernel<128, true>);
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
