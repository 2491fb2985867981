// The slot write with the position rotation on the way: q and k of each new token
// are rotated, q into its own tensor, k (and v as it is) into its paged slot.
//
// One pass: every number of q, k and v is read once and written once, where rotating
// first reads and writes q and k and then k and v again.  A thread takes 16 numbers
// of one row, or of two (32 bytes of bf16 each), D / 16 threads a row, 256 threads a CTA; the rows of a
// token are its q heads, then its k heads, then its v heads.  The table row of a token
// (4 n bytes) is read once per row through L1.
#include "pa_rope.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr long long kManyThreads = 1LL << 21;  // of one row each: above, a bf16 thread takes two (see below)

struct RopeWrite {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements
  void *q_out, *k_cache, *v_cache;
  const int64_t* slots;
  int num_tokens, q_rows, kv_rows;  // rows of a token: q heads, k (and v) heads
  long long num_slots;
  float k_scale, v_scale;
  int32_t* status;
  RopeParams rope;
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// E4M3 codes of 8 bf16 numbers over the scale, as the slot write forms them
__device__ __forceinline__ uint2 codes8(const Eight<__nv_bfloat16>& e, float scale) {
  float x[8];
  e.get(x);
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = e4m3x2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
  return make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
}

// kTimes rows a thread, their loads together.  Two are faster where the rows come from and go to DRAM (32768 tokens
// of 32 / 8 heads, D 128: 142 -> 124 us, 98 % of the copy bandwidth; 8192: 37.5 -> 36.1), one
// where they fit L2 (2048 tokens: 10.8 and 11.2 us; 4: 2.1 and 2.5), in FP8 (32768 tokens: 133 and
// 154) and in float32 (239 and 242), whose registers then leave fewer warps.
template <typename T, int D, bool F8, int kTimes>
__global__ void __launch_bounds__(kThreads, F8 ? 8 : 6) rope_write_kernel(const RopeWrite p) {
  launch_dependents();  // a following plan kernel may start; it waits for this grid
  constexpr int kLanes = D / 16;  // threads of a row
  const int j = threadIdx.x % kLanes;
  const unsigned g = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const unsigned rows = p.q_rows + 2 * p.kv_rows, step = (rows + kTimes - 1) / kTimes;
  const unsigned t = g / step;
  if (t >= static_cast<unsigned>(p.num_tokens)) return;
  const int row = static_cast<int>(g - t * step);
  const bool pairs = p.rope.pairs != 0;
  const int n = p.rope.size;
  const bool in_rope = j * 16 < n;
  auto kind_of = [&](int r) { return r < p.q_rows ? 0 : r < p.q_rows + p.kv_rows ? 1 : 2; };  // q, k, v
  auto offsets = [&](int kind, int& oa, int& ob) {
    oa = 16 * j, ob = oa + 8;
    if (kind != 2 && in_rope) rope_groups(j, n, pairs, oa, ob);
  };
  // (the numbers are on their way while the token's position and slot are looked up)
  Eight<T> a[kTimes], b[kTimes];
#pragma unroll
  for (int i = 0; i < kTimes; ++i) {
    const int r = row + i * step;
    if (kTimes > 1 && r >= static_cast<int>(rows)) break;
    const int kind = kind_of(r);
    const int head = kind == 0 ? r : r - p.q_rows - (kind == 2 ? p.kv_rows : 0);
    const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                   t * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride) + head * D;
    int oa, ob;
    offsets(kind, oa, ob);
    a[i].load(src + oa);
    b[i].load(src + ob);
  }
  const int64_t s = kTimes == 1 && row < p.q_rows ? 0 : __ldg(p.slots + t);
  const float* table = rope_row(p.rope, t, j == 0, p.status);
  if (!table) return;
#pragma unroll
  for (int i = 0; i < kTimes; ++i) {
    const int r = row + i * step;
    if (kTimes > 1 && r >= static_cast<int>(rows)) break;
    const int kind = kind_of(r);
    const int head = kind == 0 ? r : r - p.q_rows - (kind == 2 ? p.kv_rows : 0);
    if (kind != 0 && s >= p.num_slots && j == 0) flag_error(p.status, PA_DEV_SLOT_RANGE);
    if (kind != 0 && (s < 0 || s >= p.num_slots)) continue;
    int oa, ob;
    offsets(kind, oa, ob);
    if (kind != 2 && in_rope) rope_turn(a[i], b[i], table, j, n, pairs);
    if (kind == 0) {
      T* dst = static_cast<T*>(p.q_out) + (static_cast<long long>(t) * p.q_rows + head) * D;
      a[i].store(dst + oa);
      b[i].store(dst + ob);
      continue;
    }
    const long long at = (s * p.kv_rows + head) * D;
    void* cache = kind == 2 ? p.v_cache : p.k_cache;
    if constexpr (F8) {
      unsigned char* dst = static_cast<unsigned char*>(cache) + at;
      const float scale = kind == 2 ? p.v_scale : p.k_scale;
      *reinterpret_cast<uint2*>(dst + oa) = codes8(a[i], scale);
      *reinterpret_cast<uint2*>(dst + ob) = codes8(b[i], scale);
    } else {
      T* dst = static_cast<T*>(cache) + at;
      a[i].store(dst + oa);
      b[i].store(dst + ob);
    }
  }
}

template <typename T, int D, bool F8, int kTimes>
cudaError_t launch_times(const RopeWrite& p, cudaStream_t stream) {
  constexpr long long kRows = kThreads / (D / 16);
  const long long rows = static_cast<long long>(p.num_tokens) * ((p.q_rows + 2 * p.kv_rows + kTimes - 1) / kTimes);
  if (rows == 0) return cudaSuccess;
  rope_write_kernel<T, D, F8, kTimes>
      <<<static_cast<unsigned>((rows + kRows - 1) / kRows), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, int D, bool F8>
cudaError_t launch(const RopeWrite& p, cudaStream_t stream) {
  const long long threads = static_cast<long long>(p.num_tokens) * (p.q_rows + 2 * p.kv_rows) * (D / 16);
  if constexpr (sizeof(T) == 2 && !F8)
    if (threads >= kManyThreads) return launch_times<T, D, F8, 2>(p, stream);
  return launch_times<T, D, F8, 1>(p, stream);
}

}  // namespace

cudaError_t launch_rope_write(const RopeWriteArgs& a, const pa_layout& L, cudaStream_t stream) {
  RopeWrite p{a.q, a.k, a.v, a.q_stride, a.k_stride, a.v_stride, a.q_out, a.k_cache, a.v_cache,
              a.slots, a.num_tokens, a.q ? L.num_q_heads : 0, L.num_kv_heads,
              static_cast<long long>(L.num_blocks) * kBlockSize, L.k_scale, L.v_scale, a.status,
              rope_params(a.rope)};
  const bool d64 = L.head_size == 64;
  if (L.cache_dtype == PA_INT4) {
    // k and v by the 4-bit slot write's kernel, which quantises whole groups of a
    // row; q by the kernel above (32768 tokens of 32 / 8 heads, D 128: 170-180 us, 109 at the copy bandwidth; 2048: 18)
    p.kv_rows = 0;
    const cudaError_t e = d64 ? launch<__nv_bfloat16, 64, false>(p, stream)
                              : launch<__nv_bfloat16, 128, false>(p, stream);
    return e != cudaSuccess ? e : launch_rope_write_int4(a, L, stream);
  }
  if (L.dtype == PA_F32) return d64 ? launch<float, 64, false>(p, stream) : launch<float, 128, false>(p, stream);
  if (L.cache_dtype == PA_FP8_E4M3)
    return d64 ? launch<__nv_bfloat16, 64, true>(p, stream) : launch<__nv_bfloat16, 128, true>(p, stream);
  return d64 ? launch<__nv_bfloat16, 64, false>(p, stream) : launch<__nv_bfloat16, 128, false>(p, stream);
}

}  // namespace pa
