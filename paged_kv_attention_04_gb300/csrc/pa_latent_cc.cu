// Latent attention on the CUDA cores, absorbed and expanded: fp32 (whose 1e-5 needs fp32
// products).
//
// Absorbed: a warp takes one head of one new token, a CTA eight heads that read the same
// keys, staged a 16-token block at a time; every key costs a dot product over the lanes
// (R + 64 products, five shuffles) and an update of R sums, held by the lanes.  The running
// maximum and sum of the softmax move with every block, so the keys are read once.  A request's
// keys are cut into `splits` pieces so that few requests fill the GPU; a second kernel
// joins the pieces in order.  Bound by instruction issue: a key costs five shuffles that wait for one another.
// Expanded: the same with a warp per (token, head) and that head's own keys.
//
// Measured: absorbed (R = 512) 32 decodes of 16 heads over 1024 keys 116 us, 256 of 32 heads 1290 us (14 TFLOP/s),
// 2 of 16 heads over 32768 keys 244 us; expanded (D = 128) 512 tokens of 16 heads 268 us, 2048 of 32
// heads 6.0 ms (7 TFLOP/s).
#include <math_constants.h>

#include "pa_device.cuh"
#include "pa_latent.h"

namespace pa {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The request of row t: the last r with qsl[r] <= t (the array is nondecreasing; where it
// is not, the check below refuses the step).
__device__ __forceinline__ int request_of(const int32_t* qsl, int num_seqs, int t) {
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(qsl + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Whether a start array is 0-based, nondecreasing and ends at `end` (whole CTA).
__device__ bool starts_ok(const int32_t* starts, int n, int end) {
  bool bad = threadIdx.x == 0 && (__ldg(starts) != 0 || __ldg(starts + n) != end);
  for (int r = threadIdx.x; r < n; r += blockDim.x) bad |= __ldg(starts + r) > __ldg(starts + r + 1);
  return !__syncthreads_or(bad);
}

// one key's logit x (base 2) into a running softmax; returns the key's weight,
// `old` the factor of what was summed before
__device__ __forceinline__ float softmax_step(float x, float& m, float& l, float& old) {
  const float nm = fmaxf(m, x);  // (a NaN leaves the maximum as it is)
  old = m == nm ? 1.f : exp2f(m - nm);
  // no finite logit yet: against 0, so that -inf weighs 0 (such logits alone: 0 / 0 at the end) and NaN is kept
  const float w = exp2f(x - (nm == -CUDART_INF_F ? 0.f : nm));
  m = nm;
  l = l * old + w;
  return w;
}

template <int R>
__global__ void __launch_bounds__(kWarps * 32) latent_cc_kernel(const LatentParams p) {
  constexpr int W = R + kLatentRope, kPer = W / 32, kOut = R / 32;
  __shared__ __align__(16) float keys[kBlockSize][W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (p.num_heads + kWarps - 1) / kWarps;
  const int t = blockIdx.x / groups, h = (blockIdx.x % groups) * kWarps + warp;
  if (!starts_ok(p.qsl, p.num_seqs, p.num_tokens)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) flag_error(p.status, PA_DEV_QSL);
    return;
  }
  // (every request is checked by the CTA of its first row; one without rows by the first CTA)
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int r = threadIdx.x; r < p.num_seqs; r += blockDim.x)
      if (__ldg(p.qsl + r) == __ldg(p.qsl + r + 1)) flag_error(p.status, PA_DEV_LENGTHS);
  const int r = request_of(p.qsl, p.num_seqs, t);
  const int a = __ldg(p.qsl + r), L = __ldg(p.qsl + r + 1) - a, S = __ldg(p.seq_lens + r);
  if (L < 1 || L > S || S > p.max_seq_len || L > p.max_query_len) {
    if (threadIdx.x == 0) flag_error(p.status, PA_DEV_LENGTHS);
    return;
  }
  const int seen = S - L + (t - a) + 1;  // keys this row sees
  const int blocks = (seen + kBlockSize - 1) / kBlockSize;
  const int b0 = static_cast<int>(static_cast<long long>(blocks) * blockIdx.y / p.splits);
  const int b1 = static_cast<int>(static_cast<long long>(blocks) * (blockIdx.y + 1) / p.splits);
  const bool mine = h < p.num_heads;
  const float* q = static_cast<const float*>(p.q) + (static_cast<long long>(t) * p.num_heads + (mine ? h : 0)) * W;
  float x[kPer], acc[kOut], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = __ldg(q + i * 32 + lane);
#pragma unroll
  for (int i = 0; i < kOut; ++i) acc[i] = 0.f;
  for (int b = b0; b < b1; ++b) {
    const int rows = min(kBlockSize, seen - b * kBlockSize);
    const int ph = __ldg(p.block_tables + static_cast<long long>(r) * p.max_blocks_per_seq + b);
    const bool ok = ph >= 0 && ph < p.num_blocks;
    if (!ok && threadIdx.x == 0) flag_error(p.status, PA_DEV_BLOCK_RANGE);
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (W / 4); i += kWarps * 32)
      reinterpret_cast<float4*>(&keys[0][0])[i] =
          ok ? __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.cache) +
                                                     static_cast<long long>(ph) * kBlockSize * W) + i)
             : make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    for (int k = 0; k < rows; ++k) {
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) dot = fmaf(x[i], keys[k][i * 32 + lane], dot);
      float old;
      const float w = softmax_step(warp_sum(dot) * p.scale_log2, m, l, old);
#pragma unroll
      for (int i = 0; i < kOut; ++i) acc[i] = fmaf(acc[i], old, w * keys[k][i * 32 + lane]);
    }
  }
  if (!mine) return;
  const long long row = static_cast<long long>(t) * p.num_heads + h;
  if (p.splits == 1) {
    const float inv = 1.f / l;
#pragma unroll
    for (int i = 0; i < kOut; ++i) static_cast<float*>(p.out)[row * R + i * 32 + lane] = acc[i] * inv;
    return;
  }
  const long long part = row * p.splits + blockIdx.y;
#pragma unroll
  for (int i = 0; i < kOut; ++i) p.part_acc[part * R + i * 32 + lane] = acc[i];
  if (lane == 0) reinterpret_cast<float2*>(p.part_ml)[part] = make_float2(m, l);
}

// Join the pieces of a row, in order: one CTA a row.
template <int R>
__global__ void __launch_bounds__(128) latent_cc_join_kernel(const LatentParams p) {
  const long long row = blockIdx.x;
  const int t = static_cast<int>(row / p.num_heads);
  if (!starts_ok(p.qsl, p.num_seqs, p.num_tokens)) return;
  const int r = request_of(p.qsl, p.num_seqs, t);
  const int L = __ldg(p.qsl + r + 1) - __ldg(p.qsl + r), S = __ldg(p.seq_lens + r);
  if (L < 1 || L > S || S > p.max_seq_len || L > p.max_query_len) return;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + row * p.splits;
  float m = -CUDART_INF_F, l = 0.f, acc[R / 128];
  // NaN sums must reach the row, whatever their maximum
  for (int s = 0; s < p.splits; ++s) m = fmaxf(m, ml[s].x);
#pragma unroll
  for (int i = 0; i < R / 128; ++i) acc[i] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    if (ml[s].y == 0.f) continue;  // a piece without keys
    const float f = exp2f(ml[s].x - m);
    l += ml[s].y * f;
#pragma unroll
    for (int i = 0; i < R / 128; ++i)
      acc[i] = fmaf(p.part_acc[(row * p.splits + s) * R + i * 128 + threadIdx.x], f, acc[i]);
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < R / 128; ++i) static_cast<float*>(p.out)[row * R + i * 128 + threadIdx.x] = acc[i] * inv;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) expanded_cc_kernel(const ExpandedParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!starts_ok(p.qsl, p.num_seqs, p.num_tokens) || !starts_ok(p.kvsl, p.num_seqs, p.num_kv_tokens)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) flag_error(p.status, PA_DEV_QSL);
    return;
  }
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r < p.num_seqs; r += blockDim.x)
      if (__ldg(p.qsl + r) == __ldg(p.qsl + r + 1)) flag_error(p.status, PA_DEV_LENGTHS);
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int t = static_cast<int>(row / p.num_heads), h = static_cast<int>(row % p.num_heads);
  if (t >= p.num_tokens) return;
  const int r = request_of(p.qsl, p.num_seqs, t);
  const int a = __ldg(p.qsl + r), L = __ldg(p.qsl + r + 1) - a;
  const int ka = __ldg(p.kvsl + r), S = __ldg(p.kvsl + r + 1) - ka;
  if (L < 1 || L > S || S > p.max_kv_len || L > p.max_query_len) {
    if (lane == 0) flag_error(p.status, PA_DEV_LENGTHS);
    return;
  }
  const float* q = static_cast<const float*>(p.q) + t * p.q_stride + h * p.q_head_stride;
  constexpr int kPer = D / 32;
  float x[kPer], xr[2], acc[kPer], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = __ldg(q + i * 32 + lane), acc[i] = 0.f;
  xr[0] = __ldg(q + D + lane);
  xr[1] = __ldg(q + D + 32 + lane);
  const int seen = S - L + (t - a) + 1;
  for (int k = ka; k < ka + seen; ++k) {
    const float* kn = static_cast<const float*>(p.k) + k * p.k_stride + h * p.k_head_stride;
    const float* kr = static_cast<const float*>(p.kr) + k * p.kr_stride;
    const float* v = static_cast<const float*>(p.v) + k * p.v_stride + h * p.v_head_stride;
    float dot = fmaf(xr[0], __ldg(kr + lane), xr[1] * __ldg(kr + 32 + lane));
#pragma unroll
    for (int i = 0; i < kPer; ++i) dot = fmaf(x[i], __ldg(kn + i * 32 + lane), dot);
    float old;
    const float w = softmax_step(warp_sum(dot) * p.scale_log2, m, l, old);
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = fmaf(acc[i], old, w * __ldg(v + i * 32 + lane));
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < kPer; ++i) static_cast<float*>(p.out)[row * D + i * 32 + lane] = acc[i] * inv;
}

}  // namespace

cudaError_t launch_latent_cc(const LatentParams& p, int latent_size, cudaStream_t stream) {
  const long long groups = (p.num_heads + kWarps - 1) / kWarps;
  const dim3 grid(static_cast<unsigned>(p.num_tokens * groups), static_cast<unsigned>(p.splits));
  const unsigned rows = static_cast<unsigned>(static_cast<long long>(p.num_tokens) * p.num_heads);
  if (latent_size == 512) latent_cc_kernel<512><<<grid, kWarps * 32, 0, stream>>>(p);
  else latent_cc_kernel<256><<<grid, kWarps * 32, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  if (latent_size == 512) latent_cc_join_kernel<512><<<rows, 128, 0, stream>>>(p);
  else latent_cc_join_kernel<256><<<rows, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_expanded_cc(const ExpandedParams& p, int head_size, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.num_tokens) * p.num_heads;
  const unsigned ctas = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
  if (head_size == 128) expanded_cc_kernel<128><<<ctas, kWarps * 32, 0, stream>>>(p);
  else expanded_cc_kernel<64><<<ctas, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
