// The slot write into a latent cache, and the read-back.
//
// A token's row is [latent, shared key part]: the latent is divided by its root mean
// square and weighted (or copied), the key part rotated, and the queries' parts that meet
// it are rotated in the same launch.  One pass, every number read and written once, so HBM
// bounds it (launch latency for few tokens).
// A warp takes either a token's cache row (a lane R / 32 numbers of the latent in chunks of
// 16 bytes that lie side by side over the warp; four lanes the key part) or the
// parts of 16 of its heads (four lanes a head, eight heads at once, their loads ahead of the position:
// 34.3 us for 16384 tokens of 32 heads, 75 % of the copy bandwidth; with 8 heads a warp 40.9, with 32 37.0;
// fp32 69 us, 75 % too).
#include "pa_latent.h"
#include "pa_rope.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kHeadsAtOnce = 8, kTimes = 2, kHeadsPerWarp = kHeadsAtOnce * kTimes;

struct LatentWrite {
  LatentWriteArgs a;
  RopeParams rope;
  int num_heads;  // 0: no queries
  unsigned jobs;  // warps of a token: its row, then its heads
  long long num_slots;
};

template <typename T, int R>
__global__ void __launch_bounds__(kThreads) latent_write_kernel(const LatentWrite p) {
  launch_dependents();
  constexpr int kRow = R + kLatentRope;
  constexpr int kGroups = R / 256;  // groups of 8 numbers a lane
  const unsigned w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const unsigned t = w / p.jobs;
  if (t >= static_cast<unsigned>(p.a.num_tokens)) return;  // whole warps
  const int job = static_cast<int>(w - t * p.jobs);
  const bool pairs = p.rope.pairs != 0;
  const int j = lane & 3;
  int oa, ob;
  rope_groups(j, kLatentRope, pairs, oa, ob);
  // (the numbers are on their way while the token's position and slot are looked up)
  if (job > 0) {
    const int h = (job - 1) * kHeadsPerWarp + (lane >> 2);
    const T* src = static_cast<const T*>(p.a.q) + t * p.a.q_stride + h * p.a.q_head_stride;
    Eight<T> a[kTimes], b[kTimes];
#pragma unroll
    for (int i = 0; i < kTimes; ++i)
      if (h + i * kHeadsAtOnce < p.num_heads) {
        a[i].load(src + i * kHeadsAtOnce * p.a.q_head_stride + oa);
        b[i].load(src + i * kHeadsAtOnce * p.a.q_head_stride + ob);
      }
    const float* table = rope_row(p.rope, t, lane == 0, p.a.status);
    if (!table) return;
    T* dst = static_cast<T*>(p.a.q_out) + t * p.a.qo_stride + h * p.a.qo_head_stride;
#pragma unroll
    for (int i = 0; i < kTimes; ++i)
      if (h + i * kHeadsAtOnce < p.num_heads) {
        rope_turn(a[i], b[i], table, j, kLatentRope, pairs);
        a[i].store(dst + i * kHeadsAtOnce * p.a.qo_head_stride + oa);
        b[i].store(dst + i * kHeadsAtOnce * p.a.qo_head_stride + ob);
      }
    return;
  }
  Eight<T> a, b;
  const T* c = static_cast<const T*>(p.a.c) + t * p.a.c_stride;
  Eight<T> e[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) e[g].load(c + g * 256 + lane * 8);
  if (lane < 4) {
    const T* k = static_cast<const T*>(p.a.k) + t * p.a.k_stride;
    a.load(k + oa);
    b.load(k + ob);
  }
  const int64_t s = __ldg(p.a.slots + t);
  const float* table = rope_row(p.rope, t, lane == 0, p.a.status);
  if (!table) return;
  if (s >= p.num_slots && lane == 0) flag_error(p.a.status, PA_DEV_SLOT_RANGE);
  if (s < 0 || s >= p.num_slots) return;
  T* row = static_cast<T*>(p.a.cache) + s * kRow;
  if (lane < 4) {
    rope_turn(a, b, table, j, kLatentRope, pairs);
    a.store(row + R + oa);
    b.store(row + R + ob);
  }
  __syncwarp();
  if (p.a.weight) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float x[8];
      e[g].get(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = 1.f / sqrtf(sum * (1.f / R) + p.a.eps);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float x[8], y[8];
      Eight<T> we;
      we.load(static_cast<const T*>(p.a.weight) + g * 256 + lane * 8);
      we.get(y);
      e[g].get(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * y[i];
      e[g].set(x);
    }
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) e[g].store(row + g * 256 + lane * 8);
}

// A thread one 16-byte chunk of a row.
template <int kChunks, int kLatentChunks>
__global__ void __launch_bounds__(kThreads) latent_read_kernel(
    const uint4* cache, const int64_t* slots, int num_tokens, uint4* c, uint4* k, long long num_slots, int32_t* status) {
  const long long total = static_cast<long long>(num_tokens) * kChunks;
  const long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x;
  if (i >= total) return;  // (a CTA's end lets dependents start too)
  const long long t = i / kChunks;
  const int at = static_cast<int>(i - t * kChunks);
  wait_prior_grid();
  launch_dependents();
  const int64_t s = slots[t];
  if (s < 0) return;
  if (s >= num_slots) {
    if (at == 0) flag_error(status, PA_DEV_SLOT_RANGE);
    return;
  }
  const uint4 x = cache[s * kChunks + at];
  if (at < kLatentChunks) c[t * kLatentChunks + at] = x;
  else k[t * (kChunks - kLatentChunks) + at - kLatentChunks] = x;
}

template <typename T, int R>
cudaError_t launch_write(const LatentWrite& p, cudaStream_t stream) {
  constexpr long long kWarps = kThreads / 32;
  const long long warps = static_cast<long long>(p.a.num_tokens) * p.jobs;
  latent_write_kernel<T, R>
      <<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_write(const LatentWriteArgs& a, const pa_latent_layout& L, cudaStream_t stream) {
  const int heads = a.q ? L.num_heads : 0;
  const LatentWrite p{a, rope_params(a.rope), heads,
                      1u + static_cast<unsigned>((heads + kHeadsPerWarp - 1) / kHeadsPerWarp),
                      static_cast<long long>(L.num_blocks) * kBlockSize};
  if (L.dtype == PA_F32)
    return L.latent_size == 512 ? launch_write<float, 512>(p, stream) : launch_write<float, 256>(p, stream);
  return L.latent_size == 512 ? launch_write<__nv_bfloat16, 512>(p, stream)
                              : launch_write<__nv_bfloat16, 256>(p, stream);
}

cudaError_t launch_latent_read(const void* cache, const int64_t* slots, int num_tokens, void* c,
                               void* k, const pa_latent_layout& L, int32_t* status,
                               cudaStream_t stream) {
  const int e = L.dtype == PA_F32 ? 4 : 2;
  const long long total = static_cast<long long>(num_tokens) * (L.latent_size + kLatentRope) * e / 16;
  auto go = [&](auto kernel) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((total + kThreads - 1) / kThreads));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint4*>(cache), slots, num_tokens,
                              static_cast<uint4*>(c), static_cast<uint4*>(k),
                              static_cast<long long>(L.num_blocks) * kBlockSize, status);
  };
  if (L.latent_size == 512) return e == 4 ? go(latent_read_kernel<144, 128>) : go(latent_read_kernel<72, 64>);
  return e == 4 ? go(latent_read_kernel<80, 64>) : go(latent_read_kernel<40, 32>);
}

}  // namespace pa
