// Attention over a 4-bit cache for decode and few-token tiles (bf16 q/out):
// split-KV, warp-level f16 matrix products, bulk copies of whole pages, a fused
// log-sum-exp merge.  Work lists, units and the merge are those of the bf16
// kernel (pa_attn_mma.cuh); the plan kernel writes them.
//
// What bounds it: the pages, 20 D bytes per block and kv head, from HBM: at its
// copy rate an SM takes one 2560-byte block (D = 128) per ~110 clocks, so each
// of its four schedulers has ~440 issue slots per block.  So the codes are
// never widened by conversions:
//   K  S = sum_g s_g (q_g . c_g) + z_g sum(q_g) over the groups g of 32 dims.
//      A code masked out of its word is an f16 subnormal: c 2^-24 (nibbles 0
//      of each half) or c 2^-20 (nibbles 1), exact as a matrix operand, so 8
//      codes take 4 ANDs and a shift.  q is staged in f16, scaled by a power of
//      two per row (largest |q| in [2^9, 2^10)) and by 16 more for the dims
//      whose codes are the c 2^-24, exact but for q below 2^-33 of the row's
//      largest.  Each group accumulates by itself (two MMAs), the scales are
//      applied to the float32 sums; the zeros term is one more MMA, z against
//      the group sums of q split into three f16 parts (33 bits).
//   V  v = fma(16 + c, s, z - 16 s) in f16, where 16 + c is the code placed in
//      the top mantissa bits of 16.0: a shift, a masked OR and an FMA per two
//      values.  Rounding z - 16 s (2^-12 of at most 1.6 times the group's
//      range) and v to f16 is an eighth of what the bf16 output's rounding is.
//
// The tile: S^T = K Q^T and O^T += V^T P^T with the 16 keys of a block, then 16
// head dims, as the MMA's M, and the query rows as N: 8 (decode: the G heads
// that share a kv head) or 16 (few tokens: 16 / G positions x G heads).
// Lane (g, c) = (lane / 4, lane % 4) holds S^T at keys g, g + 8 and rows 2c,
// 2c + 1 of each n-tile, and O^T at dims (D/8) g + 2 mt, + 1 of m-tile mt: its
// V codes are one run of the page, all of group g / (32 / (D/8)).
//
// The softmax keeps a running maximum per row that moves only when a logit
// exceeds it by 2^8 (base 2), found by a vote; most blocks need no shuffle and
// no rescaling.  P <= 2^8 in f16, sums in float32.
//
// A CTA has NW compute warps and one scheduler warp (roles as in
// pa_attn_mma.cuh).  Each compute warp streams its blocks through a ring of
// NS stages, two bulk copies a block, one mbarrier a stage; every wait is
// bounded: a warp that gives up flags PA_DEV_TIMEOUT and goes on with what the
// stage holds, so the CTA ends.
#include <cuda_fp16.h>

#include "pa_attn_mma.cuh"
#include "pa_int4.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

constexpr uint32_t kI4WaitLimit = 1u << 22;
constexpr float kI4Rescale = 8.f;  // base-2 logit growth that moves the running maximum

template <int D, int G, int P, int NW, int NS>
struct I4Cfg {
  using Pg = I4Page<D>;
  static constexpr int kR = P * G;               // real query rows
  static constexpr int kNT = (kR + 7) / 8;       // n-tiles of 8 query rows
  static constexpr int kRows = 8 * kNT;          // with padding
  static constexpr int kGroups = D / 32;
  static constexpr int kMT = D / 16;             // m-tiles of O^T
  static constexpr int kThreads = (NW + 1) * 32;
  static constexpr int kStageBytes = 2 * Pg::kBytes;
  static constexpr int kRingBytes = NW * NS * kStageBytes;
  // q buffer: rows of D f16, then per row 16 f16 (group sums) and a float factor
  static constexpr int kQRowBytes = D * 2;
  static constexpr int kQBufBytes = kRows * (kQRowBytes + 32 + 4);
  static constexpr int kQOff = kRingBytes;
  static constexpr int kCombOff = kQOff + 2 * kQBufBytes;
  static constexpr int kCombBytes = 2 * NW * kR * D * 4;  // two units in flight
  static constexpr int kMlOff = kCombOff + kCombBytes;
  static constexpr int kMlBytes = 2 * NW * kR * 2 * 4;
  static constexpr int kMetaOff = (kMlOff + kMlBytes + 15) / 16 * 16;
  static constexpr int kBarOff = kMetaOff + 3 * (static_cast<int>(sizeof(UnitMeta)) + 15) / 16 * 16;
  static constexpr int kSmemBytes = kBarOff + NW * NS * 8;
  static constexpr int kFit = (228 * 1024) / (kSmemBytes + 1024 + 64);
  static constexpr int kMinCtas = kFit >= 3 ? 3 : (kFit >= 2 ? 2 : 1);
  static_assert(kR <= 16 && kGroups <= 4, "at most 16 query rows and 4 groups");
  static_assert(kStageBytes % 16 == 0 && kQBufBytes % 16 == 0, "16-byte stages");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA exceeds 227 KB");
};

// D = A(16x16, row) * B(16x8, col), f16 inputs, fp32 accumulators from zero.
__device__ __forceinline__ void mma_f16_zero(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
  else
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}
__device__ __forceinline__ float2 half2_floats(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;\n" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// 16 + c as f16 for nibble n of both halves of w
template <int N>
__device__ __forceinline__ uint32_t code_plus_16(uint32_t w) {
  constexpr int s = 6 - 4 * N;  // the nibble goes to bits 6-9
  const uint32_t x = s >= 0 ? w << (s >= 0 ? s : 0) : w >> (s >= 0 ? 0 : -s);
  return (x & 0x03c003c0u) | 0x4c004c00u;
}

}  // namespace

template <int D, int G, int P, int NW, int NS>
__global__ void __launch_bounds__(I4Cfg<D, G, P, NW, NS>::kThreads, I4Cfg<D, G, P, NW, NS>::kMinCtas)
    attn_int4_kernel(const AttnParams p) {
  using C = I4Cfg<D, G, P, NW, NS>;
  using Pg = typename C::Pg;
  constexpr int R = C::kR, NT = C::kNT, NG = C::kGroups, MT = C::kMT;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ UnitTail s_tail;
  __shared__ int s_abort;

  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int warp = tid >> 5;
  const bool sched = warp == NW;
  const int Hkv = p.num_kv_heads, Hq = p.num_q_heads;
  UnitMeta* meta = reinterpret_cast<UnitMeta*>(smem + C::kMetaOff);
  float* comb = reinterpret_cast<float*>(smem + C::kCombOff);
  float* comb_ml = reinterpret_cast<float*>(smem + C::kMlOff);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
  const uint32_t ring = smem_u32(smem) + warp * (NS * C::kStageBytes);
  const uint32_t bars = smem_u32(smem + C::kBarOff) + warp * (NS * 8);
  if (tid < NW * NS) mbar_init(smem_u32(smem + C::kBarOff) + tid * 8, 1);
  if (tid == 0) {
    s_abort = 0;
    s_tail.valid = 0;
  }
  mbar_fence_init();
  wait_prior_grid();  // the plan's work lists
  // (not through the read-only path, whose loads may be moved above the wait)
  const int n_units = __ldcg(p.n_items) * Hkv;

  // ---- scheduler-warp helpers -------------------------------------------
  auto fetch_unit = [&](UnitMeta& m, int u) {  // whole scheduler warp
    if (u >= n_units) {
      if (lane == 0) m.valid = 0;
      return;
    }
    const int k = u / Hkv;
    const int item = p.order ? __ldg(p.order + k) : k;
    const UnitRec* rec = p.recs + item;
    const int4 ra = __ldg(&rec->a), rb = __ldg(&rec->b), rc = __ldg(&rec->c);
    const int32_t* row = p.block_tables + static_cast<long long>(ra.x) * p.max_blocks_per_seq;
    for (int i = lane; i < ra.w - ra.z; i += 32) m.bt[i] = __ldg(row + ra.z + i);
    if (lane == 0) {
      m.valid = 1; m.item = item; m.g = u - k * Hkv; m.r = ra.x; m.a = rb.w; m.j0 = ra.y;
      m.npos = rc.x; m.pos0 = rc.y; m.kv_hi = rc.z; m.b0 = ra.z; m.b1 = ra.w;
      m.tile = rb.x; m.first = rb.y; m.nsplit = rb.z;
    }
  };
  auto claim = [&]() -> int {
    int u = 0;
    if (lane == 0) u = atomicAdd(p.next, 1);
    return __shfl_sync(0xffffffffu, u, 0);
  };
  // q rows of unit m (row = position row/G, head row%G): loaded into registers
  // first and staged later, so the loads overlap other scheduler work.
  constexpr int kRowChunks = D / 8;                       // 8 dims a chunk
  constexpr int kQPerLane = C::kRows * kRowChunks / 32;   // a row's chunks sit in adjacent lanes
  auto load_q = [&](const UnitMeta& m, uint4 (&qv)[kQPerLane]) {
#pragma unroll
    for (int i = 0; i < kQPerLane; ++i) {
      const int idx = lane + 32 * i;
      const int row = idx / kRowChunks, c = idx - row * kRowChunks;
      const int jj = row / G, hh = row - jj * G;
      qv[i] = make_uint4(0, 0, 0, 0);
      if (m.valid && row < R && jj < m.npos) {
        const long long tok = m.a + m.j0 + jj;
        qv[i] = __ldg(reinterpret_cast<const uint4*>(q + (tok * Hq + m.g * G + hh) * D) + c);
      }
    }
  };
  auto store_q = [&](const uint4 (&qv)[kQPerLane], int buf) {
    unsigned char* qb = smem + C::kQOff + buf * C::kQBufBytes;
#pragma unroll
    for (int i = 0; i < kQPerLane; ++i) {
      const int idx = lane + 32 * i;
      const int row = idx / kRowChunks, c = idx - row * kRowChunks;
      float x[8];
      Chunk<__nv_bfloat16>::unpack(qv[i], x);
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
      for (int o = 1; o < kRowChunks; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // 2^(9 - exponent) and its inverse
      const int ex = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
      const float f = __uint_as_float(static_cast<uint32_t>(9 - ex + 127) << 23);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= f;
        sum += x[e];
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      // the fragments of the group's two k-steps: nibbles (0, 4), (2, 6) and (1, 5), (3, 7)
      *reinterpret_cast<uint4*>(qb + row * C::kQRowBytes + c * 16) =
          make_uint4(pack_f16(16.f * x[0], 16.f * x[4]), pack_f16(16.f * x[2], 16.f * x[6]),
                     pack_f16(x[1], x[5]), pack_f16(x[3], x[7]));
      // group sums in three f16 parts: element NG j + g is part j of group g
      __half* zs = reinterpret_cast<__half*>(qb + C::kRows * C::kQRowBytes + row * 32);
      if ((c & 3) == 0) {
        const int g = c >> 2;
#pragma unroll
        for (int j = 0; j < 16 / NG; ++j) {
          const __half part = __float2half_rn(j < 3 ? sum : 0.f);
          zs[NG * j + g] = part;
          sum -= __half2float(part);
        }
      }
      if (c == 0)  // S = acc 2^20 / f, times the softmax scale
        *reinterpret_cast<float*>(qb + C::kRows * (C::kQRowBytes + 32) + row * 4) =
            p.scale_log2 * 1048576.f * __uint_as_float(static_cast<uint32_t>(ex - 9 + 127) << 23);
    }
  };

  if (sched) {
    // a second unit is claimed up front only if every CTA can still get one
    const int u0 = claim();
    const int u1 = u0 + static_cast<int>(gridDim.x) < n_units ? claim() : n_units;
    fetch_unit(meta[0], u0);
    fetch_unit(meta[1], u1);
    __syncwarp();
    uint4 qv[kQPerLane];
    load_q(meta[0], qv);
    store_q(qv, 0);
  }
  __syncthreads();

  // ---- compute-warp stream: its share of unit k's blocks, then of unit k+1's
  int iss_unit = 0, iss_i = 0;  // next block to issue: (unit sequence, index in warp share)
  int iss_st = 0, cur_st = 0;   // ring stages of the next issue and of the next block to compute
  uint32_t cur_par = 0;         // its mbarrier phase
  int in_flight = 0;

  auto share = [&](const UnitMeta& m) -> int {
    const int n = m.b1 - m.b0 - warp;
    return (m.valid && n > 0) ? (n + NW - 1) / NW : 0;
  };
  // Issue the next block of the stream if it lies in unit `limit` or earlier.
  auto issue_one = [&](int limit) -> bool {
    while (iss_unit <= limit) {
      if (iss_i < share(meta[iss_unit % 3])) break;
      ++iss_unit;
      iss_i = 0;
    }
    if (iss_unit > limit) return false;
    const UnitMeta& m = meta[iss_unit % 3];
    const int phys = m.bt[warp + iss_i * NW];
    const uint32_t st = ring + iss_st * C::kStageBytes, bar = bars + iss_st * 8;
    if (phys >= 0 && phys < p.num_blocks) {
      if (lane == 0) {
        const long long off = (static_cast<long long>(phys) * Hkv + m.g) * Pg::kBytes;
        mbar_arrive_expect_tx(bar, C::kStageBytes);
        bulk_load(st, static_cast<const unsigned char*>(p.k_cache) + off, Pg::kBytes, bar);
        bulk_load(st + Pg::kBytes, static_cast<const unsigned char*>(p.v_cache) + off, Pg::kBytes, bar);
      }
    } else {  // a bad table entry reads as zeros
      for (int i = lane; i < C::kStageBytes / 16; i += 32)
        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(st + i * 16), "r"(0u) : "memory");
      fence_proxy_async_smem();  // before a later copy into this stage
      __syncwarp();
      if (lane == 0) {
        flag_error(p.status, PA_DEV_BLOCK_RANGE);
        mbar_arrive(bar);
      }
    }
    iss_st = iss_st + 1 == NS ? 0 : iss_st + 1;
    ++iss_i;
    ++in_flight;
    return true;
  };
  auto wait_block = [&]() {  // the next block to compute has landed
    const uint32_t bar = bars + cur_st * 8;
    if (!mbar_try_wait(bar, cur_par)) {
      const uint32_t limit = *reinterpret_cast<volatile int*>(&s_abort) ? 1024u : kI4WaitLimit;
      if (!mbar_wait(bar, cur_par, limit)) {
        s_abort = 1;
        flag_error(p.status, PA_DEV_TIMEOUT);
      }
    }
    __syncwarp();
  };

  if (!sched) {
    while (in_flight < NS && issue_one(1)) {
    }
  }

  // ---- scheduler warp: join the warps' states of a finished unit, write the
  // output or the split's partial, and merge the splits if it is the last.
  auto finish_unit = [&](const UnitTail& u, int buf) {
    const float* cb = comb + buf * NW * R * D;
    const float* cm = comb_ml + buf * NW * R * 2;
    const long long part_base = (static_cast<long long>(u.item) * Hkv + u.g) * R;
    for (int idx = lane; idx < R * D / 4; idx += 32) {
      const int row = (idx * 4) / D, d = idx * 4 - row * D;
      const int jj = row / G, hh = row - jj * G;
      if (jj >= u.npos) continue;
      float M = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, cm[(w * R + row) * 2]);
      float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
      float den = 0.f;
      if (M != -CUDART_INF_F) {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = ex2_approx(cm[(w * R + row) * 2] - M);
          const float4 c4 = *reinterpret_cast<const float4*>(cb + (w * R + row) * D + d);
          num.x = fmaf(c4.x, f, num.x); num.y = fmaf(c4.y, f, num.y);
          num.z = fmaf(c4.z, f, num.z); num.w = fmaf(c4.w, f, num.w);
          den = fmaf(cm[(w * R + row) * 2 + 1], f, den);
        }
      }
      if (u.nsplit == 1) {
        const long long tok = u.a + u.j0 + jj;
        const float inv = p.out_scale / den;
        *reinterpret_cast<uint2*>(out + (tok * Hq + u.g * G + hh) * D + d) =
            make_uint2(pack_bf16(num.x * inv, num.y * inv), pack_bf16(num.z * inv, num.w * inv));
      } else {
        *reinterpret_cast<float4*>(p.part_acc + (part_base + row) * D + d) = num;
        if (d == 0) *reinterpret_cast<float2*>(p.part_ml + (part_base + row) * 2) = make_float2(M, den);
      }
    }
    if (u.nsplit > 1) {
      __threadfence();
      __syncwarp();
      int last = 0;
      if (lane == 0) last = atomicAdd(p.merge_cnt + u.tile * Hkv + u.g, 1) == u.nsplit - 1;
      last = __shfl_sync(0xffffffffu, last, 0);
      if (last) {
        __threadfence();
        // groups of kMergeChunk partials, loaded before any is used: one L2
        // round trip a group
        constexpr int kMergeChunk = 4;
#pragma unroll 2
        for (int idx = lane; idx < R * D / 4; idx += 32) {
          const int row = (idx * 4) / D, d = idx * 4 - row * D;
          const int jj = row / G, hh = row - jj * G;
          if (jj >= u.npos) continue;
          float M = -CUDART_INF_F, den = 0.f;
          float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int sp0 = 0; sp0 < u.nsplit; sp0 += kMergeChunk) {
            float2 ml[kMergeChunk];
            float4 a4[kMergeChunk];
#pragma unroll
            for (int j = 0; j < kMergeChunk; ++j) {
              ml[j] = make_float2(-CUDART_INF_F, 0.f);
              a4[j] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (sp0 + j < u.nsplit) {
                const long long pb = (static_cast<long long>(u.first + sp0 + j) * Hkv + u.g) * R + row;
                ml[j] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + pb * 2));
                a4[j] = __ldcg(reinterpret_cast<const float4*>(p.part_acc + pb * D + d));
              }
            }
            // a split with no visible key for this row holds (-inf, 0) and zeros
            float mc = M;
#pragma unroll
            for (int j = 0; j < kMergeChunk; ++j) mc = fmaxf(mc, ml[j].x);
            if (mc == -CUDART_INF_F) continue;
            if (mc > M) {  // rescale the running sums to the new maximum
              const float sc = ex2_approx(M - mc);  // 0 while nothing was visible
              num.x *= sc; num.y *= sc; num.z *= sc; num.w *= sc; den *= sc;
              M = mc;
            }
#pragma unroll
            for (int j = 0; j < kMergeChunk; ++j) {
              const float f = ex2_approx(ml[j].x - M);  // 0 for an empty split
              num.x = fmaf(a4[j].x, f, num.x); num.y = fmaf(a4[j].y, f, num.y);
              num.z = fmaf(a4[j].z, f, num.z); num.w = fmaf(a4[j].w, f, num.w);
              den = fmaf(ml[j].y, f, den);
            }
          }
          const long long tok = u.a + u.j0 + jj;
          const float inv = p.out_scale / den;
          *reinterpret_cast<uint2*>(out + (tok * Hq + u.g * G + hh) * D + d) =
              make_uint2(pack_bf16(num.x * inv, num.y * inv), pack_bf16(num.z * inv, num.w * inv));
        }
      }
    }
  };

  const int g = lane >> 2, c4 = lane & 3;
  int k = 0;
  for (;; ++k) {
    const UnitMeta& cur = meta[k % 3];
    if (!cur.valid) break;
    if (sched) {
      // while the compute warps stream unit k: load unit k+1's q, finish unit
      // k-1, stage the q rows, claim and decode unit k+2
      uint4 qv[kQPerLane];
      load_q(meta[(k + 1) % 3], qv);
      const UnitTail tail = s_tail;
      if (tail.valid) finish_unit(tail, (k - 1) & 1);
      store_q(qv, (k + 1) & 1);
      const int nu = meta[(k + 1) % 3].valid ? claim() : n_units;
      fetch_unit(meta[(k + 2) % 3], nu);
      __syncwarp();
      if (lane == 0) {
        s_tail.valid = 1; s_tail.item = cur.item; s_tail.g = cur.g; s_tail.a = cur.a;
        s_tail.j0 = cur.j0; s_tail.npos = cur.npos; s_tail.tile = cur.tile;
        s_tail.nsplit = cur.nsplit; s_tail.first = cur.first;
      }
      __syncwarp();
    } else {
      // Every block of units < k has been issued and computed; move the issue
      // pointer off unit k-1, whose metadata slot is now being overwritten.
      if (iss_unit < k) {
        iss_unit = k;
        iss_i = 0;
      }
      while (in_flight < NS && issue_one(k + 1)) {  // stages left free while unit k + 1 was unknown
      }
      // q^T fragments, the group sums' and the rows' factors
      uint32_t qb[NT][NG][4], zb[NT][2];
      float rm[NT][2];
      {
        const unsigned char* buf = smem + C::kQOff + (k & 1) * C::kQBufBytes;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t row = smem_u32(buf) + (8 * n + g) * C::kQRowBytes;
#pragma unroll
          for (int e = 0; e < NG; ++e) lds_words<4>(row + (4 * e + c4) * 16, qb[n][e]);
          const uint32_t* zs = reinterpret_cast<const uint32_t*>(buf + C::kRows * C::kQRowBytes + (8 * n + g) * 32);
          zb[n][0] = zs[c4];
          zb[n][1] = zs[4 + c4];
          const float* fr = reinterpret_cast<const float*>(buf + C::kRows * (C::kQRowBytes + 32)) + 8 * n;
          rm[n][0] = fr[2 * c4];
          rm[n][1] = fr[2 * c4 + 1];
        }
      }
      float o[NT][MT][4];
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < MT; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
        m[n][0] = m[n][1] = -CUDART_INF_F;
        l[n][0] = l[n][1] = 0.f;
      }
      const int nb = share(cur);
      for (int i = 0; i < nb; ++i) {
        wait_block();
        const uint32_t kp = ring + cur_st * C::kStageBytes, vp = kp + Pg::kBytes;
        const int tok0 = (cur.b0 + warp + i * NW) * kBlockSize;
        // S^T of keys g, g + 8
        float s[NT][4];
        {
          uint32_t kw[2][NG], pw[2][NG];  // codes; scales then zeros as f16 pairs
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            lds_words<NG>(kp + Pg::k_word(g + 8 * h, 0, c4), kw[h]);
            lds_words<NG>(kp + Pg::k_scale(g + 8 * h, 0), pw[h]);
          }
          // zeros: lane c4 takes groups 2 c4, 2 c4 + 1 (modulo the groups)
          uint32_t za[4];
          za[0] = za[2] = NG == 4 ? ((c4 & 1) ? pw[0][NG - 1] : pw[0][NG / 2]) : pw[0][1];
          za[1] = za[3] = NG == 4 ? ((c4 & 1) ? pw[1][NG - 1] : pw[1][NG / 2]) : pw[1][1];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16_zero(s[n], za, zb[n][0], zb[n][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] *= 0x1p-20f;
          }
#pragma unroll
          for (int e = 0; e < NG; ++e) {
            uint32_t a[4], b[4];
            a[0] = kw[0][e] & 0x000f000fu;
            a[1] = kw[1][e] & 0x000f000fu;
            b[0] = kw[0][e] & 0x00f000f0u;
            b[1] = kw[1][e] & 0x00f000f0u;
            const uint32_t k0 = kw[0][e] >> 8, k1 = kw[1][e] >> 8;
            a[2] = k0 & 0x000f000fu;
            a[3] = k1 & 0x000f000fu;
            b[2] = k0 & 0x00f000f0u;
            b[3] = k1 & 0x00f000f0u;
            const float2 f0 = half2_floats(pw[0][e / 2]), f1 = half2_floats(pw[1][e / 2]);
            const float s0 = (e & 1) ? f0.y : f0.x, s1 = (e & 1) ? f1.y : f1.x;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float acc[4];
              mma_f16_zero(acc, a, qb[n][e][0], qb[n][e][1]);
              mma_f16(acc, b, qb[n][e][2], qb[n][e][3]);
              s[n][0] = fmaf(acc[0], s0, s[n][0]);
              s[n][1] = fmaf(acc[1], s0, s[n][1]);
              s[n][2] = fmaf(acc[2], s1, s[n][2]);
              s[n][3] = fmaf(acc[3], s1, s[n][3]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            s[n][0] *= rm[n][0]; s[n][1] *= rm[n][1];
            s[n][2] *= rm[n][0]; s[n][3] *= rm[n][1];
          }
        }
        // V parameters: scales and zeros of tokens (2 c4, 2 c4 + 1) and
        // (2 c4 + 8, 2 c4 + 9), all in the group of the lane's run of dims
        uint32_t vq[4];
        lds_words<4>(vp + Pg::kCodeBytes + (g * Pg::kRun / 32) * 64 + c4 * 16, vq);
        if (tok0 + kBlockSize - 1 > cur.pos0 || tok0 + kBlockSize > cur.kv_hi) {
          // causal edge or unwritten slots (their K, V and parameters may be anything)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = tok0 + g + 8 * (e >> 1);
              const int jj = (8 * n + 2 * c4 + (e & 1)) / G;
              if (tok >= cur.kv_hi || tok > cur.pos0 + jj) s[n][e] = -CUDART_INF_F;
            }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int left = cur.kv_hi - (tok0 + 2 * c4 + 8 * h);  // written tokens of the pair
            const uint32_t keep = left >= 2 ? 0xffffffffu : (left == 1 ? 0x0000ffffu : 0u);
            vq[h] &= keep;
            vq[2 + h] &= keep;
          }
        }
        // online softmax (base 2)
        float pr[NT][4];
        bool grew = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          grew |= fmaxf(s[n][0], s[n][2]) > m[n][0] + kI4Rescale ||
                  fmaxf(s[n][1], s[n][3]) > m[n][1] + kI4Rescale;
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(m[n][e], fmaxf(s[n][e], s[n][2 + e]));
#pragma unroll
              for (int o8 = 4; o8 < 32; o8 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o8));
              if (mx > m[n][e]) {
                const float corr = ex2_approx(m[n][e] - mx);  // 0 before the first visible key
                m[n][e] = mx;
                l[n][e] *= corr;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  o[n][mt][e] *= corr;
                  o[n][mt][2 + e] *= corr;
                }
              }
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ms = m[n][e] == -CUDART_INF_F ? 0.f : m[n][e];
            pr[n][e] = ex2_approx(s[n][e] - ms);
            pr[n][2 + e] = ex2_approx(s[n][2 + e] - ms);
            l[n][e] += pr[n][e] + pr[n][2 + e];
          }
          // P^T as the B operand: an 8 x 8 transpose per half of the block's keys
          pb[n][0] = movm_trans(pack_f16(pr[n][0], pr[n][1]));
          pb[n][1] = movm_trans(pack_f16(pr[n][2], pr[n][3]));
        }
        // O^T += V^T P^T
        {
          const uint32_t minus16 = 0xcc00cc00u;
          const uint32_t z0 = fma_half2(vq[0], minus16, vq[2]), z1 = fma_half2(vq[1], minus16, vq[3]);
          uint32_t vw[2][NG];
#pragma unroll
          for (int h = 0; h < 2; ++h) lds_words<NG>(vp + h * 4 * D + g * (D / 2) + c4 * Pg::kRun, vw[h]);
          __syncwarp();  // the stage has been read
#pragma unroll
          for (int w = 0; w < NG; ++w) {
            uint32_t a[4], b[4];
            a[0] = fma_half2(code_plus_16<0>(vw[0][w]), vq[0], z0);
            a[1] = fma_half2(code_plus_16<1>(vw[0][w]), vq[0], z0);
            a[2] = fma_half2(code_plus_16<0>(vw[1][w]), vq[1], z1);
            a[3] = fma_half2(code_plus_16<1>(vw[1][w]), vq[1], z1);
            b[0] = fma_half2(code_plus_16<2>(vw[0][w]), vq[0], z0);
            b[1] = fma_half2(code_plus_16<3>(vw[0][w]), vq[0], z0);
            b[2] = fma_half2(code_plus_16<2>(vw[1][w]), vq[1], z1);
            b[3] = fma_half2(code_plus_16<3>(vw[1][w]), vq[1], z1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_f16(o[n][2 * w], a, pb[n][0], pb[n][1]);
              mma_f16(o[n][2 * w + 1], b, pb[n][0], pb[n][1]);
            }
          }
        }
        // this stage is free: the stream's next block goes into it
        if (++cur_st == NS) {
          cur_st = 0;
          cur_par ^= 1;
        }
        --in_flight;
        issue_one(k + 1);
      }
      // the warp's state for this unit -> shared memory (real rows only)
      float* cb = comb + (k & 1) * NW * R * D;
      float* cm = comb_ml + (k & 1) * NW * R * 2;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[n][e];
#pragma unroll
          for (int o8 = 4; o8 < 32; o8 <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o8);
          const int row = 8 * n + 2 * c4 + e;
          if (row < R) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              *reinterpret_cast<float2*>(cb + (warp * R + row) * D + (D / 8) * g + 2 * mt) =
                  make_float2(o[n][mt][e], o[n][mt][2 + e]);
            if (g == 0) {
              cm[(warp * R + row) * 2] = m[n][e];
              cm[(warp * R + row) * 2 + 1] = sum;
            }
          }
        }
    }
    __syncthreads();
  }
  if (sched) {
    const UnitTail tail = s_tail;
    if (tail.valid) finish_unit(tail, (k - 1) & 1);
  }
}

namespace {

// Launches the kernel, or with grid_only set only stores the grid size it
// would use (CTAs per SM by occupancy x SMs).
template <int D, int G, int P, int NW, int NS>
cudaError_t launch_i4(const AttnParams& p, int num_sms, cudaStream_t stream, int* grid_only) {
  using C = I4Cfg<D, G, P, NW, NS>;
  static int ctas_per_sm[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (ctas_per_sm[dev] == 0) {
    e = cudaFuncSetAttribute(attn_int4_kernel<D, G, P, NW, NS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_int4_kernel<D, G, P, NW, NS>, C::kThreads,
                                                      C::kSmemBytes);
    if (e != cudaSuccess) return e;
    ctas_per_sm[dev] = n > 0 ? n : 1;
  }
  if (grid_only) {
    *grid_only = num_sms * ctas_per_sm[dev];
    return cudaSuccess;
  }
  // right after the plan kernel the launch may overlap its tail (the kernel
  // waits for the plan before reading the work lists)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms * ctas_per_sm[dev]);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.after_plan ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_int4_kernel<D, G, P, NW, NS>, p);
}

template <int D, int G>
cudaError_t dispatch_positions_int4(const AttnParams& p, int positions, int num_sms,
                                    cudaStream_t stream, int* grid_only) {
  constexpr int NS = D == 128 ? 4 : 8;
  return positions == 1 ? launch_i4<D, G, 1, 4, NS>(p, num_sms, stream, grid_only)
                        : launch_i4<D, G, kSmallRows / G, 4, NS>(p, num_sms, stream, grid_only);
}

template <int D>
cudaError_t dispatch_group_int4(const AttnParams& p, int group, int positions, int num_sms,
                                cudaStream_t stream, int* grid_only) {
  switch (group) {
    case 1: return dispatch_positions_int4<D, 1>(p, positions, num_sms, stream, grid_only);
    case 2: return dispatch_positions_int4<D, 2>(p, positions, num_sms, stream, grid_only);
    case 4: return dispatch_positions_int4<D, 4>(p, positions, num_sms, stream, grid_only);
    case 8: return dispatch_positions_int4<D, 8>(p, positions, num_sms, stream, grid_only);
    default: return cudaErrorInvalidValue;
  }
}
}  // namespace

cudaError_t launch_attn_int4(const AttnParams& p, int head_size, int group, int positions,
                             int num_sms, cudaStream_t stream, int* grid_only) {
  switch (head_size) {
    case 64: return dispatch_group_int4<64>(p, group, positions, num_sms, stream, grid_only);
    case 128: return dispatch_group_int4<128>(p, group, positions, num_sms, stream, grid_only);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
