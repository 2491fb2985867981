// Attention over a 4-bit cache for decode and few-token tiles (bf16 q/out):
// split-KV, warp-level f16 matrix products, a fused log-sum-exp merge.  Work lists
// and units are those of the bf16 kernel (pa_attn_mma.cuh); the plan kernel writes
// them.
//
// What bounds it: the pages, 20 D bytes per block and kv head, from HBM: at its
// copy rate an SM takes one 2560-byte block (D = 128) per ~110 clocks, so each
// of its four schedulers has ~440 issue slots per block, and the integer pipe
// (one instruction in two clocks) half as many.  So the codes are never widened
// by conversions:
//   K  S = sum_g s_g (q_g . c_g) + z_g sum(q_g) over the groups g of 32 dims.
//      A code masked out of its word is an f16 subnormal: c 2^-24 (nibbles 0
//      of each half) or c 2^-20 (nibbles 1), exact as a matrix operand, so 8
//      codes take 4 ANDs and a shift.  q is staged in f16, scaled by a power of
//      two per row (largest |q| in [2^10, 2^11)) and by 16 more for the dims
//      whose codes are the c 2^-24: exact down to 2^-27 of the row's largest (a bf16
//      q has 8 bits and f16 ends at 2^-24), below it off by 2^-35 of the largest at
//      most.  Each group accumulates by itself (two MMAs) and the scales are
//      applied to the float32 sums; the zeros term is one more MMA, z against
//      the group sums of q 2^-20 split into f16 parts (off by 2^-25 at most, 2^-15 of
//      the row's largest q).
//   V  v = c s + z in f16, rounded once: a masked OR, an exact subtraction and an FMA
//      per two values (pa_int4.cuh).
//
// The tile: S^T = K Q^T and O^T += V^T P^T with the 16 keys of a block, then 16
// head dims, as the MMA's M, and up to 8 query rows as N: the G heads that share a
// kv head (decode) or 8 / G positions of them (few tokens).  Tiles of 16 rows in
// two n-tiles unpack the codes half as often, but their registers leave 9 compute
// warps an SM instead of 12: 48 requests of 2-8 tokens after 256-4096, 32/8 heads,
// took 130 us instead of 112 (kernel and plan).
// Lane (g, c) = (lane / 4, lane % 4) holds S^T at keys g, g + 8 and rows 2c,
// 2c + 1, and O^T at dims (D/8) g + 2 mt, + 1 of m-tile mt: its V codes are one
// run of the page, all of one group.
//
// The softmax keeps a running maximum per row that moves only when a logit
// exceeds it by 2^4 (base 2), found by a vote; most steps need no shuffle and
// no rescaling.  P is held as f16 of 2^11 P <= 2^15, so that a weight keeps its 11
// bits down to 2^-25 of the largest (long contexts beside a dominant key live on
// such weights); the factor cancels in the normalisation.  Sums in float32.
//
// A CTA has NW compute warps and one scheduler warp.  A compute warp takes pairs
// of blocks w, w + NW, ... of a unit through a ring of NS stages of 16-byte
// asynchronous copies that runs on into the next unit.  (Whole pages by bulk copy
// were slower: a warp's four are issued one lane after the other.)  The scheduler
// warp claims and stages one unit ahead and joins the finished one; where that
// completes a split tile, the merge goes to the compute warps as their next
// unit.  The roles meet on mbarriers only (unit ready, warp states written, warp
// states read), so a warp that is done goes on.  Every wait is bounded: one that
// gives up flags PA_DEV_TIMEOUT and ends the CTA after its copies have landed.
// Measured on Llama-3-8B heads: 256 requests of median 1024 keys 81 us (4 950 GB/s of
// pages and the rest), 16 of 32768-131072 295 us with the plan (5 800 GB/s).
#include <cuda_fp16.h>

#include "pa_attn_mma.cuh"
#include "pa_int4.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

constexpr unsigned long long kI4WaitNs = 2000000000ull;  // a wait gives up after two seconds
constexpr float kI4Rescale = 4.f;  // base-2 logit growth that moves the running maximum
constexpr float kI4Lift = 11.f;    // P is held times 2^11: at most 2^15 in f16

template <int D, int G, int P, int NW, int NS>
struct I4Cfg {
  using Pg = I4Page<D>;
  static constexpr int kR = P * G;               // real query rows
  static constexpr int kGroups = D / 32;
  static constexpr int kMT = D / 16;             // m-tiles of O^T
  static constexpr int kThreads = (NW + 1) * 32;
  static constexpr int kBlockBytes = 2 * Pg::kBytes;  // K and V page of a block
  static constexpr int kStageBytes = 2 * kBlockBytes;
  static constexpr int kRingBytes = NW * NS * kStageBytes;
  // q buffer: rows of D f16, then per row 16 f16 (group sums) and a float factor
  static constexpr int kQRowBytes = D * 2;
  static constexpr int kQBufBytes = (kR * (kQRowBytes + 32 + 4) + 15) / 16 * 16;
  static constexpr int kQOff = kRingBytes;
  // the warps' states of finished units: two units' up to 4 rows, one unit's with
  // more (16 KB at 8 rows; a third CTA would not fit beside two)
  static constexpr int kNB = kR <= 4 ? 2 : 1;
  static constexpr int kCombOff = kQOff + 2 * kQBufBytes;
  static constexpr int kCombBytes = kNB * NW * kR * D * 4;
  static constexpr int kMlOff = kCombOff + kCombBytes;
  static constexpr int kMlBytes = kNB * NW * kR * 2 * 4;
  static constexpr int kMetaOff = (kMlOff + kMlBytes + 15) / 16 * 16;
  static constexpr int kBarOff = kMetaOff + 2 * ((static_cast<int>(sizeof(UnitMeta)) + 15) / 16 * 16);
  static constexpr int kNumBars = 2 + 2 * kNB;
  static constexpr int kSmemBytes = kBarOff + kNumBars * 8;
  static constexpr int kFit = (228 * 1024) / (kSmemBytes + 1024 + 64);
  static constexpr int kMinCtas = kFit < 3 ? kFit : 3;
  static_assert(kR <= 8 && kGroups <= 4, "at most 8 query rows and 4 groups");
  static_assert(kStageBytes % 16 == 0 && kQBufBytes % 16 == 0, "16-byte stages");
  static_assert(kNumBars <= kThreads, "one thread initialises each barrier");
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
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(w[0]) : "r"(addr));
}
__device__ __forceinline__ float2 half2_floats(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t));
  return t;
}
// Whether phase `parity` has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

}  // namespace

template <int D, int G, int P, int NW, int NS>
__global__ void __launch_bounds__(I4Cfg<D, G, P, NW, NS>::kThreads, I4Cfg<D, G, P, NW, NS>::kMinCtas)
    attn_int4_kernel(const AttnParams p) {
  using C = I4Cfg<D, G, P, NW, NS>;
  using Pg = typename C::Pg;
  constexpr int R = C::kR, NG = C::kGroups, MT = C::kMT, NB = C::kNB;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_abort;

  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int warp = tid >> 5;
  const int Hkv = p.num_kv_heads, Hq = p.num_q_heads;
  float* comb = reinterpret_cast<float*>(smem + C::kCombOff);
  float* comb_ml = reinterpret_cast<float*>(smem + C::kMlOff);
  auto meta = [&](int k) -> UnitMeta& {  // of unit k of this CTA's sequence
    return *reinterpret_cast<UnitMeta*>(smem + C::kMetaOff +
                                        (k & 1) * ((static_cast<int>(sizeof(UnitMeta)) + 15) / 16 * 16));
  };
  // mbarriers
  const uint32_t bar_unit = smem_u32(smem + C::kBarOff);  // [2] unit published (scheduler)
  const uint32_t bar_full = bar_unit + 16;        // [NB] states written (NW warps)
  const uint32_t bar_free = bar_full + NB * 8;    // [NB] ... and read (scheduler)
  if (tid < C::kNumBars) {
    const bool full = tid >= 2 && tid < 2 + NB;
    mbar_init(bar_unit + tid * 8, full ? NW : 1);
  }
  if (tid == 0) s_abort = 0;
  mbar_fence_init();
  __syncthreads();
  wait_prior_grid();  // the plan's work lists

  // Bounded wait (whole warp) for phase `parity`; false if it gave up.
  auto wait_for = [&](uint32_t bar, uint32_t parity) -> bool {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
      const unsigned long long t0 = now_ns();
      while (!ok && *reinterpret_cast<volatile int*>(&s_abort) == 0 && now_ns() - t0 < kI4WaitNs)
        ok = mbar_try_wait(bar, parity);
      if (!ok) {
        s_abort = 1;
        flag_error(p.status, PA_DEV_TIMEOUT);
      }
    }
    return __all_sync(0xffffffffu, ok);
  };

  if (warp == NW) {
    // ---------------------------------------------------------- scheduler warp
    // (what the plan wrote is not read through the read-only path, whose loads may
    // be moved above the wait)
    const int n_units = __ldcg(p.n_items) * Hkv;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
    // Metadata of unit u into m: one precomputed record and the unit's slice of
    // the block table.
    auto fetch_unit = [&](UnitMeta& m, int u) {
      const int k = u / Hkv;
      const int item = p.order ? __ldcg(p.order + k) : k;
      const UnitRec* rec = p.recs + item;
      const int4 ra = __ldcg(&rec->a), rb = __ldcg(&rec->b), rc = __ldcg(&rec->c);
      const int32_t* row = p.block_tables + static_cast<long long>(ra.x) * p.max_blocks_per_seq;
      // a bad entry, and the one after an odd count, become -1: a block of zeros
      const int n = ra.w - ra.z;
      for (int i = lane; i < n; i += 32) {
        int b = __ldg(row + ra.z + i);
        if (static_cast<uint32_t>(b) >= static_cast<uint32_t>(p.num_blocks)) {
          flag_error(p.status, PA_DEV_BLOCK_RANGE);
          b = -1;
        }
        m.bt[i] = b;
      }
      if (lane == 0 && (n & 1)) m.bt[n] = -1;
      if (lane == 0) {
        m.valid = 1; m.item = item; m.g = u - k * Hkv; m.r = ra.x; m.a = rb.w; m.j0 = ra.y;
        m.npos = rc.x; m.pos0 = rc.y; m.kv_hi = rc.z; m.b0 = ra.z; m.b1 = ra.w;
        m.tile = rb.x; m.first = rb.y; m.nsplit = rb.z;
      }
      __syncwarp();
    };
    // q rows of unit m (row = position row/G, head row%G) into buffer buf, eight
    // dims a lane and step, a row's chunks in adjacent lanes.
    constexpr int kRowChunks = D / 8;
    constexpr int kQPerLane = (R * kRowChunks + 31) / 32;
    auto stage_q = [&](const UnitMeta& m, int buf) {
      unsigned char* qb = smem + C::kQOff + buf * C::kQBufBytes;
      uint4 qv[kQPerLane];
#pragma unroll
      for (int i = 0; i < kQPerLane; ++i) {
        const int idx = lane + 32 * i;
        const int row = idx / kRowChunks, c = idx - row * kRowChunks;
        const int jj = row / G, hh = row - jj * G;
        qv[i] = make_uint4(0, 0, 0, 0);
        if (row < R && jj < m.npos) {
          const long long tok = m.a + m.j0 + jj;
          qv[i] = __ldg(reinterpret_cast<const uint4*>(q + (tok * Hq + m.g * G + hh) * D) + c);
        }
      }
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
        // 2^(10 - exponent), with the softmax scale's sign; the inverse goes into
        // the row's factor
        const int ex = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
        const float f = copysignf(__uint_as_float(static_cast<uint32_t>(10 - ex + 127) << 23), p.scale_log2);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= f;
          sum += x[e];
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        // the fragments of the group's two k-steps: nibbles (0, 4), (2, 6) and (1, 5), (3, 7)
        if (row >= R) continue;
        *reinterpret_cast<uint4*>(qb + row * C::kQRowBytes + c * 16) =
            make_uint4(pack_f16(16.f * x[0], 16.f * x[4]), pack_f16(16.f * x[2], 16.f * x[6]),
                       pack_f16(x[1], x[5]), pack_f16(x[3], x[7]));
        // group sums x 2^-20 in f16 parts: element NG j + g is part j of group g
        __half* zs = reinterpret_cast<__half*>(qb + R * C::kQRowBytes + row * 32);
        if ((c & 3) == 0) {
          const int g = c >> 2;
          sum *= 0x1p-20f;
#pragma unroll
          for (int j = 0; j < 16 / NG; ++j) {
            const __half part = __float2half_rn(j < 3 ? sum : 0.f);
            zs[NG * j + g] = part;
            sum -= __half2float(part);
          }
        }
        if (c == 0) {  // base-2 logit = (accumulated sum) x factor; kept positive and finite
          const float f = fabsf(p.scale_log2) * 1048576.f *
                          __uint_as_float(static_cast<uint32_t>(ex - 10 + 127) << 23);
          *reinterpret_cast<float*>(qb + R * (C::kQRowBytes + 32) + row * 4) =
              fminf(fmaxf(f, 1e-37f), 3e38f);
        }
      }
    };
    auto publish = [&](int k, int u) {  // unit k of the sequence is unit u of the list
      UnitMeta& m = meta(k);
      fetch_unit(m, u);
      stage_q(m, k & 1);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_unit + (k & 1) * 8);
    };
    // Join the warps' states of a finished unit and write the output or the split's
    // partial; true if that was the tile's last split.
    auto finish_unit = [&](const UnitTail& u, int buf) -> bool {
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
        } else {  // no visible key (0), or logits of NaN alone (NaN)
#pragma unroll
          for (int w = 0; w < NW; ++w) den += cm[(w * R + row) * 2 + 1];
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
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_free + buf * 8);  // the states have been read
      if (u.nsplit == 1) return false;
      __threadfence();
      __syncwarp();
      int last = 0;
      if (lane == 0) {
        last = atomicAdd(p.merge_cnt + u.tile * Hkv + u.g, 1) == u.nsplit - 1;
        __threadfence();
      }
      return __shfl_sync(0xffffffffu, last, 0) != 0;
    };
    // A CTA's first unit is its own index, later ones count on from the grid
    // size; a second one is claimed up front only if every CTA can still get one.
    const int grid = static_cast<int>(gridDim.x);
    auto claim = [&]() -> int {
      int u = 0;
      if (lane == 0) u = grid + atomicAdd(p.next, 1);
      return __shfl_sync(0xffffffffu, u, 0);
    };
    auto publish_merge = [&](int k, const UnitTail& t) {  // a merge as unit k
      __syncwarp();
      if (lane == 0) {
        UnitMeta& m = meta(k);
        m.valid = 2; m.g = t.g; m.a = t.a; m.j0 = t.j0; m.npos = t.npos;
        m.nsplit = t.nsplit; m.first = t.first; m.b0 = 0; m.b1 = 0;
        mbar_arrive(bar_unit + (k & 1) * 8);
      }
      __syncwarp();
    };
    int published = 0;  // units published so far
    bool left = true;   // the list may hold more
    auto publish_next = [&](int u) {
      left = u < n_units;
      if (left) publish(published++, u);
    };
    publish_next(blockIdx.x);
    if (left) publish_next(static_cast<int>(blockIdx.x) + grid < n_units ? claim() : n_units);
    UnitTail merge;
    merge.valid = 0;  // a merge to publish
    int k = 0;
    for (; k < published; ++k) {
      if (!wait_for(bar_full + (k % NB) * 8, (k / NB) & 1)) return;
      const UnitMeta& m = meta(k);
      UnitTail t;
      t.valid = m.valid; t.item = m.item; t.g = m.g; t.a = m.a; t.j0 = m.j0;
      t.npos = m.npos; t.tile = m.tile; t.nsplit = m.nsplit; t.first = m.first;
      __syncwarp();
      // the finished unit's slot takes the next one, a merge before a new unit
      if (merge.valid) {
        publish_merge(published++, merge);
        merge.valid = 0;
      } else if (left) {
        publish_next(claim());
      }
      if (t.valid == 1) {
        if (finish_unit(t, k % NB)) merge = t;
      } else if (lane == 0) {
        mbar_arrive(bar_free + (k % NB) * 8);
      }
      if (merge.valid && published <= k + 2) {
        publish_merge(published++, merge);
        merge.valid = 0;
      }
    }
    if (lane == 0) {  // the end
      meta(k).valid = 0;
      mbar_arrive(bar_unit + (k & 1) * 8);
    }
    return;
  }

  // ------------------------------------------------------------ compute warps
  const int g = lane >> 2, c4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * (NS * C::kStageBytes);
  const I4Magic magic;

  // ---- the stream of block pairs: this warp's share of unit k, then of unit k+1
  int iss_unit = -1;                // unit being issued
  int iss_bl = 0, iss_n = 0;        // its next pair's first block, its blocks
  const unsigned char* iss_k = nullptr;  // block 0's K page of its head, at this lane's 16 bytes
  const uint32_t block_stride = static_cast<uint32_t>(Hkv) * Pg::kBytes;
  const long long k_to_v = static_cast<const unsigned char*>(p.v_cache) -
                           static_cast<const unsigned char*>(p.k_cache) - Pg::kBytes;
  bool iss_end = false;             // no unit after it
  int iss_st = 0, in_flight = 0;    // ring stage of the next issue, stages under way

  // Issue the next pair if it lies in unit `limit` or earlier and is known.
  auto issue_one = [&](int limit) -> bool {
    while (iss_bl >= iss_n) {
      if (iss_unit >= limit || iss_end) return false;
      const int k = iss_unit + 1;
      // (one answer for the warp: lanes that saw the unit at different steps would
      // fill different stages)
      if (!__all_sync(0xffffffffu, mbar_test(bar_unit + (k & 1) * 8, (k >> 1) & 1))) return false;
      const UnitMeta& m = meta(k);
      iss_unit = k;
      iss_end = m.valid == 0;
      iss_n = m.valid ? m.b1 - m.b0 : 0;
      iss_bl = 2 * warp;
      iss_k = static_cast<const unsigned char*>(p.k_cache) + m.g * Pg::kBytes + lane * 16;
    }
    const uint32_t st = ring + iss_st * C::kStageBytes + lane * 16;
    const int32_t* bt = meta(iss_unit).bt + iss_bl;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int phys = bt[b];
      const int bytes = phys >= 0 ? 16 : 0;
      const unsigned char* ks = iss_k + static_cast<unsigned long long>(static_cast<uint32_t>(max(phys, 0))) * block_stride;
      const unsigned char* vs = ks + k_to_v;
#pragma unroll
      for (int i = 0; i < C::kBlockBytes; i += 512)  // the K page, then the V page, 512 bytes a step
        if (i + 512 <= C::kBlockBytes || lane * 16 < C::kBlockBytes - i)
          cp_async16(st + b * C::kBlockBytes + i, (i + lane * 16 < Pg::kBytes ? ks : vs) + i, bytes);
    }
    cp_async_commit();
    iss_st = iss_st + 1 == NS ? 0 : iss_st + 1;
    iss_bl += 2 * NW;
    ++in_flight;
    return true;
  };

  // Merge of a split tile, one float4 of the output a thread; the partials of
  // kMergeChunk splits are loaded before any is used: one L2 round trip for all.
  auto merge_splits = [&](const UnitMeta& u) {
    constexpr int kMergeChunk = 8;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
    for (int idx = warp * 32 + lane; idx < R * D / 4; idx += NW * 32) {
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
        // a split with no visible key for this row holds (-inf, 0) and zeros, one
        // with logits of NaN alone (-inf, NaN)
        float mc = M;
#pragma unroll
        for (int j = 0; j < kMergeChunk; ++j) mc = fmaxf(mc, ml[j].x);
        if (mc == -CUDART_INF_F) {
#pragma unroll
          for (int j = 0; j < kMergeChunk; ++j) den += ml[j].y;  // 0, or NaN
          continue;
        }
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
  };

  int cur_st = 0;  // ring stage of the next pair to compute
  for (int k = 0;; ++k) {
    if (!wait_for(bar_unit + (k & 1) * 8, (k >> 1) & 1)) break;
    const UnitMeta& cur = meta(k);
    if (!cur.valid) break;
    if (iss_unit < k - 1) {  // units before this one need no copies any more
      iss_unit = k - 1;
      iss_n = 0;
    }
    if (cur.valid == 2) {
      merge_splits(cur);
      // (an arrival for this unit must not count for the one before, see below)
      if (k >= NB && !wait_for(bar_free + (k % NB) * 8, (k / NB - 1) & 1)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_full + (k % NB) * 8);
      continue;
    }
    while (in_flight < NS && issue_one(k + 1)) {
    }
    const int nblk = cur.b1 - cur.b0;
    const int pos0 = cur.pos0, kv_hi = cur.kv_hi;
    const int plain_end = min(pos0 + 1, kv_hi) - 2 * kBlockSize;  // no mask up to this first key
    // q^T fragments, the group sums' and the rows' factors
    uint32_t qb[NG][4], zb[2];
    float rm[2];
    {
      const unsigned char* buf = smem + C::kQOff + (k & 1) * C::kQBufBytes;
      const int r = min(g, R - 1);  // (columns past the last row repeat it)
      const uint32_t row = smem_u32(buf) + r * C::kQRowBytes + c4 * 16;
#pragma unroll
      for (int e = 0; e < NG; ++e) lds_words<4>(row + e * 64, qb[e]);
      const uint32_t* zs = reinterpret_cast<const uint32_t*>(buf + R * C::kQRowBytes + r * 32);
      zb[0] = zs[c4];
      zb[1] = zs[4 + c4];
      const float* fr = reinterpret_cast<const float*>(buf + R * (C::kQRowBytes + 32));
      rm[0] = fr[min(2 * c4, R - 1)];
      rm[1] = fr[min(2 * c4 + 1, R - 1)];
    }
    // running state of rows 2 c4, 2 c4 + 1: maximum (before the row factor), the
    // value that moves it, the lift minus the maximum's logit, sum; O^T
    float o[MT][4];
    float m[2], thr[2], mneg[2], l[2];
#pragma unroll
    for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    m[0] = m[1] = thr[0] = thr[1] = -CUDART_INF_F;
    mneg[0] = mneg[1] = l[0] = l[1] = 0.f;
    for (int bl = 2 * warp; bl < nblk; bl += 2 * NW) {
      if (in_flight == NS) cp_async_wait<NS - 1>(); else cp_async_wait<0>();
      __syncwarp();
      const uint32_t stage = ring + cur_st * C::kStageBytes;
      const int tok0 = (cur.b0 + bl) * kBlockSize;
      // S^T of keys g, g + 8 of both blocks
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t kp = stage + j * C::kBlockBytes;
        uint32_t kw[2][NG], sw[2][NG / 2], zw[2][1];  // codes, scales, the lane's pair of zeros
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          lds_words<NG>(kp + Pg::k_word(g + 8 * h, 0, c4), kw[h]);
          lds_words<NG / 2>(kp + Pg::k_scale(g + 8 * h, 0), sw[h]);
          // lane c4 takes groups 2 c4, 2 c4 + 1 (modulo the groups)
          lds_words<1>(kp + Pg::k_scale(g + 8 * h, 0) + 2 * NG + (NG == 4 ? (c4 & 1) * 4 : 0), zw[h]);
        }
        const uint32_t za[4] = {zw[0][0], zw[1][0], zw[0][0], zw[1][0]};
        mma_f16_zero(s[j], za, zb[0], zb[1]);
#pragma unroll
        for (int e = 0; e < NG; ++e) {
          const uint32_t k0 = kw[0][e] >> 8, k1 = kw[1][e] >> 8;
          const uint32_t a[4] = {kw[0][e] & 0x000f000fu, kw[1][e] & 0x000f000fu, k0 & 0x000f000fu,
                                 k1 & 0x000f000fu};
          const uint32_t b[4] = {kw[0][e] & 0x00f000f0u, kw[1][e] & 0x00f000f0u, k0 & 0x00f000f0u,
                                 k1 & 0x00f000f0u};
          const float2 f0 = half2_floats(sw[0][e / 2]), f1 = half2_floats(sw[1][e / 2]);
          const float s0 = (e & 1) ? f0.y : f0.x, s1 = (e & 1) ? f1.y : f1.x;
          float acc[4];
          mma_f16_zero(acc, a, qb[e][0], qb[e][1]);
          mma_f16(acc, b, qb[e][2], qb[e][3]);
          s[j][0] = fmaf(acc[0], s0, s[j][0]);
          s[j][1] = fmaf(acc[1], s0, s[j][1]);
          s[j][2] = fmaf(acc[2], s1, s[j][2]);
          s[j][3] = fmaf(acc[3], s1, s[j][3]);
        }
      }
      // V parameters: scales and zeros of tokens (2 c4, 2 c4 + 1) and
      // (2 c4 + 8, 2 c4 + 9), all in the group of the lane's run of dims
      uint32_t vq[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        lds_words<4>(stage + j * C::kBlockBytes + Pg::kBytes + Pg::kCodeBytes + (g * Pg::kRun / 32) * 64 +
                         c4 * 16,
                     vq[j]);
      if (tok0 > plain_end) {
        // causal edge, unwritten slots or no second block (K, V and parameters
        // there may be anything)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int tj = tok0 + j * kBlockSize;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = tj + g + 8 * (e >> 1);
            const int jj = (2 * c4 + (e & 1)) / G;
            if (tok >= kv_hi || tok > pos0 + jj) s[j][e] = -CUDART_INF_F;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int left = kv_hi - (tj + 2 * c4 + 8 * h);  // written tokens of the pair
            const uint32_t keep = left >= 2 ? 0xffffffffu : (left == 1 ? 0x0000ffffu : 0u);
            vq[j][h] &= keep;
            vq[j][2 + h] &= keep;
          }
        }
      }
      // online softmax
      auto step_max = [&](int e) {
        return fmaxf(fmaxf(s[0][e], s[0][2 + e]), fmaxf(s[1][e], s[1][2 + e]));
      };
      if (__any_sync(0xffffffffu, step_max(0) > thr[0] || step_max(1) > thr[1])) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(m[e], step_max(e));
#pragma unroll
          for (int o8 = 4; o8 < 32; o8 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o8));
          if (mx > m[e]) {
            // (rounded down: at logits of 2^23, whose steps are 1, roundings to nearest
            // could put P past f16's end)
            const float mn = __fmaf_rd(-mx, rm[e], kI4Lift);
            const float corr = m[e] == -CUDART_INF_F ? 0.f : ex2_approx(mn - mneg[e]);
            m[e] = mx;
            thr[e] = __fadd_rd(mx, kI4Rescale / rm[e]);
            mneg[e] = mn;
            l[e] *= corr;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[mt][e] *= corr;
              o[mt][2 + e] *= corr;
            }
          }
        }
      }
      uint32_t pb[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[e] = ex2_approx(fmaf(s[j][e], rm[e & 1], mneg[e & 1]));
        l[0] += pr[0] + pr[2];
        l[1] += pr[1] + pr[3];
        // P^T as the B operand: an 8 x 8 transpose per half of the block's keys
        pb[j][0] = movm_trans(pack_f16(pr[0], pr[1]));
        pb[j][1] = movm_trans(pack_f16(pr[2], pr[3]));
      }
      // O^T += V^T P^T
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t vp = stage + j * C::kBlockBytes + Pg::kBytes;
        uint32_t vw[2][NG];
#pragma unroll
        for (int h = 0; h < 2; ++h) lds_words<NG>(vp + h * 4 * D + g * (D / 2) + c4 * Pg::kRun, vw[h]);
        const uint32_t s0 = vq[j][0], s1 = vq[j][1], z0 = vq[j][2], z1 = vq[j][3];
#pragma unroll
        for (int w = 0; w < NG; ++w) {
          const uint32_t w0 = vw[0][w] >> 8, w1 = vw[1][w] >> 8;
          const uint32_t a[4] = {int4_values<0>(vw[0][w], s0, z0, magic), int4_values<1>(vw[0][w], s0, z0, magic),
                                 int4_values<0>(vw[1][w], s1, z1, magic), int4_values<1>(vw[1][w], s1, z1, magic)};
          const uint32_t b[4] = {int4_values<0>(w0, s0, z0, magic), int4_values<1>(w0, s0, z0, magic),
                                 int4_values<0>(w1, s1, z1, magic), int4_values<1>(w1, s1, z1, magic)};
          mma_f16(o[2 * w], a, pb[j][0], pb[j][1]);
          mma_f16(o[2 * w + 1], b, pb[j][0], pb[j][1]);
        }
      }
      __syncwarp();  // the stage has been read: the stream's next pair goes into it
      cur_st = cur_st + 1 == NS ? 0 : cur_st + 1;
      --in_flight;
      issue_one(k + 1);
    }
    // the warp's state for this unit -> shared memory (real rows only), once the
    // unit that used the buffer before has been read: by then every warp has
    // arrived for that unit, so no phase completes without one of them
    if (k >= NB && !wait_for(bar_free + (k % NB) * 8, (k / NB - 1) & 1)) break;
    float* cb = comb + (k % NB) * NW * R * D;
    float* cm = comb_ml + (k % NB) * NW * R * 2;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[e];
#pragma unroll
      for (int o8 = 4; o8 < 32; o8 <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o8);
      const int row = 2 * c4 + e;
      if (row < R) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          *reinterpret_cast<float2*>(cb + (warp * R + row) * D + (D / 8) * g + 2 * mt) =
              make_float2(o[mt][e], o[mt][2 + e]);
        if (g == 0) {
          // (the logit whose P is 1, so that the lift cancels in the merges)
          cm[(warp * R + row) * 2] = m[e] == -CUDART_INF_F ? m[e] : -mneg[e];
          cm[(warp * R + row) * 2 + 1] = sum;
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_full + (k % NB) * 8);
  }
  cp_async_wait<0>();
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

// CTAs of four compute warps, three to an SM at 128 registers a thread.  Two stages
// of two blocks (head size 64: four) keep 120 KB of pages per SM in flight or in
// use; three stages and two CTAs, or four CTAs of three warps, were slower (long
// context: 375 and 347 us instead of 320).
template <int D, int G>
cudaError_t dispatch_positions_int4(const AttnParams& p, int positions, int num_sms,
                                    cudaStream_t stream, int* grid_only) {
  return positions == 1
             ? launch_i4<D, G, 1, 4, D == 128 ? 2 : 4>(p, num_sms, stream, grid_only)
             : launch_i4<D, G, kSmallRowsInt4 / G, 4, D == 128 ? 2 : 4>(p, num_sms, stream, grid_only);
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
