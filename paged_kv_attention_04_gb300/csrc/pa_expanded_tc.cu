// Latent attention in the expanded form on the 5th-generation tensor cores: ragged requests whose heads
// have keys [k_nope (D), k_rope (64, shared by the heads)] and values (D) of their own, causal
// from the bottom right.
//
// A (query, key) pair costs 2 (2 D + 64) flops and no bytes worth counting, so the tensor cores
// bound it.  A unit is 256 rows of one head of a request, two tiles of 128 that read every
// staged K and V tile.  S = Q K' takes Q and K from shared memory, O += P V takes P from tensor memory.
// A step of 80 keys leaves room in tensor memory for P beside its S (2 x (80 + 40) columns, and the two
// O in the other half), so the next S is formed while the softmax works on this one, and neither
// the tensor cores nor the softmax wait for a hand-over.  (With P over S, 96 keys: 2870 cycles a step of
// which the products are 2112; 128 keys, one and a half stages of K and V: 4400 of 2560.)
// Shared memory holds the two Q tiles, K of three key tiles and V of two (D = 64: four), in slices of 64
// numbers (128-byte swizzle).
//
// Roles: warps 0-3 and 4-7 softmax and output of one tile each, a thread a row: no
// trade between threads; O is rescaled only when a row's maximum grows by more than 2^8.  Warp 8
// units and copies of Q and K, warp 11 copies of V, warp 9 issues the S products, warp 10 the O
// products (while S is formed, shared memory is busy and a wait costs some 200 cycles even for what
// is there: each hides the other's).
// A thread holds a row's 80 logits, so the softmax warps take 208 registers of the 168 that the launch
// gives every thread, the others 88.
//
// Work: where a CTA gets a few long units, they lie on a line in request, head, row order, each as long
// as its key tiles; every CTA takes an equal stretch, cut units leave partial states (two a
// CTA at most), and a second kernel joins them in order.  Where it gets many, whole units are
// dealt out by length, the longest first and every other round backwards (of more than 32 requests:
// the units whose middle lies in the CTA's stretch).
//
// Measured (D = 128, 32 heads): 2048 tokens over 8192 keys 221 us (301 GFLOP, 71 % of the bf16 peak; 2430 cycles a
// step whose products are 1888), 6 prompts of 300 to 2048 tokens 109 us.
#include <math_constants.h>

#include "pa_latent.h"
#include "pa_tc_util.cuh"

namespace pa {

namespace {

using namespace tc;

constexpr int kRows = 128, kUnitRows = 256, kKeys = 80;
constexpr int kCopyWarp = 8, kSWarp = 9, kOWarp = 10, kVWarp = 11;
constexpr int kThreads = 384;
constexpr int kSoftRegs = 208, kOtherRegs = 88;  // 256 x 208 + 128 x 88 = 384 x 168
constexpr int kQSlice = kRows * 128, kKSlice = kKeys * 128;  // bytes of 64 numbers of a tile
constexpr float kGrowth = 8.f;
constexpr int kUnitCost = 0;       // what a unit costs beside its key tiles (measured: nothing, its start
                                   // and output run beside other units' products)
// Fewest key tiles of a piece.  32 heads, 2048 rows over 8192 keys: 220 us with 3, 221 with 6, 226 with 12, 247 with
// 24; few short units (4 heads, 300 rows over 3000 keys) 20, 24, 37 and 55.
constexpr int kMinPiece = 6;
// Units are cut where a request may be this long and a CTA would get fewer units than kCutUnits if the step's rows
// were one request's (requests of few rows are more units than that).  Measured in us, cut and whole, D = 128, 32 heads
// unless said: rows over 8192 keys: 32: 37 and 78, 256: 51 and 134, 1024: 128 and 136, 2048: 221 and 233, 4096 (3.4
// units a CTA): 360 and 380, 8192 (6.7): 494 and 490; 96 heads, 2048 rows (5.1): 630 and 750.  256 rows over 512 keys:
// 18 and 14, over 1024: 27 and 22, over 2048: 28 and 38.  What the rule does not look at, and cuts at a loss: prompts
// with few earlier tokens (2048 rows over 2048 keys 55 and 41, 4096 over 4096 150 and 131) and many short
// chunks (64 of 32 rows over 4128 keys 783 and 720).
constexpr int kCutKeys = 1024, kCutUnits = 5;

template <int D>
struct ECfg {
  static constexpr int kQSlices = D / 64 + 1, kVSlices = D / 64;
  static constexpr int kQBytes = kQSlices * kQSlice;
  static constexpr int kKBytes = kQSlices * kKSlice, kVBytes = kVSlices * kKSlice;
  // (S runs a step ahead, so K needs a stage more than V: with two of each 254 us a 2048-token chunk)
  static constexpr int kKStages = D == 128 ? 3 : 4, kVStages = D == 128 ? 2 : 4;
  static constexpr int kKOff = 2 * kQBytes, kVOff = kKOff + kKStages * kKBytes;
  static constexpr int kSmallOff = kVOff + kVStages * kVBytes;
  static constexpr int kSmemBytes = kSmallOff + 1024;
  // row tile w: S at 128 w, its P behind it, O at 256 + D w
  static constexpr int kTmemP = kKeys, kTmemO = 256;
  static_assert(kKeys + kKeys / 2 <= kRows, "P fits behind S");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA exceeds 227 KB");
};

struct EUnit {
  int r;       // < 0: no more units
  int head;
  int row0;    // first row of the step
  int rows;    // valid rows (up to 256)
  int pos0;    // key position of the first row
  int key0;    // first key of the request in the step
  int seq;     // keys of the request
  int t0;      // first key tile
  int n[2];    // key tiles of each row tile, from t0 on
  int slot;    // partial state, -1: the whole unit
};

enum EBar : int {
  eUnitFull = 0,   // [2]
  eUnitEmpty = 2,  // [2] (8 softmax warps, 2 MMA, V)
  eQFull = 4,      // [2] TMA, by row tile
  eQEmpty = 6,     // [2] the unit's last S of the row tile done
  eSFull = 8,      // [2] S done, by row tile
  eSRead = 10,     // [2] ... and read (4 warps)
  ePFull = 12,     // [2] P written, O rescaled (4 warps)
  eODone = 14,     // [2] O += P V done
  eVLand = 16,     // a V tile whose last rows are zeroed landed
  eDrain = 17,     // [2]
  eKFull = 19,     // [4] K landed, by stage
  eKEmpty = 23,    // [4] ... and read
  eVFull = 27,     // [4]
  eVEmpty = 31,    // [4]
  eNumBars = 35
};

struct ESmall {
  uint64_t bars[eNumBars];
  EUnit units[2];
  long long sums[kThreads / 32];
  long long start_pos, total;
  uint32_t tmem;
  int abort, bad, start_r, ctas;
};
static_assert(sizeof(ESmall) <= 1024, "small shared memory");

struct ESpan {
  int a, L, ka, S, tiles;  // rows, keys, row units of a head
  long long head_len;      // line length of one head
};

// key tiles that rows up to position `last` see
__device__ __forceinline__ int tiles_to(int last) { return last / kKeys + 1; }
__device__ __forceinline__ int unit_len(const ESpan& s, int m) {
  return tiles_to(s.S - s.L + min((m + 1) * kUnitRows, s.L) - 1) + kUnitCost;
}

__device__ __forceinline__ int span_of(const ExpandedParams& p, int r, ESpan& s) {
  s.a = __ldg(p.qsl + r);
  s.ka = __ldg(p.kvsl + r);
  const int b = __ldg(p.qsl + r + 1), kb = __ldg(p.kvsl + r + 1);
  s.L = b - s.a;
  s.S = kb - s.ka;
  s.tiles = 0;
  s.head_len = 0;
  if (s.L < 0 || s.a < 0 || b > p.num_tokens || s.S < 0 || s.ka < 0 || kb > p.num_kv_tokens ||
      (r == 0 && (s.a != 0 || s.ka != 0)) ||
      (r == p.num_seqs - 1 && (b != p.num_tokens || kb != p.num_kv_tokens)))
    return PA_DEV_QSL;
  if (s.L < 1 || s.L > s.S || s.S > p.max_kv_len || s.L > p.max_query_len) return PA_DEV_LENGTHS;
  s.tiles = (s.L + kUnitRows - 1) / kUnitRows;
  for (int m = 0; m < s.tiles; ++m) s.head_len += unit_len(s, m);
  return 0;
}

struct EMaps {
  CUtensorMap q, k, kr, v;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// (a0, a1) = (a0, a1) * b + c in one instruction
__device__ __forceinline__ void fma2(float& a0, float& a1, float b, float c) {
  asm("{\n .reg .b64 ra, rb, rc;\n mov.b64 ra, {%0, %1};\n mov.b64 rb, {%2, %2};\n"
      " mov.b64 rc, {%3, %3};\n fma.rn.f32x2 ra, ra, rb, rc;\n mov.b64 {%0, %1}, ra;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
  asm("{\n .reg .b64 ra, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rd, {%0, %1};\n"
      " add.rn.f32x2 rd, rd, ra;\n mov.b64 {%0, %1}, rd;\n}\n"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    expanded_tc_kernel(const ExpandedParams p, const __grid_constant__ EMaps maps) {
  using C = ECfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  ESmall& sm = *reinterpret_cast<ESmall*>(smem + C::kSmallOff);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sm.abort;
  auto bar = [&](int i) { return smem_u32(&sm.bars[i]); };

  if (tid == kCopyWarp * 32) {
    prefetch_map(&maps.q);
    prefetch_map(&maps.k);
    prefetch_map(&maps.kr);
    prefetch_map(&maps.v);
  }
  // few requests and whole units: the copy warp alone looks at the lengths, a lane a request
  const bool dealt = !p.part_acc && p.num_seqs <= 32;
  ESpan mine{};
  int err = 0;
  if (tid == 0) {
    for (int i = 0; i < eNumBars; ++i) {
      uint32_t n = 1;
      if (i == eUnitEmpty || i == eUnitEmpty + 1) n = 11;
      if (i >= eSRead && i < eSRead + 4) n = 4;  // (eSRead, ePFull)
      mbar_init(bar(i), n);
    }
    // (the swizzled tiles need the alignment that the declaration asks for)
    sm.abort = (sbase & 1023) != 0;
    if (sbase & 1023) flag_error(p.status, PA_DEV_TIMEOUT);
    sm.bad = 0;
    sm.start_r = -1;
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(smem_u32(&sm.tmem), 512);
  wait_prior_grid();  // (the lengths, like everything else, may be the kernel's before)
  launch_dependents();  // (the joining kernel's launch; it waits for this grid)
  if (dealt && warp == kCopyWarp && lane < p.num_seqs) err = span_of(p, lane, mine);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  // ---- this CTA's stretch of the line, beginning in request start_r
  long long lo = 0, hi = 0;
  if (!dealt) {
    const int per = (p.num_seqs + kThreads - 1) / kThreads;
    const int ra = min(tid * per, p.num_seqs), rb = min(ra + per, p.num_seqs);
    long long line = 0, total = 0;  // this thread's requests, all
#pragma unroll 1
    for (int r = ra; r < rb; ++r) {
      ESpan s;
      err |= span_of(p, r, s);
      line += s.head_len * p.num_heads;
    }
    if (err) {
      if (blockIdx.x == 0) flag_error(p.status, err);
      if (err & PA_DEV_QSL) sm.bad = 1;
    }
    long long before = line;  // inclusive scan over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    if (lane == 31) sm.sums[warp] = before;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sm.sums[w];
      total += sm.sums[w];
    }
    before -= line;
    if (sm.bad) total = 0;
    // (cut units: every stretch is long enough for a piece)
    const long long ctas = p.part_acc ? max(1LL, min(static_cast<long long>(gridDim.x), total / (kUnitCost + kMinPiece)))
                                      : gridDim.x;
    if (blockIdx.x < ctas) {
      lo = total * blockIdx.x / ctas;
      hi = total * (blockIdx.x + 1) / ctas;
    }
    if (tid == 0) {
      sm.total = total;
      sm.ctas = static_cast<int>(ctas);
    }
    if (lo < hi && before <= lo && lo < before + line) {
      long long pos = before;
#pragma unroll 1
      for (int r = ra; r < rb; ++r) {
        ESpan s;
        span_of(p, r, s);
        const long long len = s.head_len * p.num_heads;
        if (lo < pos + len) {
          sm.start_r = r;
          sm.start_pos = pos;
          break;
        }
        pos += len;
      }
    }
    __syncthreads();
  }

  if (warp >= kCopyWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == kCopyWarp) {
      // ------------------------------------------------------------ units and copies
      int uc = 0;                    // units published
      uint32_t nk = 0;               // K tiles copied
      uint32_t nq[2] = {0, 0};       // Q tiles copied
      bool ok = !*abort;
      if (lane < 2 && p.recs) p.recs[blockIdx.x * 2 + lane] = make_int4(0, 0, 0, 0);
      __syncwarp();
      auto publish = [&](const EUnit& u) {
        const int s = uc & 1;
        if (uc >= 2 && !wait_bar(bar(eUnitEmpty + s), ((uc >> 1) - 1) & 1, abort, p.status)) return false;
        if (lane == 0) {
          sm.units[s] = u;
          mbar_arrive(bar(eUnitFull + s));
        }
        __syncwarp();
        ++uc;
        return true;
      };
      auto load_q = [&](const EUnit& u, int w) {
        if (u.n[w] == 0) return true;
        if (nq[w] > 0 && !wait_bar(bar(eQEmpty + w), (nq[w] - 1) & 1, abort, p.status)) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(eQFull + w), C::kQBytes);
#pragma unroll
          for (int s = 0; s < C::kQSlices; ++s)
            tma_load_3d(sbase + w * C::kQBytes + s * kQSlice, &maps.q, s * 64, u.head, u.row0 + w * kRows,
                        bar(eQFull + w));
        }
        __syncwarp();
        ++nq[w];
        return true;
      };
      auto load_k = [&](const EUnit& u, int t) {
        const uint32_t b = nk % C::kKStages;
        if (nk >= C::kKStages && !wait_bar(bar(eKEmpty + b), (nk / C::kKStages - 1) & 1, abort, p.status)) return false;
        if (lane == 0) {
          const uint32_t full = bar(eKFull + b);
          mbar_arrive_expect_tx(full, C::kKBytes);
#pragma unroll
          for (int s = 0; s < C::kQSlices; ++s) {
            const uint32_t dst = sbase + C::kKOff + b * C::kKBytes + s * kKSlice;
            if (s < C::kVSlices) tma_load_3d(dst, &maps.k, s * 64, u.head, u.key0 + t * kKeys, full);
            else tma_load_2d(dst, &maps.kr, 0, u.key0 + t * kKeys, full);
          }
        }
        __syncwarp();
        ++nk;
        return true;
      };
      auto run = [&](const EUnit& u) {
        const int n = max(u.n[0], u.n[1]);
        if (!publish(u) || !load_k(u, u.t0) || !load_q(u, 0) || !load_q(u, 1)) return false;
        for (int t = 1; t < n; ++t)
          if (!load_k(u, u.t0 + t)) return false;
        return true;
      };
      auto unit_of = [&](const ESpan& s, int r, int h, int m) {
        EUnit u;
        u.r = r;
        u.head = h;
        u.row0 = s.a + m * kUnitRows;
        u.rows = min(kUnitRows, s.L - m * kUnitRows);
        u.pos0 = s.S - s.L + m * kUnitRows;
        u.key0 = s.ka;
        u.seq = s.S;
        u.t0 = 0;
        u.n[0] = tiles_to(u.pos0 + min(kRows, u.rows) - 1);
        u.n[1] = u.rows > kRows ? tiles_to(u.pos0 + u.rows - 1) : 0;
        u.slot = -1;
        return u;
      };
      if (dealt) {
        // a lane a request: its units have levels, 256 keys apart, and come in order of these
        ESpan s = mine;
        err = __reduce_or_sync(0xffffffffu, err);
        if (err && blockIdx.x == 0 && lane == 0) flag_error(p.status, err);
        if (err & PA_DEV_QSL) s.tiles = 0;
        const int low = (s.S - s.L) / kUnitRows;
        int level = __reduce_max_sync(0xffffffffu, s.tiles ? low + s.tiles - 1 : -1);
        long long base = 0;  // units of higher levels
        for (int round = 0; ok && level >= 0; ++round) {
          const long long i = static_cast<long long>(round) * gridDim.x +
                              ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
          uint32_t with = 0;
          for (; level >= 0; --level) {
            with = __ballot_sync(0xffffffffu, level >= low && level < low + s.tiles);
            const long long n = static_cast<long long>(__popc(with)) * p.num_heads;
            if (i < base + n) break;
            base += n;
          }
          if (level < 0) break;
          const int j = static_cast<int>(i - base), r = __fns(with, 0, j / p.num_heads + 1);
          ESpan t;
          t.a = __shfl_sync(0xffffffffu, s.a, r);
          t.L = __shfl_sync(0xffffffffu, s.L, r);
          t.ka = __shfl_sync(0xffffffffu, s.ka, r);
          t.S = __shfl_sync(0xffffffffu, s.S, r);
          ok = run(unit_of(t, r, j % p.num_heads, level - (t.S - t.L) / kUnitRows));
        }
      } else if (ok && sm.start_r >= 0) {
        long long pos = sm.start_pos;
        for (int r = sm.start_r; ok && r < p.num_seqs && pos < hi; ++r) {
          ESpan s;
          span_of(p, r, s);
          if (s.tiles == 0) continue;
          int h = lo > pos ? static_cast<int>((lo - pos) / s.head_len) : 0;
          for (; ok && h < p.num_heads; ++h) {
            long long at = pos + h * s.head_len;
            if (at >= hi) break;
            for (int m = 0; ok && m < s.tiles; ++m) {
              const int len = unit_len(s, m);
              const long long at0 = at;
              at += len;
              if (at <= lo) continue;
              if (at0 >= hi) break;
              // where a border of the line cuts the unit: 0 (in front of it) .. len (behind it)
              auto cut = [&](long long x) {
                if (x <= at0) return 0;
                if (x >= at) return len;
                const int rel = static_cast<int>(x - at0);
                if (!p.part_acc) return 2 * rel > len ? len : 0;
                return rel < kUnitCost + kMinPiece ? 0 : len - rel < kMinPiece ? len : rel;
              };
              const int c0 = cut(lo), c1 = cut(hi);
              if (c0 >= c1) continue;
              EUnit u = unit_of(s, r, h, m);
              const int t1 = c1 == len ? len - kUnitCost : c1 - kUnitCost;
              u.t0 = c0 == 0 ? 0 : c0 - kUnitCost;
              u.n[0] = max(0, min(t1, u.n[0]) - u.t0);
              if (u.n[1]) u.n[1] = t1 - u.t0;
              const bool whole = c0 == 0 && c1 == len;
              u.slot = whole ? -1 : static_cast<int>(blockIdx.x) * 2 + (c0 == 0);
              if (!whole) {  // borders inside the unit, before this piece and behind it
                int piece = 0, pieces = 1;
                for (int c = blockIdx.x; c > 0 && cut(sm.total * c / sm.ctas) > 0; --c) ++piece;
                for (int c = blockIdx.x + 1; c < sm.ctas && cut(sm.total * c / sm.ctas) < len; ++c) ++pieces;
                if (lane == 0) p.recs[u.slot] = make_int4(u.row0, u.rows, h, piece | (piece + pieces) << 16);
              }
              ok = run(u);
            }
          }
          pos += s.head_len * p.num_heads;
        }
      }
      EUnit end{};
      end.r = -1;
      if (ok) publish(end);
      if (*abort) {  // let every copy issued land before the CTA ends
        for (uint32_t i = nk > C::kKStages ? nk - C::kKStages : 0; i < nk; ++i)
          drain_wait(bar(eKFull + i % C::kKStages), (i / C::kKStages) & 1);
        for (int w = 0; w < 2; ++w)
          if (nq[w] > 0) drain_wait(bar(eQFull + w), (nq[w] - 1) & 1);
      }
      __syncwarp();
    } else if (warp == kVWarp) {
      // ------------------------------------------------------------ copies of V
      uint32_t nv = 0, nland = 0;    // V tiles copied, those of them whose last rows are zeroed
      bool landing = false, ok = !*abort;
      auto load_v = [&](const EUnit& u, int t) {
        const uint32_t b = nv % C::kVStages;
        if (nv >= C::kVStages && !wait_bar(bar(eVEmpty + b), (nv / C::kVStages - 1) & 1, abort, p.status)) return false;
        // rows behind the request's last key hold another's values or nothing: zeros, so that
        // a weight of zero meets no NaN
        const int rows = u.seq - t * kKeys;
        const bool trim = rows < kKeys;
        const uint32_t full = bar(eVFull + b), land = trim ? bar(eVLand) : full, dst = sbase + C::kVOff + b * C::kVBytes;
        if (lane == 0) {
          mbar_arrive_expect_tx(land, C::kVBytes);
#pragma unroll
          for (int s = 0; s < C::kVSlices; ++s)
            tma_load_3d(dst + s * kKSlice, &maps.v, s * 64, u.head, u.key0 + t * kKeys, land);
        }
        __syncwarp();
        if (trim) {
          landing = true;
          if (!wait_bar(land, nland & 1, abort, p.status)) return false;
          landing = false;
          ++nland;
          for (int i = lane; i < (kKeys - rows) * C::kVSlices * 8; i += 32) {
            const int c = i % 8, s = i / 8 % C::kVSlices, row = rows + i / (8 * C::kVSlices);
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(dst + s * kKSlice + row * 128 + c * 16),
                         "r"(0u)
                         : "memory");
          }
          fence_proxy_async_smem();
          warp_arrive(full);
        }
        ++nv;
        return true;
      };
      for (int uc = 0; ok; ++uc) {
        if (!wait_bar(bar(eUnitFull + (uc & 1)), (uc >> 1) & 1, abort, p.status)) break;
        const EUnit u = sm.units[uc & 1];
        warp_arrive(bar(eUnitEmpty + (uc & 1)));
        if (u.r < 0) break;
        for (int t = 0; ok && t < max(u.n[0], u.n[1]); ++t) ok = load_v(u, u.t0 + t);
      }
      if (*abort) {
        for (uint32_t i = nv > C::kVStages ? nv - C::kVStages : 0; i < nv; ++i)
          drain_wait(bar(eVFull + i % C::kVStages), (i / C::kVStages) & 1);
        if (landing) drain_wait(bar(eVLand), nland & 1);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ MMA issue, one thread each
      if (elect_one() && !*abort) {
        auto adv = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };
        auto wait = [&](int i, uint32_t parity) { return wait_one(bar(i), parity, abort, p.status); };
        uint32_t b = 0, phase = 0;   // stage of the step's K (V), and its round
        uint32_t num[2] = {0, 0};    // tiles of each row tile so far
        uint32_t nq[2] = {0, 0};     // Q tiles so far
        bool ok = true;
        for (int uc = 0; ok; ++uc) {
          const int slot = uc & 1;
          if (!wait(eUnitFull + slot, (uc >> 1) & 1)) break;
          const bool end = sm.units[slot].r < 0;
          const int n[2] = {sm.units[slot].n[0], sm.units[slot].n[1]};
          mbar_arrive(bar(eUnitEmpty + slot));
          if (end) break;
          const int steps = max(n[0], n[1]);
          if (warp == kSWarp) {
            constexpr uint32_t kId = idesc_bf16(kRows, kKeys, 0);
            for (int t = 0; ok && t < steps; ++t) {
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                if (!ok || t >= n[w]) continue;
                if (t == 0) ok = wait(eQFull + w, nq[w]++ & 1);
                // (phase -1 of a barrier counts as complete)
                if (ok) ok = wait_both(bar(eKFull + b), phase, bar(eSRead + w), (num[w] - 1) & 1, abort, p.status);
                if (!ok) continue;
                ++num[w];
                tc_fence_after();
                // (slices one by one: unrolled, the descriptors of all of them spill, and an MMA waits
                // for its own)
                uint64_t qb = smem_desc_sw128(sbase + w * C::kQBytes, 16, 1024);
                uint64_t kb = smem_desc_sw128(sbase + C::kKOff + b * C::kKBytes, 16, 1024);
#pragma unroll 1
                for (int i = 0; i < C::kQSlices; ++i) {
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    tc_mma_f16(tmem + w * kRows, adv(qb, j * 32), adv(kb, j * 32), kId, i > 0 || j > 0);
                  qb = adv(qb, kQSlice);
                  kb = adv(kb, kKSlice);
                }
                tc_commit(bar(eSFull + w));
                if (t == n[w] - 1) tc_commit(bar(eQEmpty + w));
              }
              if (++b == C::kKStages) b = 0, phase ^= 1;
            }
          } else {
            constexpr uint32_t kId = idesc_bf16(kRows, D, 1);
            for (int t = 0; ok && t < steps; ++t) {
              const uint64_t vb = smem_desc_sw128(sbase + C::kVOff + b * C::kVBytes, kKSlice, 1024);
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                if (!ok || t >= n[w]) continue;
                ok = wait_both(bar(eVFull + b), phase, bar(ePFull + w), num[w]++ & 1, abort, p.status);
                if (!ok) continue;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i)
                  tc_mma_f16_ts(tmem + C::kTmemO + w * D, tmem + w * kRows + C::kTmemP + i * 8, adv(vb, i * 2048),
                                kId, t > 0 || i > 0);
                tc_commit(bar(eODone + w));
              }
              if (ok) tc_commit(bar(eVEmpty + b));
              if (++b == C::kVStages) b = 0, phase ^= 1;
            }
          }
        }
      }
      __syncwarp();
      if (*abort) {  // nothing may still run on tensor memory when it is freed
        const int d = eDrain + (warp == kOWarp);
        if (elect_one()) tc_commit(bar(d));
        __syncwarp();
        drain_wait(bar(d), 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    // ------------------------------------------------------------ softmax and output
    const int w = warp >> 2, i = tid & 127;  // row tile, row
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + w * kRows + lanes, to = tmem + C::kTmemO + w * D + lanes;
    // maxima are taken of logits that grow with S: a negative scale turns S over
    const bool minus = p.scale_log2 < 0.f;
    const float scale = fabsf(p.scale_log2);
    uint32_t ns = 0;    // tiles of this row tile so far
    uint32_t step = 0;  // steps of both
    bool ok = !*abort;
    for (int uc = 0; ok; ++uc) {
      if (!wait_bar(bar(eUnitFull + (uc & 1)), (uc >> 1) & 1, abort, p.status)) break;
      const EUnit u = sm.units[uc & 1];
      warp_arrive(bar(eUnitEmpty + (uc & 1)));
      if (u.r < 0) break;
      const int n = w ? u.n[1] : u.n[0];
      const uint32_t first = step;  // the unit's first step
      if (n == 0) {                 // (no rows, or no key of the piece)
        step += max(u.n[0], u.n[1]);
        if (u.slot >= 0) p.part_ml[static_cast<long long>(u.slot) * kUnitRows + w * kRows + i] = make_float2(-CUDART_INF_F, 0.f);
        continue;
      }
      const int pos = u.pos0 + w * kRows + i;  // keys up to here are seen
      float m = -CUDART_INF_F, l = 0.f;
      for (int t = 0; t < n; ++t, ++ns) {
        if (!wait_bar(bar(eSFull + w), ns & 1, abort, p.status)) { ok = false; break; }
        // K is read, unless row tile 1 is still to take it (here, not by a commit more of the issuing thread)
        if (i == 0 && (w || t >= u.n[1])) mbar_arrive(bar(eKEmpty + step % C::kKStages));
        ++step;
        tc_fence_after();
        float x[kKeys];
        {
          uint32_t(&r)[kKeys] = reinterpret_cast<uint32_t(&)[kKeys]>(x);
          PA_TMEM_LD32(ts, (r + 0));
          PA_TMEM_LD32(ts + 32, (r + 32));
          tmem_ld(ts + 64, reinterpret_cast<uint32_t(&)[16]>(r[64]));
          tmem_wait_ld();
        }
        tc_fence_before();
        warp_arrive(bar(eSRead + w));
        if (minus) {
#pragma unroll
          for (int j = 0; j < kKeys; ++j) x[j] = -x[j];
        }
        if ((u.t0 + t + 1) * kKeys - 1 > u.pos0 + w * kRows) {
          const int last = pos - (u.t0 + t) * kKeys;
#pragma unroll
          for (int j = 0; j < kKeys; ++j)
            if (j > last) x[j] = -CUDART_INF_F;
        }
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(x[j], x[j + 4]);
#pragma unroll
        for (int j = 8; j < kKeys; j += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[j + e], x[j + 4 + e]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
        float f = 1.f;
        if (top > m + kGrowth) {  // (also the first finite maximum: m = -inf)
          f = ex2(m - top);
          m = top;
          l *= f;
        }
        const float ref = m == -CUDART_INF_F ? 0.f : -m;  // (no key seen yet: every weight 0)
        uint32_t pk[kKeys / 2];
#pragma unroll
        for (int j = 0; j < kKeys; j += 2) {
          float &a = x[j], &b = x[j + 1];
          fma2(a, b, scale, ref);
          a = ex2(a);
          b = ex2(b);
          pk[j / 2] = pack_bf16(a, b);
        }
        if (ns > 0 && !wait_bar(bar(eODone + w), (ns - 1) & 1, abort, p.status)) { ok = false; break; }
        tc_fence_after();
        if (t > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld(to + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st(to + c, o);
          }
        }
        PA_TMEM_ST32(ts + C::kTmemP, pk);
        tmem_st(ts + C::kTmemP + 32, reinterpret_cast<uint32_t(&)[8]>(pk[32]));
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar(ePFull + w));
        // the sums while the products run
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kKeys; j += 4) {
          add2(sum[0], sum[1], x[j], x[j + 1]);
          add2(sum[2], sum[3], x[j + 2], x[j + 3]);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      if (!ok) break;
      step = first + max(u.n[0], u.n[1]);
      if (!wait_bar(bar(eODone + w), (ns - 1) & 1, abort, p.status)) break;
      tc_fence_after();
      const int row = w * kRows + i;
      if (u.slot >= 0) {
        // (chunks of 4 numbers by row: a warp's lanes write side by side)
        const long long base = static_cast<long long>(u.slot) * kUnitRows;
        float4* part = p.part_acc + base * (D / 4) + row;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          PA_TMEM_LD32(to + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            part[(c + j) / 4 * kUnitRows] = make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]),
                                                        __uint_as_float(o[j + 2]), __uint_as_float(o[j + 3]));
        }
        p.part_ml[base + row] = make_float2(m, l);
        tc_fence_before();
        continue;
      }
      const float inv = 1.f / l;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) +
                           (static_cast<long long>(u.row0 + row) * p.num_heads + u.head) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        PA_TMEM_LD32(to + c, o);
        tmem_wait_ld();
        if (row < u.rows) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(o[j + e]) * inv;
            *reinterpret_cast<uint4*>(out + c + j) = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                                                pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
          }
        }
      }
      tc_fence_before();
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins the pieces of cut units, in the order of their keys.  Every piece has left a record {first row,
// rows, head, piece and pieces}, and has 8 CTAs; a lane a row, a warp 8 of its numbers, 4 pieces' loads at
// once.  The unit's D warps of work go to the pieces in order, 64 a piece: those of the first piece take
// all of D = 64, those of the first two all of D = 128.
template <int D>
__global__ void __launch_bounds__(256) expanded_join_kernel(const ExpandedParams p) {
  constexpr int kAtOnce = 4;
  wait_prior_grid();
  launch_dependents();  // a following kernel may set up; it waits for this grid
  const int4 recs[2] = {p.recs[blockIdx.x * 2], p.recs[blockIdx.x * 2 + 1]};
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int piece = recs[which].w & 0xffff, pieces = recs[which].w >> 16;
    const int first = blockIdx.x - piece;  // CTA of the first piece
    if (pieces == 0) continue;
    for (int item = (piece * 8 + blockIdx.y) * 8 + (threadIdx.x >> 5); item < kUnitRows / 32 * (D / 8);
         item += pieces * 64) {
      const int row = item / (D / 8) * 32 + (threadIdx.x & 31), chunk = item % (D / 8) * 2;
      if (row >= recs[which].y) break;
      float m = -CUDART_INF_F, l = 0.f;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < pieces; k += kAtOnce) {
        float2 ml[kAtOnce];
        float4 x[kAtOnce][2];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          ml[j].y = 0.f;
          if (k + j < pieces) {  // the first CTA's slot 1, then slot 0 of the following ones
            const long long base = (static_cast<long long>(first + k + j) * 2 + (k + j == 0)) * kUnitRows;
            ml[j] = p.part_ml[base + row];
#pragma unroll
            for (int i = 0; i < 2; ++i) x[j][i] = p.part_acc[base * (D / 4) + (chunk + i) * kUnitRows + row];
          }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          if (ml[j].y == 0.f) continue;  // no key of the piece is seen
          const float nm = fmaxf(m, ml[j].x);
          const float fa = m == nm ? 1.f : ex2(m - nm), fb = ml[j].x == nm ? 1.f : ex2(ml[j].x - nm);
          m = nm;
          l = l * fa + ml[j].y * fb;
          const float y[8] = {x[j][0].x, x[j][0].y, x[j][0].z, x[j][0].w, x[j][1].x, x[j][1].y, x[j][1].z, x[j][1].w};
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = acc[i] * fa + y[i] * fb;
        }
      }
      const float inv = 1.f / l;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] *= inv;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) +
                           (static_cast<long long>(recs[which].x + row) * p.num_heads + recs[which].z) * D;
      *reinterpret_cast<uint4*>(out + chunk * 4) = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                                             pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
    }
  }
}

namespace {

template <int D>
cudaError_t launch_expanded(const ExpandedParams& args, int num_sms, cudaStream_t stream) {
  using C = ECfg<D>;
  static bool configured[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(expanded_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  ExpandedParams p = args;
  // (a scale of zero would make NaN of the masked logits' -inf)
  if (p.scale_log2 == 0.f) p.scale_log2 = 1e-37f;
  EMaps maps;
  const cuuint32_t qbox[3] = {64, 1, kRows}, kbox[3] = {64, 1, kKeys}, rbox[2] = {64, kKeys};
  auto rows3 = [&](CUtensorMap* m, const void* base, int size, long long head_stride, long long stride, int n,
                   const cuuint32_t* box) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(size), static_cast<cuuint64_t>(p.num_heads),
                                static_cast<cuuint64_t>(n)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(stride) * 2};
    return encode_bf16(m, base, 3, dims, strides, box);
  };
  const cuuint64_t dims2[2] = {kLatentRope, static_cast<cuuint64_t>(p.num_kv_tokens)};
  const cuuint64_t strides2[1] = {static_cast<cuuint64_t>(p.kr_stride) * 2};
  if (!rows3(&maps.q, p.q, D + kLatentRope, p.q_head_stride, p.q_stride, p.num_tokens, qbox) ||
      !rows3(&maps.k, p.k, D, p.k_head_stride, p.k_stride, p.num_kv_tokens, kbox) ||
      !rows3(&maps.v, p.v, D, p.v_head_stride, p.v_stride, p.num_kv_tokens, kbox) ||
      !encode_bf16(&maps.kr, p.kr, 2, dims2, strides2, rbox))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  const unsigned ctas = num_sms < kLatentMaxCtas ? num_sms : kLatentMaxCtas;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, expanded_tc_kernel<D>, p, maps);
  if (e != cudaSuccess || !p.part_acc) return e;
  cfg.gridDim = dim3(ctas, 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, expanded_join_kernel<D>, p);
}

}  // namespace

size_t expanded_tc_partial_rows(int num_heads, int num_tokens, int max_kv_len) {
  const long long units = static_cast<long long>(num_heads) * ((num_tokens + kUnitRows - 1) / kUnitRows);
  return max_kv_len < kCutKeys || units >= kCutUnits * kLatentMaxCtas ? 0 : 2 * kLatentMaxCtas * kUnitRows;
}

cudaError_t launch_expanded_tc(const ExpandedParams& p, int head_size, int num_sms, cudaStream_t stream) {
  return head_size == 128 ? launch_expanded<128>(p, num_sms, stream) : launch_expanded<64>(p, num_sms, stream);
}

}  // namespace pa
