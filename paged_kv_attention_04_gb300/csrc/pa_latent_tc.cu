// Attention over a latent cache (absorbed form) on the 5th-generation tensor cores.
//
// All heads of a token read the same row [L, K] of a key (R + 64 numbers, 1152 bytes at
// R = 512), whose first R numbers are the value too: 2 (2 R + 64) flops per head and key
// on 2 (R + 64) bytes, 60 flop/byte at 32 heads, so decode is bound by HBM up to about 128 query
// rows a key.  Every key is staged once and used for both products.
//
// The products are taken transposed, with the keys as M, so that few query rows do not
// pad a tile to 128 rows: S' = [L, K] q' (M = 64 keys, N rows, K = R + 64) and
// O' += L' P' (M = 128 numbers of the latent, R / 128 of them, N rows, K = 64 keys).  N is
// 16, 32 or 64 query rows, a row being a (token, head) of a request.  O' takes R / 128 x N
// columns of tensor memory: 64 rows of 512 are half of it.
// The 64-key tile lies in shared memory as four 16-token pages (a TMA box per 8 keys and part):
//   [8-key group][64-number slice][8 keys][128 bytes], 128-byte swizzle.
// Read with the keys as rows (K-major) it is A of the first product, with the numbers
// as rows (MN-major) A of the second, so there is one copy of it.
//
// Roles: warps 0-3 and 4-7 softmax and output of half of the query rows each, warp 8 units and copies
// (of Q and of the first part of every tile, warp 11 of the second), warps 9 and 10 the issue of S and of
// O.  Two 64-key tiles of R = 512 fill shared memory, and a tile stays for its copy (2 us from HBM),
// S, softmax and O, so this chain is kept short: the copies of the tiles after them are begun as
// prefetches to L2; a tile comes and goes in two parts (half of the latent each, the second with the key
// part), S beginning on the first and O freeing it; P takes the place of the key part, which only
// S reads; O does not wait for the issue of the next S.
// S' has a key per TMEM lane (16 of every 32) and is read as matrix fragments: column maxima by
// shuffles over lanes and a trade between the four warps in shared memory.  The reference
// of a column moves only when its maximum grows by more than 2^8; P is written transposed
// to shared memory by stmatrix as B of the second product.
//
// Work: units (request, N rows) lie on a line, each as long as its keys' tiles plus a
// constant; every CTA takes an equal stretch, computed by itself from the lengths.  Units
// cut by a border leave partial states (at most two a CTA) that a second kernel joins in order.
//
// Measured (R = 512): 256 decodes of 32 heads over a median of 1024 keys 82 us (383 MB, 57 us at the copy
// bandwidth), 16 of 16 heads over 32768 to 131072 keys 250 us (228), 48 requests of 2 to 8 tokens of 32
// heads after 256 to 4096 keys 75 us (bound by the chain above).  So are decodes of more heads: 256 of 64
// heads over that median 94 us (60), of 128 heads 134 us (65), 16 of 128 heads over 8192 to 32768 keys 126 us (58).
#include <math_constants.h>

#include "pa_latent.h"
#include "pa_tc_util.cuh"

namespace pa {

namespace {

using namespace tc;

constexpr int kKeys = 64;           // keys of a tile
constexpr int kPages = kKeys / kBlockSize;
constexpr int kCopyWarp = 8, kSWarp = 9, kOWarp = 10, kCopy2Warp = 11;
constexpr int kThreads = 384;
constexpr int kSoftThreads = 256;
constexpr int kAhead = 2;           // tiles that are prefetched to L2 behind the one to be copied
constexpr float kGrowth = 8.f;      // base-2 growth of a maximum that moves the reference
constexpr int kUnitCost = 2;        // what a unit costs beside its tiles, in tiles
constexpr int kMinStretch = kUnitCost + 1;  // shortest stretch of the line for a CTA: a unit of one tile
constexpr int kWholeTiles = 6;      // units of up to so many tiles are not cut: a join costs 3.5 us

template <int R, int N>
struct Cfg {
  static constexpr int kSlices = (R + kLatentRope) / 64;
  static constexpr int kGroupBytes = kSlices * 1024;       // 8 keys
  static constexpr int kPageBytes = 2 * kGroupBytes;
  static constexpr int kTileBytes = kPages * kPageBytes;
  static constexpr int kQBytes = N * (R + kLatentRope) * 2;  // [slice][N rows][128 bytes]
  static constexpr int kBufs = R == 512 ? 2 : 4;   // tiles
  // P's barriers, one a tile buffer: P of tile g + kBufs waits for the buffer, so for O of tile g, whose issue
  // has then seen this phase.  (Of two in turn with four buffers, P of tile g + 2 could complete the barrier again
  // before the issue of O looked for P of tile g.)
  static constexpr int kPBars = kBufs;
  static constexpr int kQs = N == 64 ? 1 : 2;
  static constexpr int kQOff = kBufs * kTileBytes;
  static constexpr int kSmallOff = kQOff + kQs * kQBytes;
  static constexpr int kSmemBytes = kSmallOff + 3072;
  // parts of a tile: slices 0 .. kHalf - 1, and the others with the key part; P in that one's place,
  // [N rows][128 bytes] with the slice's 1 KB a group of 8
  static constexpr int kHalf = R / 128;
  __host__ __device__ static constexpr int part_bytes(int h) { return kKeys * (kHalf + h) * 128; }
  static constexpr int kPOff = (kSlices - 1) * 1024;
  static constexpr int kBlocks = R / 128;          // of 128 latent numbers
  static constexpr int kTmemS = 256;               // S of even and odd tiles behind O
  static_assert(kBlocks * N <= 256, "O fits beside S");
  static_assert(kPBars <= 4 && (kPBars & (kPBars - 1)) == 0, "P's barriers; tile numbers wrap");
  static_assert(N <= kKeys, "P fits the key part");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA exceeds 227 KB");
};

struct Unit {
  int r;        // request; < 0: no more units
  int row0;     // first row of q and out
  int rows;     // rows of the unit
  int first;    // first row's index in the request (token x heads + head)
  int prior;    // S - L
  int seq;      // S
  int t0, n;    // key tiles
  int slot;     // partial state, -1: the whole unit
};

enum Bar : int {
  kUnitFull = 0,   // [2]
  kUnitEmpty = 2,  // [2] (8 softmax warps, S, O, second copy warp)
  kQFull = 4,      // [2] TMA
  kQEmpty = 6,     // [2] the unit's last S done
  kKFull = 8,      // [4] TMA, the tile's first part; [4] its second
  kKEmpty = 16,    // [4] O += of the first part done: frees it; [4] the second's, and P
  kSFull = 24,     // [2] S done
  kPFull = 26,     // [4] S read, P written, O rescaled (8 warps), by buffer
  kTrade = 30,     // [2] the softmax warps of a half meet (4 warps)
  kDrain = 32,     // [2]
  kNumBars = 34
};

// The line: what request r (rows a .. a + L - 1 of the step, S keys) takes of it.
struct Span {
  int a, L, S, units, len;  // units of this way, each len long
};

struct Small {
  uint64_t bars[kNumBars];
  Unit units[2];
  float mx[2][4][64];   // per warp: column maxima, by tile parity (and row sums)
  float f[64];          // factors of a moved reference; 1 / sum
  uint32_t tmem;
  int abort;
  int start_r;
  int bad;
  long long start_pos;
  Span start;
};
static_assert(sizeof(Small) <= 3072, "small shared memory");

struct Maps {
  CUtensorMap q;
  CUtensorMap part[2];  // the parts of 8 keys of a page
  CUtensorMap page;     // a page, for prefetches
};

struct Shape {
  int ways, way;     // a request's row tiles are dealt to `ways` CTAs that read the same keys
  int groups, group; // stretches of the line
};

template <int N>
__device__ __forceinline__ int span_of(const LatentParams& p, const Shape& sh, int r, Span& s) {
  s.a = __ldg(p.qsl + r);
  const int b = __ldg(p.qsl + r + 1);
  s.S = __ldg(p.seq_lens + r);
  s.L = b - s.a;
  s.units = s.len = 0;
  if (s.L < 0 || s.a < 0 || b > p.num_tokens || (r == 0 && s.a != 0) ||
      (r == p.num_seqs - 1 && b != p.num_tokens))
    return PA_DEV_QSL;
  if (s.L < 1 || s.L > s.S || s.S > p.max_seq_len || s.L > p.max_query_len) return PA_DEV_LENGTHS;
  const int tiles = static_cast<int>((static_cast<long long>(s.L) * p.num_heads + N - 1) / N);
  s.units = (tiles + sh.ways - 1) / sh.ways;
  s.len = (s.S + kKeys - 1) / kKeys + kUnitCost;
  return 0;
}

// The stretch that position x of the line belongs to.
__device__ __forceinline__ int group_of(long long x, long long total, int groups) {
  return static_cast<int>(((x + 1) * groups - 1) / total);
}

}  // namespace

template <int R, int N>
__global__ void __launch_bounds__(kThreads, 1)
    latent_tc_kernel(const LatentParams p, const __grid_constant__ Maps maps, const int ways, const bool whole) {
  using C = Cfg<R, N>;
  extern __shared__ __align__(1024) unsigned char smem[];
  Small& sm = *reinterpret_cast<Small*>(smem + C::kSmallOff);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sm.abort;
  auto bar = [&](int i) { return smem_u32(&sm.bars[i]); };

  // ---- this CTA's place, and this thread's requests of the step
  Shape sh;
  sh.ways = ways;
  sh.way = blockIdx.x % ways;
  sh.group = blockIdx.x / ways;
  sh.groups = gridDim.x / ways;
  const int per = (p.num_seqs + kThreads - 1) / kThreads;
  const int ra = min(tid * per, p.num_seqs), rb = min(ra + per, p.num_seqs);

  if (tid == kCopyWarp * 32) {
    prefetch_map(&maps.q);
    prefetch_map(&maps.page);
    prefetch_map(&maps.part[0]);
    prefetch_map(&maps.part[1]);
  }
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t n = 1;
      if (i == kUnitEmpty || i == kUnitEmpty + 1) n = 11;
      if (i >= kPFull && i < kTrade) n = 8;
      if (i == kTrade || i == kTrade + 1) n = 4;
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
  Span s0{};
  int err = ra < rb ? span_of<N>(p, sh, ra, s0) : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  // ---- this CTA's stretch of the line: [lo, hi), beginning in request start_r
  long long lo = 0, hi = 0, total = 0;
  {
    long long mine = static_cast<long long>(s0.units) * s0.len;
#pragma unroll 1
    for (int r = ra + 1; r < rb; ++r) {
      Span s;
      err |= span_of<N>(p, sh, r, s);
      mine += static_cast<long long>(s.units) * s.len;
    }
    if (err) {
      if (blockIdx.x == 0) flag_error(p.status, err);
      if (err & PA_DEV_QSL) sm.bad = 1;
    }
    long long before = mine;  // inclusive scan over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    long long* sums = reinterpret_cast<long long*>(&sm.mx[0][0][0]);
    if (lane == 31) sums[warp] = before;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    before -= mine;
    if (sm.bad) total = 0;
    const long long most = total / kMinStretch;
    sh.groups = static_cast<int>(min(static_cast<long long>(sh.groups), most < 1 ? 1 : most));
    if (sh.group < sh.groups) {
      lo = total * sh.group / sh.groups;
      hi = total * (sh.group + 1) / sh.groups;
    }
    if (lo < hi && before <= lo && lo < before + mine) {
      long long pos = before;
      Span s = s0;
#pragma unroll 1
      for (int r = ra; r < rb; ++r) {
        if (r > ra) span_of<N>(p, sh, r, s);
        const long long len = static_cast<long long>(s.units) * s.len;
        if (lo < pos + len) {
          sm.start_r = r;
          sm.start_pos = pos;
          sm.start = s;
          break;
        }
        pos += len;
      }
    }
    __syncthreads();
  }

  // ---- what both copy warps do: part h of the tiles of a unit
  // table entries of the pages of 8 tiles, one a lane: of group i of unit u, -1 past the request's keys
  auto entries = [&](const Unit& u, int i) {
    const int b = i * 32 + lane;
    return b * kBlockSize < u.seq ? __ldg(p.block_tables + static_cast<long long>(u.r) * p.max_blocks_per_seq + b) : -1;
  };
  // tile t, the g-th of the CTA; now: the entries of its group
  auto copy_part = [&](const Unit& u, int h, int t, uint32_t g, int now) {
    const int b = g % C::kBufs, page = (lane & 7) >> 1;  // 8 lanes, one for every 8 keys
    int cur = __shfl_sync(0xffffffffu, now, (t & 7) * kPages + page);
    // a page past the keys or with a bad table entry is read out of bounds: zeros
    if (cur < 0 || cur >= p.num_blocks) {
      if (lane < 8 && (t * kPages + page) * kBlockSize < u.seq) flag_error(p.status, PA_DEV_BLOCK_RANGE);
      cur = p.num_blocks;
    }
    if (g >= C::kBufs && !wait_bar(bar(kKEmpty + 4 * h + b), (g / C::kBufs - 1) & 1, abort, p.status)) return false;
    if (lane == 0) mbar_arrive_expect_tx(bar(kKFull + 4 * h + b), C::part_bytes(h));
    __syncwarp();
    if (lane < 8)
      tma_load_5d(sbase + b * C::kTileBytes + lane * C::kGroupBytes + h * C::kHalf * 1024, &maps.part[h], 0, 0,
                  h * C::kHalf, lane & 1, cur, bar(kKFull + 4 * h + b));
    return true;
  };
  // (after a timeout: let every copy issued land before the CTA ends)
  auto drain_part = [&](int h, uint32_t g) {
    for (uint32_t i = g > C::kBufs ? g - C::kBufs : 0; i < g; ++i)
      drain_wait(bar(kKFull + 4 * h + i % C::kBufs), (i / C::kBufs) & 1);
  };

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------ units and copies
    if (lane < 2) p.recs[blockIdx.x * 2 + lane] = make_int4(0, 0, 0, 0);
    __syncwarp();
    int uc = 0;        // units published
    uint32_t g = 0;    // tiles copied
    bool ok = !*abort;
    auto publish = [&](const Unit& u) {
      const int slot = uc & 1;
      if (uc >= 2 && !wait_bar(bar(kUnitEmpty + slot), ((uc >> 1) - 1) & 1, abort, p.status)) return false;
      if (lane == 0) {
        sm.units[slot] = u;
        mbar_arrive(bar(kUnitFull + slot));
      }
      __syncwarp();
      return true;
    };
    auto run = [&](const Unit& u) {
      int now = entries(u, u.t0 / 8), then = entries(u, u.t0 / 8 + 1);
      if (!publish(u)) return false;
      const int qs = uc % C::kQs;
      if (uc >= C::kQs && !wait_bar(bar(kQEmpty + qs), (uc / C::kQs - 1) & 1, abort, p.status)) return false;
      if (lane == 0) mbar_arrive_expect_tx(bar(kQFull + qs), C::kQBytes);
      __syncwarp();
      if (lane < C::kSlices)
        tma_load_2d(sbase + C::kQOff + qs * C::kQBytes + lane * N * 128, &maps.q, lane * 64, u.row0,
                    bar(kQFull + qs));
      ++uc;
      // block of page `lane` (< 4) of tile t: `now`'s group or the next
      auto block_of = [&](int t, int group) {
        const int src = (t & 7) * kPages + (lane & (kPages - 1));
        const int a = __shfl_sync(0xffffffffu, now, src), b = __shfl_sync(0xffffffffu, then, src);
        return (t >> 3) == group ? a : b;
      };
      const int end = u.t0 + u.n;
      int fetched = u.t0 + 1;  // tiles before it are copied or on their way to L2
      for (int t = u.t0; t < end; ++t, ++g) {
        if ((t & 7) == 0 && t > u.t0) {
          now = then;
          then = entries(u, t / 8 + 1);
        }
        for (; fetched <= t + kAhead && fetched < end; ++fetched) {
          const int ph = block_of(fetched, t >> 3);
          if (lane < kPages && ph >= 0 && ph < p.num_blocks) tma_prefetch_5d(&maps.page, 0, 0, 0, 0, ph);
        }
        if (!copy_part(u, 0, t, g, now)) return false;
      }
      return true;
    };
    if (ok && sm.start_r >= 0) {
      long long pos = sm.start_pos;
      Span s = sm.start;
      for (int r = sm.start_r; ok && r < p.num_seqs && pos < hi; ++r) {
        if (r > sm.start_r) span_of<N>(p, sh, r, s);
        const long long skip = s.len && lo > pos ? (lo - pos) / s.len : 0;
        for (int j = static_cast<int>(skip); ok && j < s.units; ++j) {
          const long long ua = pos + static_cast<long long>(j) * s.len;
          if (ua >= hi) break;
          const long long m = static_cast<long long>(j) * sh.ways + sh.way;
          const long long first = m * N;
          const long long rows = static_cast<long long>(s.L) * p.num_heads - first;
          if (rows <= 0) continue;
          Unit u;
          u.r = r;
          u.rows = static_cast<int>(min(rows, static_cast<long long>(N)));
          u.first = static_cast<int>(first);
          u.row0 = static_cast<int>(static_cast<long long>(s.a) * p.num_heads + first);
          u.prior = s.S - s.L;
          u.seq = s.S;
          // tiles that some row of the unit sees
          const int seen = u.prior + (u.first + u.rows - 1) / p.num_heads + 1;
          const int nk = (seen + kKeys - 1) / kKeys;
          const long long f = ua + kUnitCost;  // the first tile's place
          u.t0 = static_cast<int>(max(0LL, lo - f));
          int t1 = static_cast<int>(min(static_cast<long long>(nk), hi - f));
          if (whole) {  // the CTA in whose stretch its middle lies takes it
            const long long middle = ua + s.len / 2;
            u.t0 = 0;
            t1 = middle >= lo && middle < hi ? nk : 0;
          }
          if (u.t0 >= t1) continue;
          u.n = t1 - u.t0;
          u.slot = u.n == nk ? -1 : static_cast<int>(blockIdx.x) * 2 + (u.t0 == 0);
          if (u.slot >= 0 && lane == 0) {
            const int first = group_of(f, total, sh.groups);
            p.recs[u.slot] = make_int4(u.row0, u.rows, sh.group - first, group_of(f + nk - 1, total, sh.groups) - first + 1);
          }
          ok = run(u);
        }
        pos += static_cast<long long>(s.units) * s.len;
      }
    }
    Unit end{};
    end.r = -1;
    if (ok) publish(end);
    if (*abort) {
      drain_part(0, g);
      for (int i = uc > C::kQs ? uc - C::kQs : 0; i < uc; ++i)
        drain_wait(bar(kQFull + i % C::kQs), (i / C::kQs) & 1);
    }
    __syncwarp();
  } else if (warp == kCopy2Warp) {
    // ------------------------------------------------------------ copies of the second parts
    uint32_t g = 0;
    bool ok = !*abort;
    for (int uc = 0; ok; ++uc) {
      if (!wait_bar(bar(kUnitFull + (uc & 1)), (uc >> 1) & 1, abort, p.status)) break;
      const Unit u = sm.units[uc & 1];
      warp_arrive(bar(kUnitEmpty + (uc & 1)));
      if (u.r < 0) break;
      int now = entries(u, u.t0 / 8), then = entries(u, u.t0 / 8 + 1);
      for (int t = u.t0; t < u.t0 + u.n; ++t, ++g) {
        if ((t & 7) == 0 && t > u.t0) {
          now = then;
          then = entries(u, t / 8 + 1);
        }
        ok = copy_part(u, 1, t, g, now);
        if (!ok) break;
      }
    }
    if (*abort) drain_part(1, g);
    __syncwarp();
  } else if (warp >= kSWarp) {
    // ------------------------------------------------------------ MMA issue, one thread each
    if (elect_one() && !*abort) {
      auto adv = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };
      auto wait = [&](int i, uint32_t parity) { return wait_one(bar(i), parity, abort, p.status); };
      const uint64_t dk = smem_desc_sw128(sbase, 16, C::kGroupBytes);
      const uint64_t dv = smem_desc_sw128(sbase, 1024, C::kGroupBytes);
      const uint64_t dq = smem_desc_sw128(sbase + C::kQOff, 16, 1024);
      uint32_t g = 0, b = 0, phase = 0;  // tiles, and the buffer and its round
      bool ok = true;
      for (int uc = 0; ok; ++uc) {
        const int slot = uc & 1;
        if (!wait(kUnitFull + slot, (uc >> 1) & 1)) break;
        const int n = sm.units[slot].r < 0 ? 0 : sm.units[slot].n;
        mbar_arrive(bar(kUnitEmpty + slot));
        if (n == 0) break;
        const int qs = uc % C::kQs;
        if (warp == kSWarp && !wait(kQFull + qs, (uc / C::kQs) & 1)) break;
        for (int t = 0; t < n; ++t, ++g) {
          if (warp == kSWarp) {
            // S of tile g - 2 is read (phase -1 of a barrier counts as complete)
            ok = wait_both(bar(kKFull + b), phase, bar(kPFull + (g - 2) % C::kPBars), ((g - 2) / C::kPBars) & 1, abort,
                           p.status);
            if (!ok) break;
            tc_fence_after();
            constexpr uint32_t kId = idesc_bf16(kKeys, N, 0);
            const uint64_t kb = adv(dk, b * C::kTileBytes), qb = adv(dq, qs * C::kQBytes);
            const uint32_t d = tmem + C::kTmemS + (g & 1) * N;
#pragma unroll
            for (int i = 0; i < C::kHalf * 4; ++i)
              tc_mma_f16(d, adv(kb, (i >> 2) * 1024 + (i & 3) * 32), adv(qb, (i >> 2) * (N * 128) + (i & 3) * 32),
                         kId, i > 0);
            ok = wait(kKFull + 4 + b, phase);
            if (!ok) break;
#pragma unroll
            for (int i = C::kHalf * 4; i < C::kSlices * 4; ++i)
              tc_mma_f16(d, adv(kb, (i >> 2) * 1024 + (i & 3) * 32), adv(qb, (i >> 2) * (N * 128) + (i & 3) * 32),
                         kId, 1);
            tc_commit(bar(kSFull + (g & 1)));
            if (t == n - 1) tc_commit(bar(kQEmpty + qs));
          } else {
            ok = wait(kPFull + b, phase);
            if (!ok) break;
            tc_fence_after();
            constexpr uint32_t kId = idesc_bf16(128, N, 0) | (1u << 15);  // A MN-major
            const uint64_t vb = adv(dv, b * C::kTileBytes), pb = adv(dk, b * C::kTileBytes + C::kPOff);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int m = h * C::kBlocks / 2; m < (h + 1) * C::kBlocks / 2; ++m)
#pragma unroll
                for (int pg = 0; pg < kPages; ++pg)
                  tc_mma_f16(tmem + m * N, adv(vb, pg * C::kPageBytes + m * 2048), adv(pb, pg * 32), kId,
                             t > 0 || pg > 0);
              tc_commit(bar(kKEmpty + 4 * h + b));
            }
          }
          if (++b == C::kBufs) b = 0, phase ^= 1;
        }
      }
    }
    __syncwarp();
    if (*abort) {  // nothing may still run on tensor memory when it is freed
      const int d = kDrain + (warp == kOWarp);
      if (elect_one()) tc_commit(bar(d));
      __syncwarp();
      drain_wait(bar(d), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax and output
    constexpr int H = N / 2, F = H / 8;  // columns of this half, column groups of a fragment
    constexpr int kStep = H < 16 ? H : 16;
    const int half = warp >> 2, quarter = warp & 3;
    const int c0 = half * H + 2 * (lane & 3);  // this lane's first column
    const int key0 = quarter * 16 + (lane >> 2);
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t g = 0;
    bool ok = !*abort;
    // phase of tile i's "O += done"
    auto wait_o = [&](uint32_t i) {
      return wait_bar(bar(kKEmpty + 4 + i % C::kBufs), (i / C::kBufs) & 1, abort, p.status);
    };
    uint32_t trades = 0;
    auto meet = [&]() {
      warp_arrive(bar(kTrade + half));
      return wait_bar(bar(kTrade + half), trades++ & 1, abort, p.status);
    };
    for (int uc = 0; ok; ++uc) {
      if (!wait_bar(bar(kUnitFull + (uc & 1)), (uc >> 1) & 1, abort, p.status)) break;
      const Unit u = sm.units[uc & 1];
      warp_arrive(bar(kUnitEmpty + (uc & 1)));
      if (u.r < 0) break;
      float m[F][2], l[F][2];  // reference and this lane's part of the sum, by column
#pragma unroll
      for (int i = 0; i < F; ++i) m[i][0] = m[i][1] = -CUDART_INF_F, l[i][0] = l[i][1] = 0.f;
      // keys up to here are seen by every row
      const int low = u.prior + u.first / p.num_heads;
      for (int t = 0; t < u.n; ++t, ++g) {
        const int k0 = (u.t0 + t) * kKeys;
        if (!wait_bar(bar(kSFull + (g & 1)), (g >> 1) & 1, abort, p.status)) { ok = false; break; }
        tc_fence_after();
        uint32_t raw[F * 4];
        tmem_ld_frag(tmem + C::kTmemS + (g & 1) * N + half * H + lanes, raw);
        tmem_wait_ld();
        float x[F][4];
#pragma unroll
        for (int i = 0; i < F * 4; ++i) x[i >> 2][i & 3] = __uint_as_float(raw[i]) * p.scale_log2;
        if (k0 + kKeys - 1 > low) {
          const int a = k0 + key0;
#pragma unroll
          for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int last = u.prior + (u.first + 8 * i + c0 + j) / p.num_heads;
              if (a > last) x[i][j] = -CUDART_INF_F;
              if (a + 8 > last) x[i][j + 2] = -CUDART_INF_F;
            }
          // slots behind the last key hold anything: zeros, so that a weight of zero meets no NaN
          const int end = u.seq - k0;  // rows of the tile that hold keys
          if (end < kKeys && (end & (kBlockSize - 1))) {
            const uint32_t page = sbase + (g % C::kBufs) * C::kTileBytes + (end / kBlockSize) * C::kPageBytes;
            const int r0 = end & (kBlockSize - 1);
            constexpr int kPer = R / 8;
            for (int i = tid; i < (kBlockSize - r0) * kPer; i += kSoftThreads) {
              const int row = r0 + i / kPer, c = i % kPer;
              asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(
                               page + (row >> 3) * C::kGroupBytes + (c >> 3) * 1024 + (row & 7) * 128 + (c & 7) * 16),
                           "r"(0u)
                           : "memory");
            }
          }
        }
        // column maxima over the warp's 16 keys: the 8 lanes that share the columns halve them among
        // themselves, so each ends with one column's; then over the four warps
        float v[2 * F];
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) v[2 * i + j] = fmaxf(x[i][j], x[i][j + 2]);
        int own = 0;  // index of this lane's column among its 2 F
#pragma unroll
        for (int n = 2 * F, o = 16; o >= 4; o >>= 1) {
          if (n > 1) {
            n /= 2;
            const bool up = (lane & o) != 0;
            if (up) own += n;
#pragma unroll
            for (int k = 0; k < n; ++k) {
              const float send = up ? v[k] : v[k + n];
              v[k] = fmaxf(up ? v[k + n] : v[k], __shfl_xor_sync(0xffffffffu, send, o));
            }
          } else {
            v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
          }
        }
        const int col = c0 + 8 * (own >> 1) + (own & 1);
        sm.mx[g & 1][quarter][col] = v[0];  // (lanes that hold the same column write the same)
        if (!meet()) { ok = false; break; }
        v[0] = fmaxf(fmaxf(sm.mx[g & 1][0][col], sm.mx[g & 1][1][col]), fmaxf(sm.mx[g & 1][2][col], sm.mx[g & 1][3][col]));
        // ... and back to all of them
#pragma unroll
        for (int n = 1, o = 64 / (2 * F) / 2 > 16 ? 16 : 64 / (2 * F) / 2; n < 2 * F; n *= 2, o <<= 1) {
          const bool up = (lane & o) != 0;
#pragma unroll
          for (int k = n - 1; k >= 0; --k) {
            const float other = __shfl_xor_sync(0xffffffffu, v[k], o);
            const float mine = v[k];
            v[k] = up ? other : mine;
            v[k + n] = up ? mine : other;
          }
        }
        bool moved = false;
#pragma unroll
        for (int i = 0; i < F; ++i) moved |= v[2 * i] > m[i][0] + kGrowth || v[2 * i + 1] > m[i][1] + kGrowth;
        moved = __any_sync(0xffffffffu, moved);
        float f[F][2];
        if (moved) {
#pragma unroll
          for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const bool up = v[2 * i + j] > m[i][j] + kGrowth;  // (also the first finite maximum: m = -inf)
              f[i][j] = up ? ex2(m[i][j] - v[2 * i + j]) : 1.f;
              if (up) m[i][j] = v[2 * i + j];
              l[i][j] *= f[i][j];
            }
        }
        // P and this lane's sums
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (no key seen yet: every logit is -inf, every weight 0)
            const float ref = m[i][j & 1] == -CUDART_INF_F ? 0.f : m[i][j & 1];
            x[i][j] = ex2(x[i][j] - ref);
            l[i][j & 1] += x[i][j];
          }
        // O' of earlier tiles takes the new references, once it is there
        if (moved && t > 0) {
          if (quarter == 0 && lane < 4) {
#pragma unroll
            for (int i = 0; i < F; ++i)
              *reinterpret_cast<float2*>(&sm.f[8 * i + c0]) = make_float2(f[i][0], f[i][1]);
          }
          if (!meet() || !wait_o(g - 1)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < C::kBlocks * H; c += kStep) {
            const uint32_t at = tmem + lanes + c / H * N + half * H + c % H;
            uint32_t o[kStep];
            tmem_ld(at, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < kStep; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sm.f[half * H + c % H + i]);
            tmem_st(at, o);
          }
          tmem_wait_st();
        }
        // P, where the key part was (S has read it)
        const uint32_t pbuf = sbase + (g % C::kBufs) * C::kTileBytes + C::kPOff;
        // (a matrix of 8 keys x 8 rows a register; lanes 8 k .. 8 k + 7 address matrix k's rows)
        if constexpr (F == 1) {
          const int row = half * H + (lane & 7), chunk = 2 * quarter + ((lane >> 3) & 1);
          asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1,%2};\n" ::"r"(
                           pbuf + (row >> 3) * C::kGroupBytes + (row & 7) * 128 + ((chunk ^ (row & 7)) << 4)),
                       "r"(pack_bf16(x[0][0], x[0][1])), "r"(pack_bf16(x[0][2], x[0][3]))
                       : "memory");
        } else {
#pragma unroll
          for (int i = 0; i < F; i += 2) {
            const int row = half * H + 8 * (i + (lane >> 4)) + (lane & 7), chunk = 2 * quarter + ((lane >> 3) & 1);
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(
                             pbuf + (row >> 3) * C::kGroupBytes + (row & 7) * 128 + ((chunk ^ (row & 7)) << 4)),
                         "r"(pack_bf16(x[i][0], x[i][1])), "r"(pack_bf16(x[i][2], x[i][3])),
                         "r"(pack_bf16(x[i + 1][0], x[i + 1][1])), "r"(pack_bf16(x[i + 1][2], x[i + 1][3]))
                         : "memory");
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(bar(kPFull + g % C::kPBars));
      }
      if (!ok) break;

      // ---- the unit's output: O' / sum, or its partial state
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[i][j] += __shfl_xor_sync(0xffffffffu, l[i][j], o);
      if (!meet()) break;  // the last tile's maxima are read
      if (lane < 4) {
#pragma unroll
        for (int i = 0; i < F; ++i)
          *reinterpret_cast<float2*>(&sm.mx[0][quarter][8 * i + c0]) = make_float2(l[i][0], l[i][1]);
        if (quarter == 0 && u.slot >= 0) {
#pragma unroll
          for (int i = 0; i < F; ++i)
            *reinterpret_cast<float2*>(&sm.mx[1][0][8 * i + c0]) = make_float2(m[i][0], m[i][1]);
        }
      }
      if (!meet()) break;
      if ((tid & 127) < H) {
        const int n = half * H + (tid & 127);
        const float sum = sm.mx[0][0][n] + sm.mx[0][1][n] + sm.mx[0][2][n] + sm.mx[0][3][n];
        sm.f[n] = u.slot >= 0 ? 1.f : 1.f / sum;
        if (u.slot >= 0)
          reinterpret_cast<float2*>(p.part_ml)[static_cast<long long>(u.slot) * N + n] = make_float2(sm.mx[1][0][n], sum);
      }
      if (!meet() || !wait_o(g - 1)) break;
      tc_fence_after();
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + static_cast<long long>(u.row0) * R;
      float* part = p.part_acc + static_cast<long long>(u.slot) * N * R;
      // (the next columns are on their way while these are written)
      uint32_t next[kStep];
      tmem_ld(tmem + lanes + half * H, next);
#pragma unroll 1
      for (int c = 0; c < C::kBlocks * H; c += kStep) {
        uint32_t o[kStep];
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < kStep; ++i) o[i] = next[i];
        const int c1 = c + kStep;
        if (c1 < C::kBlocks * H) tmem_ld(tmem + lanes + c1 / H * N + half * H + c1 % H, next);
        const int n0 = half * H + c % H;                    // rows n0 .. n0 + kStep - 1
        const int d = c / H * 128 + quarter * 32 + lane;    // this lane's number
        if (u.slot >= 0) {
#pragma unroll
          for (int i = 0; i < kStep; ++i)
            if (n0 + i < u.rows) part[(n0 + i) * R + d] = __uint_as_float(o[i]);
        } else {
          // lanes of a pair trade: the even one writes both numbers of row i, the odd one of row i + 1
#pragma unroll
          for (int i = 0; i < kStep; i += 2) {
            const float a = __uint_as_float(o[i]) * sm.f[n0 + i], b = __uint_as_float(o[i + 1]) * sm.f[n0 + i + 1];
            const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? a : b, 1);
            const int row = n0 + i + (lane & 1);
            const uint32_t w = (lane & 1) ? pack_bf16(other, b) : pack_bf16(a, other);
            if (row < u.rows) *reinterpret_cast<uint32_t*>(out + row * R + (d & ~1)) = w;
          }
        }
      }
      tc_fence_before();
      if (!meet()) break;  // the shared factors are read
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins the pieces of units that a border cut, in the order of their keys.  Every piece has left a record
// {first row, rows, piece, pieces}, and has 8 CTAs.  Of up to 8 pieces those of the first one join, a warp a row
// (64 rows at most); of more, all pieces' CTAs, each a row in turn and a warp of it every eighth piece.
// 16 float4 a lane are loaded at once, as the time is that of a few loads that wait for one another.
template <int R, int N>
__global__ void __launch_bounds__(256) latent_join_kernel(const LatentParams p, int ways) {
  constexpr int kVec = R / 128;  // float4 of a lane
  constexpr int kAtOnce = 16 / kVec, kFew = 8;
  __shared__ float4 acc_s[8][R / 4];
  __shared__ float2 ml_s[8];
  wait_prior_grid();
  launch_dependents();  // a following kernel may set up; it waits for this grid
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 recs[2] = {p.recs[blockIdx.x * 2], p.recs[blockIdx.x * 2 + 1]};
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int4 rec = which ? recs[1] : recs[0];
    const int rows = rec.y, piece = rec.z, pieces = rec.w;
    if (pieces == 0) continue;
    const int first = blockIdx.x - piece * ways;  // CTA of the first piece
    const bool few = pieces <= kFew;
    const int k0 = few ? 0 : warp, dk = few ? 1 : 8;
    const int n = few ? (piece * 8 + blockIdx.y) * 8 + warp : piece * 8 + blockIdx.y;
    if (n >= rows) continue;  // (a whole CTA where its warps share a row; 8 pieces are CTAs enough for 64)
    float m = -CUDART_INF_F, l = 0.f;
    float4 acc[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 ml, const float4 (&x)[kVec]) {
      if (ml.y == 0.f) return;  // a piece whose keys the row does not see
      const float nm = fmaxf(m, ml.x);
      const float fa = m == nm ? 1.f : ex2(m - nm), fb = ml.x == nm ? 1.f : ex2(ml.x - nm);
      m = nm;
      l = l * fa + ml.y * fb;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        acc[i].x = acc[i].x * fa + x[i].x * fb;
        acc[i].y = acc[i].y * fa + x[i].y * fb;
        acc[i].z = acc[i].z * fa + x[i].z * fb;
        acc[i].w = acc[i].w * fa + x[i].w * fb;
      }
    };
    for (int k = k0; k < pieces; k += kAtOnce * dk) {
      float2 ml[kAtOnce];
      float4 x[kAtOnce][kVec];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = k + j * dk;
        ml[j].y = 0.f;
        if (i < pieces) {  // piece i: the first CTA's slot 1, then slot 0 of the following ones
          const long long row = (static_cast<long long>(first + i * ways) * 2 + (i == 0)) * N + n;
          ml[j] = reinterpret_cast<const float2*>(p.part_ml)[row];
          const float4* src = reinterpret_cast<const float4*>(p.part_acc + row * R);
#pragma unroll
          for (int c = 0; c < kVec; ++c) x[j][c] = src[c * 32 + lane];
        }
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) add(ml[j], x[j]);
    }
    if (!few) {
      __syncthreads();  // (the row before is read)
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc_s[warp][i * 32 + lane] = acc[i];
      if (lane == 0) ml_s[warp] = make_float2(m, l);
      __syncthreads();
      if (warp != 0) continue;
      for (int w = 1; w < 8; ++w) {
        float4 x[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = acc_s[w][i * 32 + lane];
        add(ml_s[w], x);
      }
    }
    const float inv = 1.f / l;
    uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + static_cast<long long>(rec.x + n) * R);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      out[i * 32 + lane] = make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
  }
}

namespace {

template <int R, int N>
cudaError_t launch_latent(const LatentParams& p, int num_sms, cudaStream_t stream) {
  using C = Cfg<R, N>;
  constexpr int W = R + kLatentRope;
  static bool configured[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(latent_tc_kernel<R, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  Maps maps;
  {
    const cuuint64_t dims[2] = {W, static_cast<cuuint64_t>(p.num_tokens) * p.num_heads};
    const cuuint64_t strides[1] = {W * 2};
    const cuuint32_t box[2] = {64, N};
    if (!encode_bf16(&maps.q, p.q, 2, dims, strides, box)) return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[5] = {64, 8, C::kSlices, 2, static_cast<cuuint64_t>(p.num_blocks)};
    const cuuint64_t strides[4] = {W * 2, 128, 8 * W * 2, kBlockSize * W * 2};
    const cuuint32_t page[5] = {64, 8, C::kSlices, 2, 1};
    const cuuint32_t part0[5] = {64, 8, C::kHalf, 1, 1}, part1[5] = {64, 8, C::kHalf + 1, 1, 1};
    if (!encode_bf16(&maps.page, p.cache, 5, dims, strides, page) ||
        !encode_bf16(&maps.part[0], p.cache, 5, dims, strides, part0) ||
        !encode_bf16(&maps.part[1], p.cache, 5, dims, strides, part1))
      return cudaErrorInvalidValue;
  }
  // decodes of more heads than a unit's rows: CTAs side by side take the row tiles of
  // the same keys, so that all but the first read them from L2
  int ways = p.max_query_len == 1 ? (p.num_heads + N - 1) / N : 1;
  // no more CTAs than the step can have stretches
  const long long tiles = (static_cast<long long>(p.num_heads) * p.max_query_len + N - 1) / N;
  const long long line = p.num_seqs * ((tiles + ways - 1) / ways) * ((p.max_seq_len + kKeys - 1) / kKeys + kUnitCost);
  const int most = (num_sms < kLatentMaxCtas ? num_sms : kLatentMaxCtas) / ways;
  const int ctas = static_cast<int>(line / kMinStretch < most ? line / kMinStretch : most) * ways;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool whole = p.max_seq_len <= kWholeTiles * kKeys;
  e = cudaLaunchKernelEx(&cfg, latent_tc_kernel<R, N>, p, maps, ways, whole);
  if (e != cudaSuccess || whole) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, latent_join_kernel<R, N>, p, ways);
}

}  // namespace

// Query rows of a unit: the smallest tile that holds a request's rows.
static int unit_rows(int num_heads, int max_query_len) {
  const long long rows = static_cast<long long>(num_heads) * max_query_len;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

size_t latent_tc_partial_rows(int num_heads, int max_query_len) {
  return static_cast<size_t>(2) * kLatentMaxCtas * unit_rows(num_heads, max_query_len);
}

cudaError_t launch_latent_tc(const LatentParams& p, int latent_size, int num_sms, cudaStream_t stream) {
  const int n = unit_rows(p.num_heads, p.max_query_len);
  if (latent_size == 512)
    return n == 16 ? launch_latent<512, 16>(p, num_sms, stream)
         : n == 32 ? launch_latent<512, 32>(p, num_sms, stream)
                   : launch_latent<512, 64>(p, num_sms, stream);
  return n == 16 ? launch_latent<256, 16>(p, num_sms, stream)
       : n == 32 ? launch_latent<256, 32>(p, num_sms, stream)
                 : launch_latent<256, 64>(p, num_sms, stream);
}

}  // namespace pa
