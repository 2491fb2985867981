// Host side of the latent-attention calls: argument checks and launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "pa_latent.h"

namespace pa {
namespace {

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_last_error(code, buf);
}

int done(cudaError_t e, const char* what) {
  return e == cudaSuccess ? static_cast<int>(PA_OK)
                          : fail(PA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
long long cdiv(long long a, long long b) { return (a + b - 1) / b; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int elem_bytes(pa_dtype t) { return t == PA_BF16 ? 2 : 4; }

int check_common(pa_dtype dtype, int num_heads, int rope_size) {
  if (dtype != PA_F32 && dtype != PA_BF16)
    return fail(PA_ERR_INVALID, "dtype %d is not PA_F32 or PA_BF16", static_cast<int>(dtype));
  if (num_heads < 1) return fail(PA_ERR_INVALID, "num_heads %d < 1", num_heads);
  if (num_heads > kLatentMaxHeads)
    return fail(PA_ERR_UNSUPPORTED, "num_heads %d (built for up to %d)", num_heads, kLatentMaxHeads);
  if (rope_size != kLatentRope)
    return fail(PA_ERR_UNSUPPORTED, "rope_size %d (built for %d)", rope_size, kLatentRope);
  return PA_OK;
}

int check_latent(const pa_latent_layout* L) {
  if (!L) return fail(PA_ERR_INVALID, "layout is NULL");
  if (int rc = check_common(L->dtype, L->num_heads, L->rope_size)) return rc;
  if (L->latent_size != 256 && L->latent_size != 512)
    return fail(PA_ERR_UNSUPPORTED, "latent_size %d (built for 256 and 512)", L->latent_size);
  if (L->block_size != kBlockSize)
    return fail(PA_ERR_UNSUPPORTED, "block_size %d (built for 16)", L->block_size);
  if (L->num_blocks < 1) return fail(PA_ERR_INVALID, "num_blocks %d < 1", L->num_blocks);
  return PA_OK;
}

// fp32: pieces of a request's keys, so that few rows fill the GPU: as many as bring the CTAs to kCcCtas, of
// 16 blocks at least.
constexpr int kCcCtas = 4 * 152;
long long cc_most_splits(int max_seq_len) { return cdiv(max_seq_len, 16 * kBlockSize); }
int cc_splits(const pa_latent_layout* L, int num_tokens, int max_seq_len) {
  const long long rows = static_cast<long long>(num_tokens) * cdiv(L->num_heads, 8);
  const long long s = rows > 0 ? cdiv(kCcCtas, rows) : 1, most = cc_most_splits(max_seq_len);
  return static_cast<int>(s > most ? (most < 1 ? 1 : most) : s);
}
// Rows of partial states that a step of up to num_tokens tokens may leave: fewer tokens are cut into more
// pieces, so this is a bound over all of them.  With A = ceil(kCcCtas / groups of heads), t tokens are cut where
// t < A, into min(ceil(A / t), most) pieces, and t ceil(A / t) <= A + t - 1.
size_t cc_partial_rows(const pa_latent_layout* L, int num_tokens, int max_seq_len) {
  const long long most = cc_most_splits(max_seq_len), a = cdiv(kCcCtas, cdiv(L->num_heads, 8));
  const long long t = num_tokens < a ? num_tokens : a - 1;
  if (most <= 1 || t < 1) return 0;
  const long long pieces = t * most < a + t - 1 ? t * most : a + t - 1;
  return static_cast<size_t>(pieces) * L->num_heads;
}

struct LatentWs {
  size_t acc, ml, recs, total;
};
LatentWs latent_ws(const pa_latent_layout* L, int num_tokens, int max_query_len, int max_seq_len) {
  LatentWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off = align256(off + bytes); return o; };
  const size_t rows = L->dtype == PA_F32 ? cc_partial_rows(L, num_tokens, max_seq_len)
                                         : latent_tc_partial_rows(L->num_heads, max_query_len);
  w.acc = take(rows * L->latent_size * sizeof(float));
  w.ml = take(rows * 2 * sizeof(float));
  w.recs = take(2 * kLatentMaxCtas * sizeof(int4));
  w.total = off;
  return w;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_latent_write(const void* c, int64_t c_stride, const void* k_rope, int64_t k_stride,
                    const void* norm_weight, float eps, const void* q, int64_t q_stride,
                    int64_t q_head_stride, const pa_rope* rope, const int64_t* slot_mapping,
                    int num_tokens, void* q_out, int64_t qo_stride, int64_t qo_head_stride,
                    void* cache, const pa_latent_layout* layout, int32_t* status, void* stream) {
  set_last_error(PA_OK, "");
  if (int rc = check_latent(layout)) return rc;
  if (num_tokens < 0) return fail(PA_ERR_INVALID, "num_tokens %d < 0", num_tokens);
  if (num_tokens == 0) return PA_OK;
  if (int rc = check_rope(rope)) return rc;
  if (rope->rope_size != layout->rope_size)
    return fail(PA_ERR_INVALID, "rope's rope_size %d is not the layout's %d", rope->rope_size, layout->rope_size);
  if (!c || !k_rope || !slot_mapping || !cache) return fail(PA_ERR_INVALID, "null tensor pointer");
  if (!q != !q_out) return fail(PA_ERR_INVALID, "q and q_out must both be given, or neither");
  if (!aligned(c, 16) || !aligned(k_rope, 16) || !aligned(cache, 16) || !aligned(norm_weight, 16) ||
      !aligned(q, 16) || !aligned(q_out, 16))
    return fail(PA_ERR_INVALID, "c, k_rope, norm_weight, q, q_out and cache must be 16-byte aligned");
  if (!aligned(slot_mapping, 8)) return fail(PA_ERR_INVALID, "slot_mapping must be 8-byte aligned");
  if (status && !aligned(status, 4)) return fail(PA_ERR_INVALID, "status must be 4-byte aligned");
  if (norm_weight && !(std::isfinite(eps) && eps >= 0.f))
    return fail(PA_ERR_INVALID, "eps must be finite and not negative");
  const int64_t unit = 16 / elem_bytes(layout->dtype);
  if (c_stride % unit || k_stride % unit ||
      (q && (q_stride % unit || q_head_stride % unit || qo_stride % unit || qo_head_stride % unit)))
    return fail(PA_ERR_INVALID, "strides must be multiples of 16 bytes");
  if (c_stride < layout->latent_size || k_stride < layout->rope_size)
    return fail(PA_ERR_INVALID, "a token stride is smaller than the token's row");
  if (q && (q_head_stride < layout->rope_size || qo_head_stride < layout->rope_size ||
            q_stride < q_head_stride * (layout->num_heads - 1) + layout->rope_size ||
            qo_stride < qo_head_stride * (layout->num_heads - 1) + layout->rope_size))
    return fail(PA_ERR_INVALID, "q or q_out: a head or token stride is smaller than what it steps over");
  if (q && q == q_out && (q_stride != qo_stride || q_head_stride != qo_head_stride))
    return fail(PA_ERR_INVALID, "q_out may be q only with the same strides");
  if (num_tokens * (1LL + (q ? layout->num_heads : 0)) > 0x7fffffffLL)
    return fail(PA_ERR_INVALID, "too many rows for one call");
  const LatentWriteArgs a{c, k_rope, c_stride, k_stride, norm_weight, eps, q, q_stride, q_head_stride,
                          rope, slot_mapping, num_tokens, q_out, qo_stride, qo_head_stride, cache, status};
  return done(launch_latent_write(a, *layout, static_cast<cudaStream_t>(stream)), "latent write launch");
}

int pa_latent_read(const void* cache, const int64_t* slot_mapping, int num_tokens, void* c,
                   void* k_rope, const pa_latent_layout* layout, int32_t* status, void* stream) {
  set_last_error(PA_OK, "");
  if (int rc = check_latent(layout)) return rc;
  if (num_tokens < 0) return fail(PA_ERR_INVALID, "num_tokens %d < 0", num_tokens);
  if (num_tokens == 0) return PA_OK;
  if (!c || !k_rope || !slot_mapping || !cache) return fail(PA_ERR_INVALID, "null tensor pointer");
  if (!aligned(c, 16) || !aligned(k_rope, 16) || !aligned(cache, 16))
    return fail(PA_ERR_INVALID, "c, k_rope and cache must be 16-byte aligned");
  if (!aligned(slot_mapping, 8)) return fail(PA_ERR_INVALID, "slot_mapping must be 8-byte aligned");
  if (status && !aligned(status, 4)) return fail(PA_ERR_INVALID, "status must be 4-byte aligned");
  return done(launch_latent_read(cache, slot_mapping, num_tokens, c, k_rope, *layout, status,
                                 static_cast<cudaStream_t>(stream)),
              "latent read launch");
}

size_t pa_latent_workspace_size(const pa_latent_layout* layout, int num_seqs, int num_tokens,
                                int max_query_len, int max_seq_len) {
  set_last_error(PA_OK, "");
  if (check_latent(layout)) return 0;
  if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || max_seq_len < 0) {
    fail(PA_ERR_INVALID, "negative size");
    return 0;
  }
  return latent_ws(layout, num_tokens, max_query_len, max_seq_len).total;
}

int pa_latent_forward(const void* q, const void* cache, const int32_t* block_tables,
                      int max_blocks_per_seq, const int32_t* seq_lens,
                      const int32_t* query_start_loc, int num_seqs, int num_tokens,
                      int max_query_len, int max_seq_len, float scale, void* out, void* workspace,
                      size_t workspace_bytes, const pa_latent_layout* layout, int32_t* status,
                      void* stream) {
  set_last_error(PA_OK, "");
  if (int rc = check_latent(layout)) return rc;
  if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || max_seq_len < 0 || max_blocks_per_seq < 0)
    return fail(PA_ERR_INVALID, "negative size argument");
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  if (!q || !cache || !block_tables || !seq_lens || !query_start_loc || !out || !workspace)
    return fail(PA_ERR_INVALID, "null pointer argument");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache, 16))
    return fail(PA_ERR_INVALID, "q, out and cache must be 16-byte aligned");
  if (!aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4))
    return fail(PA_ERR_INVALID, "int32 arrays must be 4-byte aligned");
  if (!aligned(workspace, 256)) return fail(PA_ERR_INVALID, "workspace must be 256-byte aligned");
  if (status && !aligned(status, 4)) return fail(PA_ERR_INVALID, "status must be 4-byte aligned");
  if (!std::isfinite(scale)) return fail(PA_ERR_INVALID, "scale is not finite");
  if (max_query_len < 1 || max_seq_len < 1)
    return fail(PA_ERR_INVALID, "max_query_len and max_seq_len must be >= 1");
  if (cdiv(max_seq_len, kBlockSize) > max_blocks_per_seq)
    return fail(PA_ERR_INVALID, "max_blocks_per_seq %d < ceil(max_seq_len / 16) = %lld",
                max_blocks_per_seq, cdiv(max_seq_len, kBlockSize));
  if (num_tokens < num_seqs)
    return fail(PA_ERR_INVALID, "num_tokens %d < num_seqs %d: every request needs a new token",
                num_tokens, num_seqs);
  if (static_cast<long long>(num_tokens) * layout->num_heads > 0x7fffffffLL)
    return fail(PA_ERR_INVALID, "step too large for one call");
  const LatentWs w = latent_ws(layout, num_tokens, max_query_len, max_seq_len);
  if (workspace_bytes < w.total)
    return fail(PA_ERR_INVALID, "workspace of %zu bytes < %zu needed", workspace_bytes, w.total);
  int num_sms = 0;
  if (int rc = sms_of_current_device(&num_sms)) return rc;
  char* ws = static_cast<char*>(workspace);
  LatentParams p{};
  p.q = q;
  p.cache = cache;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.out = out;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.max_query_len = max_query_len;
  p.max_seq_len = max_seq_len;
  p.num_heads = layout->num_heads;
  p.num_blocks = layout->num_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.part_acc = reinterpret_cast<float*>(ws + w.acc);
  p.part_ml = reinterpret_cast<float*>(ws + w.ml);
  p.recs = reinterpret_cast<int4*>(ws + w.recs);
  p.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (layout->dtype == PA_F32) {
    p.splits = cc_splits(layout, num_tokens, max_seq_len);
    return done(launch_latent_cc(p, layout->latent_size, st), "latent attention launch");
  }
  return done(launch_latent_tc(p, layout->latent_size, num_sms, st), "latent attention launch");
}

// Regions of pa_expanded_forward's workspace.
static LatentWs expanded_ws(const pa_expanded_layout* L, int num_tokens, int max_kv_len) {
  LatentWs w{};
  const size_t rows = L->dtype == PA_BF16 ? expanded_tc_partial_rows(L->num_heads, num_tokens, max_kv_len) : 0;
  if (rows == 0) return w;
  w.ml = align256(rows * L->head_size * sizeof(float));
  w.recs = align256(w.ml + rows * 2 * sizeof(float));
  w.total = align256(w.recs + 2 * kLatentMaxCtas * sizeof(int4));
  return w;
}

static int check_expanded(const pa_expanded_layout* L) {
  if (!L) return fail(PA_ERR_INVALID, "layout is NULL");
  if (int rc = check_common(L->dtype, L->num_heads, L->rope_size)) return rc;
  if (L->head_size != 64 && L->head_size != 128)
    return fail(PA_ERR_UNSUPPORTED, "head_size %d (built for 64 and 128)", L->head_size);
  return PA_OK;
}

size_t pa_expanded_workspace_size(const pa_expanded_layout* layout, int num_tokens, int max_kv_len) {
  set_last_error(PA_OK, "");
  if (check_expanded(layout)) return 0;
  if (num_tokens < 0 || max_kv_len < 0) {
    fail(PA_ERR_INVALID, "negative size");
    return 0;
  }
  return expanded_ws(layout, num_tokens, max_kv_len).total;
}

int pa_expanded_forward(const void* q, const void* k_nope, const void* k_rope, const void* v,
                        const int32_t* query_start_loc, const int32_t* kv_start_loc, int num_seqs,
                        int num_tokens, int num_kv_tokens, int max_query_len, int max_kv_len,
                        float scale, void* out, void* workspace, size_t workspace_bytes,
                        const pa_expanded_layout* L, int32_t* status, void* stream) {
  set_last_error(PA_OK, "");
  if (int rc = check_expanded(L)) return rc;
  if (num_seqs < 0 || num_tokens < 0 || num_kv_tokens < 0 || max_query_len < 0 || max_kv_len < 0)
    return fail(PA_ERR_INVALID, "negative size argument");
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  if (!q || !k_nope || !k_rope || !v || !query_start_loc || !kv_start_loc || !out)
    return fail(PA_ERR_INVALID, "null pointer argument");
  if (!aligned(q, 16) || !aligned(k_nope, 16) || !aligned(k_rope, 16) || !aligned(v, 16) || !aligned(out, 16))
    return fail(PA_ERR_INVALID, "q, k_nope, k_rope, v and out must be 16-byte aligned");
  if (!aligned(query_start_loc, 4) || !aligned(kv_start_loc, 4))
    return fail(PA_ERR_INVALID, "int32 arrays must be 4-byte aligned");
  if (status && !aligned(status, 4)) return fail(PA_ERR_INVALID, "status must be 4-byte aligned");
  if (!std::isfinite(scale)) return fail(PA_ERR_INVALID, "scale is not finite");
  if (max_query_len < 1 || max_kv_len < 1)
    return fail(PA_ERR_INVALID, "max_query_len and max_kv_len must be >= 1");
  if (num_tokens < num_seqs || num_kv_tokens < num_tokens)
    return fail(PA_ERR_INVALID, "%d requests need as many new tokens (%d) and those keys (%d)", num_seqs,
                num_tokens, num_kv_tokens);
  const int64_t unit = 16 / elem_bytes(L->dtype);
  const int64_t strides[7] = {L->q_stride, L->q_head_stride, L->k_stride, L->k_head_stride,
                              L->kr_stride, L->v_stride, L->v_head_stride};
  for (int64_t s : strides)
    if (s <= 0 || s % unit || s * elem_bytes(L->dtype) >= (1LL << 40))
      return fail(PA_ERR_INVALID, "strides must be positive multiples of 16 bytes below 2^40");
  if (static_cast<long long>(num_tokens) * L->num_heads > 0x7fffffffLL)
    return fail(PA_ERR_INVALID, "step too large for one call");
  if (workspace && !aligned(workspace, 256)) return fail(PA_ERR_INVALID, "workspace must be 256-byte aligned");
  const LatentWs w = expanded_ws(L, num_tokens, max_kv_len);
  if (workspace_bytes == 0) workspace = nullptr;  // (sized for a larger step, whose units are not cut)
  if (workspace && workspace_bytes < w.total)
    return fail(PA_ERR_INVALID, "workspace of %zu bytes < %zu needed", workspace_bytes, w.total);
  int num_sms = 0;
  if (int rc = sms_of_current_device(&num_sms)) return rc;
  ExpandedParams p{q, k_nope, k_rope, v, query_start_loc, kv_start_loc, out, num_seqs, num_tokens,
                         num_kv_tokens, max_query_len, max_kv_len, L->num_heads, L->q_stride, L->q_head_stride,
                         L->k_stride, L->k_head_stride, L->kr_stride, L->v_stride, L->v_head_stride,
                         scale * 1.4426950408889634f, status, nullptr, nullptr, nullptr};
  if (workspace && w.total) {
    char* ws = static_cast<char*>(workspace);
    p.part_acc = reinterpret_cast<float4*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    p.recs = reinterpret_cast<int4*>(ws + w.recs);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return done(L->dtype == PA_F32 ? launch_expanded_cc(p, L->head_size, st)
                                 : launch_expanded_tc(p, L->head_size, num_sms, st),
              "expanded attention launch");
}

}  // extern "C"
