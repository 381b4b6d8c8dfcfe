// C entries of the paged-cache operators: validation, workspace layout and
// launches. Declarations and contracts: include/sva.h.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "host.h"
#include "paged.h"

namespace sva {
namespace {

constexpr long long kInt = 1ll << 31;

size_t elt_bytes(const sv_shape* s) { return s->dtype == SV_BF16 ? 2 : 4; }

// Workspace of the attention calls (offsets in bytes): status word, the
// scheduler's words (zero between calls), what the merge launch needs, then
// partial (m, l) and o rows.
struct PagedLayout {
  size_t sched, merge, ml, o, total;
};

PagedLayout paged_layout(size_t rows, int d) {
  PagedLayout L;
  L.sched = kStatusBytes;
  L.merge = L.sched + 256;
  L.ml = L.merge + align256(std::max(kMaxPlanCtas * sizeof(PagedJoin), kMaxSegs * sizeof(int2)));
  L.o = L.ml + align256(rows * sizeof(float2));
  L.total = L.o + align256(rows * (size_t)d * sizeof(float));
  return L;
}

// Partial rows: two slots per CTA (make_plan), a slot has the rows of a tile, or
// of the call if it has fewer. 640 CTAs of 64 rows cover 160 of 256 (tensor
// cores) as well.
static_assert(kMaxPlanCtas * kSimtRows >= kMaxTcCtas * 2 * kTcRows, "partial rows");
PagedLayout prompt_layout(const sv_shape& s, int n_rows) {
  const long long own = (long long)std::max(n_rows, 1) * (s.Hq / s.Hkv);
  const size_t rows = (size_t)2 * kMaxPlanCtas * std::min<long long>(kSimtRows, own);
  return paged_layout(rows, s.d);
}

// Partial rows: every row once in its shared tile and once in its own, and
// the items per CTA that cutting adds (make_plan): each holds a tile's rows, or those
// of its segment (the batch, a sequence's drafts) if that has fewer.
PagedLayout prefix_layout(const sv_shape& s) {
  PagedArgs a{};
  a.Hkv = s.Hkv;
  a.G = s.Hq / s.Hkv;
  const long long batch = (long long)s.B * s.T;
  size_t most = 0;
  for (int rows : {kSimtRows, kTcRows}) {
    paged_heads(&a, rows);
    const int tile = rows / a.gs * (rows == kTcRows ? 2 : 1);
    const size_t ctas = rows == kTcRows ? kMaxTcCtas : kMaxPlanCtas;
    auto item = [&](long long n) { return (size_t)std::min<long long>(tile, n) * a.gs; };
    auto padded = [&](long long n) {  // rows of the partial tiles of n tokens
      return (size_t)((n + tile - 1) / tile) * a.hv * item(n);
    };
    const size_t r = padded(batch) + s.B * padded(s.T) +
                     ctas * (kOwnItemsPerCta * item(s.T) + kSharedItemsPerCta * item(batch));
    most = std::max(most, r);
  }
  return paged_layout(most, s.d);
}

sv_status check_paged_ws(const PagedLayout& L, const void* ws, size_t bytes) {
  if (!ws) return fail(SV_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(SV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (bytes < L.total)
    return fail(SV_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, L.total);
  return SV_OK;
}

void fill_paged(PagedArgs* a, const sv_shape* s, void* ws, const PagedLayout& L) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  a->status = reinterpret_cast<unsigned*>(w);
  a->sched = reinterpret_cast<unsigned*>(w + L.sched);
  a->joins = reinterpret_cast<PagedJoin*>(w + L.merge);
  a->segs = reinterpret_cast<int2*>(w + L.merge);
  a->part_ml = reinterpret_cast<float2*>(w + L.ml);
  a->part_o = reinterpret_cast<float*>(w + L.o);
  a->B = s->B;
  a->Hq = s->Hq;
  a->Hkv = s->Hkv;
  a->G = s->Hq / s->Hkv;
  a->d = s->d;
  a->blk = s->blk;
  a->elt = (int)elt_bytes(s);
  a->scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)s->d));
}

cudaError_t launch_paged(const PagedArgs& a, int dtype, cudaStream_t st) {
  return paged_tc_applies(a, dtype) ? launch_paged_tc(a, st) : launch_paged_simt(a, dtype, st);
}

// int32 arrays that the kernels address word by word (null: not given).
sv_status check_words(const char* names, std::initializer_list<const void*> arrays) {
  for (const void* p : arrays)
    if (!aligned(p, 4)) return fail(SV_ERR_INVALID_ARG, "%s must be 4-byte aligned", names);
  return SV_OK;
}

// A strided row array: base and stride on 16-byte boundaries, rows apart.
sv_status check_rows(const sv_shape* s, const char* name, const void* p, long long stride, int heads) {
  if (!aligned(p, 16)) return fail(SV_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (stride < (long long)heads * s->d || stride * (long long)elt_bytes(s) % 16 ||
      stride >= (1ll << 38))
    return fail(SV_ERR_INVALID_ARG,
                "%s rows are %lld elements apart: need at least %d and a multiple of 16 bytes", name,
                stride, heads * s->d);
  return SV_OK;
}

sv_status check_pool(const sv_shape* s, const void* k_pool, const void* v_pool, int num_pages) {
  if (!k_pool || !v_pool) return fail(SV_ERR_INVALID_ARG, "k_pool/v_pool is NULL");
  if (num_pages < 1) return fail(SV_ERR_INVALID_ARG, "num_pages=%d", num_pages);
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16))
    return fail(SV_ERR_INVALID_ARG, "k_pool/v_pool must be 16-byte aligned");
  if ((long long)(num_pages + 1ll) * s->Hkv * s->blk >= kInt)
    return fail(SV_ERR_UNSUPPORTED, "pool of %d pages is too large", num_pages);
  return SV_OK;
}

}  // namespace
}  // namespace sva

using namespace sva;

extern "C" {

sv_status sv_build_tables(int B, int blk, const int32_t* old_len, const int32_t* new_len,
                          const int32_t* pinned, int32_t* block_table, int nb_max,
                          int num_pages, int32_t* free_pages, const int32_t* free_count,
                          int32_t* free_count_out, int32_t* cu_new, int32_t* slot_map,
                          int32_t* positions, int n_max, void* workspace, void* stream) {
  const CallRange range("sv_build_tables");
  if (B < 1 || blk < 1 || nb_max < 1 || num_pages < 1 || n_max < 0)
    return fail(SV_ERR_INVALID_ARG,
                "need B, blk, nb_max, num_pages >= 1 and n_max >= 0 (B=%d blk=%d nb_max=%d "
                "num_pages=%d n_max=%d)",
                B, blk, nb_max, num_pages, n_max);
  if ((long long)B * nb_max >= kInt - (1 << 20) || n_max > 1 << 30)
    return fail(SV_ERR_UNSUPPORTED, "a table of %d x %d blocks or n_max=%d new tokens is too large", B,
                nb_max, n_max);
  if (B > kMaxRequests) return fail(SV_ERR_UNSUPPORTED, "B=%d requests exceeds %d", B, kMaxRequests);
  if ((long long)num_pages * blk >= kInt || (long long)nb_max * blk >= kInt - blk)
    return fail(SV_ERR_UNSUPPORTED, "num_pages=%d or nb_max=%d of %d tokens reaches 2^31", num_pages,
                nb_max, blk);
  if (!old_len || !new_len || !block_table || !free_pages || !free_count || !free_count_out ||
      !cu_new || (n_max > 0 && !slot_map))
    return fail(SV_ERR_INVALID_ARG,
                "old_len/new_len/block_table/free_pages/free_count/free_count_out/cu_new/slot_map "
                "is NULL");
  const sv_status r = check_words("the arrays and the workspace",
                                  {old_len, new_len, pinned, block_table, free_pages, free_count,
                                   free_count_out, cu_new, slot_map, positions, workspace});
  if (r != SV_OK) return r;
  const TablesArgs a{old_len, new_len, pinned, block_table, free_pages, free_count, free_count_out,
                     cu_new, slot_map, positions, static_cast<unsigned*>(workspace), B, blk, nb_max,
                     num_pages, n_max, blk & (blk - 1) ? -1 : __builtin_ctz(blk)};
  const cudaError_t e = launch_build_tables(a, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "build_tables launch");
}

sv_status sv_write_kv(const sv_shape* shape, const void* k, long long k_stride, const void* v,
                      long long v_stride, const int32_t* slot_map, int n, void* k_pool,
                      void* v_pool, int num_pages, void* workspace, void* stream) {
  const CallRange range("sv_write_kv");
  sv_status r = check_shape(shape);
  if (r != SV_OK) return r;
  if (n < 0) return fail(SV_ERR_INVALID_ARG, "n=%d is negative", n);
  if ((r = check_pool(shape, k_pool, v_pool, num_pages)) != SV_OK) return r;
  if (n == 0) return SV_OK;
  if (!k || !v || !slot_map) return fail(SV_ERR_INVALID_ARG, "k/v/slot_map is NULL");
  if ((r = check_rows(shape, "k", k, k_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_rows(shape, "v", v, v_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_words("slot_map and the workspace", {slot_map, workspace})) != SV_OK) return r;
  const long long es = (long long)elt_bytes(shape);
  const WriteArgs a{k, v, slot_map, k_pool, v_pool, static_cast<unsigned*>(workspace), k_stride * es,
                    v_stride * es, n, shape->Hkv, shape->blk, num_pages, (int)(shape->d * es)};
  const cudaError_t e = launch_write_kv(a, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "write_kv launch");
}

size_t sv_prompt_workspace_bytes(const sv_shape* shape, int n_rows) {
  if (check_shape(shape) != SV_OK || n_rows < 0) return 0;
  return prompt_layout(*shape, n_rows).total;
}

size_t sv_prefix_workspace_bytes(const sv_shape* shape) {
  if (check_shape(shape) != SV_OK) return 0;
  return prefix_layout(*shape).total;
}

sv_status sv_prompt_attend(const sv_shape* shape, const void* q, long long q_stride, int n_rows,
                           const void* k_pool, const void* v_pool, const int32_t* block_table,
                           int nb_max, int num_pages, const int32_t* seq_ctx,
                           const int32_t* cu_q, void* out, void* workspace, size_t ws_bytes,
                           void* stream) {
  const CallRange range("sv_prompt_attend");
  sv_status r = check_shape(shape);
  if (r != SV_OK) return r;
  if (n_rows < 0 || nb_max < 1)
    return fail(SV_ERR_INVALID_ARG, "need n_rows >= 0 and nb_max >= 1 (n_rows=%d nb_max=%d)", n_rows,
                nb_max);
  if (shape->B > kMaxSegs - 1)
    return fail(SV_ERR_UNSUPPORTED, "B=%d sequences exceeds %d", shape->B, kMaxSegs - 1);
  if ((r = check_pool(shape, k_pool, v_pool, num_pages)) != SV_OK) return r;
  if ((long long)nb_max * shape->blk >= kInt - 1024 || (long long)shape->B * nb_max >= kInt)
    return fail(SV_ERR_UNSUPPORTED, "block table of %d x %d blocks of %d tokens is too large",
                shape->B, nb_max, shape->blk);
  if ((long long)n_rows * shape->Hq >= kInt)
    return fail(SV_ERR_UNSUPPORTED, "n_rows=%d rows of %d heads reach 2^31", n_rows, shape->Hq);
  if (!block_table || !seq_ctx || !cu_q)
    return fail(SV_ERR_INVALID_ARG, "block_table/seq_ctx/cu_q is NULL");
  if ((r = check_words("block_table/seq_ctx/cu_q", {block_table, seq_ctx, cu_q})) != SV_OK) return r;
  const PagedLayout L = prompt_layout(*shape, n_rows);
  if ((r = check_paged_ws(L, workspace, ws_bytes)) != SV_OK) return r;
  if (n_rows == 0) return SV_OK;
  if (!q || !out) return fail(SV_ERR_INVALID_ARG, "q/out is NULL");
  if ((r = check_rows(shape, "q", q, q_stride, shape->Hq)) != SV_OK) return r;
  if (!aligned(out, 16)) return fail(SV_ERR_INVALID_ARG, "out must be 16-byte aligned");
  PagedArgs a{};
  fill_paged(&a, shape, workspace, L);
  a.q = q;
  a.q_stride = q_stride;
  a.n_rows = n_rows;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.block_table = block_table;
  a.nb_max = nb_max;
  a.num_pages = num_pages;
  a.seq_ctx = seq_ctx;
  a.cu_q = cu_q;
  a.out = out;
  const cudaError_t e = launch_paged(a, shape->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "prompt_attend launch");
}

sv_status sv_prefix_attend(const sv_shape* shape, const void* q, const sv_kv* kv, int n_shared,
                           const void* draft_k, const void* draft_v,
                           const int32_t* draft_parent, void* out, void* workspace,
                           size_t ws_bytes, void* stream) {
  const CallRange range("sv_prefix_attend");
  sv_status r = check_shape(shape);
  if (r != SV_OK) return r;
  if ((r = check_kv(shape, kv, true, kMaxSegs - 1)) != SV_OK) return r;
  if (shape->B > kMaxSegs - 1)
    return fail(SV_ERR_UNSUPPORTED, "B=%d sequences exceeds %d", shape->B, kMaxSegs - 1);
  if (n_shared < 0) return fail(SV_ERR_INVALID_ARG, "n_shared=%d is negative", n_shared);
  for (int b = 0; b < (kv->seq_ctx ? shape->B : 1); ++b) {
    const int c = kv->seq_ctx ? kv->seq_ctx[b] : kv->ctx;
    if (n_shared > c / shape->blk)
      return fail(SV_ERR_INVALID_ARG, "n_shared=%d exceeds the %d full blocks of sequence %d",
                  n_shared, c / shape->blk, b);
  }
  if ((long long)shape->B * kv->nb_max >= kInt ||
      (long long)shape->B * shape->T * shape->Hq * 4 >= kInt)
    return fail(SV_ERR_UNSUPPORTED, "B=%d: the block table or the batch's rows are too many", shape->B);
  if (!q || !draft_k || !draft_v || !out)
    return fail(SV_ERR_INVALID_ARG, "q/draft_k/draft_v/out is NULL");
  if (!aligned(q, 16) || !aligned(draft_k, 16) || !aligned(draft_v, 16) || !aligned(out, 16))
    return fail(SV_ERR_INVALID_ARG, "q/draft_k/draft_v/out must be 16-byte aligned");
  if ((r = check_words("block_table", {kv->block_table})) != SV_OK) return r;
  if ((r = check_parents(draft_parent, shape->T)) != SV_OK) return r;
  const PagedLayout L = prefix_layout(*shape);
  if ((r = check_paged_ws(L, workspace, ws_bytes)) != SV_OK) return r;
  PagedArgs a{};
  fill_paged(&a, shape, workspace, L);
  a.q = q;
  a.q_stride = (long long)shape->Hq * shape->d;
  a.n_rows = shape->B * shape->T;
  int most = kv->ctx;  // the longest context
  for (int b = 0; kv->seq_ctx && b < shape->B; ++b) most = b ? std::max(most, kv->seq_ctx[b]) : kv->seq_ctx[b];
  // without a single token there need not be a pool (check_kv): none is read
  a.k_pool = most ? kv->k_pool : draft_k;
  a.v_pool = most ? kv->v_pool : draft_v;
  a.draft_k = draft_k;
  a.draft_v = draft_v;
  a.block_table = kv->block_table;
  a.nb_max = kv->nb_max;
  a.num_pages = most ? kv->num_pages : 0;
  a.out = out;
  a.prefix = 1;
  a.T = shape->T;
  a.n_shared = n_shared;
  a.ctx = kv->ctx;
  a.var = kv->seq_ctx != nullptr;
  for (int b = 0; a.var && b < shape->B; ++b) a.seq_len[b] = kv->seq_ctx[b];
  fill_ancestors(draft_parent, shape->T, a.anc);
  const cudaError_t e = launch_paged(a, shape->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "prefix_attend launch");
}

}  // extern "C"
