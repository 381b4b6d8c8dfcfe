// C entries of the operators between a fused projection and attention over a
// 4-bit cache: validation, workspace layout and launches. Declarations and
// contracts: include/sva.h.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "host.h"
#include "kv4.h"

namespace sva {
namespace {

constexpr long long kInt = 1ll << 31;

size_t elt_bytes(const sv_shape* s) { return s->dtype == SV_BF16 ? 2 : 4; }

sv_status check_words4(const char* names, std::initializer_list<const void*> arrays) {
  for (const void* p : arrays)
    if (!aligned(p, 4)) return fail(SV_ERR_INVALID_ARG, "%s must be 4-byte aligned", names);
  return SV_OK;
}

// A strided row array: base and stride on 16-byte boundaries, rows apart.
sv_status check_rows4(const sv_shape* s, const char* name, const void* p, long long stride, int heads) {
  if (!p) return fail(SV_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 16)) return fail(SV_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (stride < (long long)heads * s->d || stride >= (1ll << 38) || stride * (long long)elt_bytes(s) % 16)
    return fail(SV_ERR_INVALID_ARG,
                "%s rows are %lld elements apart: need at least %d and a multiple of 16 bytes", name, stride,
                heads * s->d);
  return SV_OK;
}

sv_status check_pools(const sv_shape* s, const void* k_pool, const void* v_pool, int num_pages) {
  if (!k_pool || !v_pool) return fail(SV_ERR_INVALID_ARG, "k_pool/v_pool is NULL");
  if (num_pages < 1) return fail(SV_ERR_INVALID_ARG, "num_pages=%d", num_pages);
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16))
    return fail(SV_ERR_INVALID_ARG, "k_pool/v_pool must be 16-byte aligned");
  if ((long long)(num_pages + 1ll) * s->Hkv * s->blk >= kInt)
    return fail(SV_ERR_UNSUPPORTED, "pool of %d pages is too large", num_pages);
  return SV_OK;
}

sv_status check_rope(const sv_shape* s, const sv_rope* r, const int32_t* positions) {
  if (!r) return fail(SV_ERR_INVALID_ARG, "rope is NULL");
  if (r->rot < 0 || r->rot > s->d || r->rot % 8)
    return fail(SV_ERR_INVALID_ARG, "rot=%d must be a multiple of 8 in [0, d=%d]", r->rot, s->d);
  if (r->rot && (!r->table || r->max_pos < 1 || !positions))
    return fail(SV_ERR_INVALID_ARG, "a rotation needs table, max_pos >= 1 (%d) and positions", r->max_pos);
  if (!(r->eps >= 0.f) || std::isinf(r->eps)) return fail(SV_ERR_INVALID_ARG, "eps=%g", (double)r->eps);
  if (!aligned(r->q_weight, 16) || !aligned(r->k_weight, 16) || !aligned(r->table, 16))
    return fail(SV_ERR_INVALID_ARG, "table/q_weight/k_weight must be 16-byte aligned");
  return check_words4("positions", {positions});
}

void fill_rope(RopeArgs* a, const sv_shape* s, const sv_rope* r, const int32_t* positions, int n, void* ws) {
  a->positions = positions;
  a->table = r->table;
  a->q_weight = r->q_weight;
  a->k_weight = r->k_weight;
  a->eps = r->eps;
  a->rot = r->rot;
  a->max_pos = r->max_pos;
  a->interleaved = r->interleaved != 0;
  a->status = static_cast<unsigned*>(ws);
  a->n = n;
  a->Hq = s->Hq;
  a->Hkv = s->Hkv;
  a->d = s->d;
  a->blk = s->blk;
}

// What every call over a 4-bit cache needs of its shape and pools.
sv_status check_shape4(const sv_shape* s) {
  const sv_status r = check_shape(s);
  if (r != SV_OK) return r;
  if (s->d % 16) return fail(SV_ERR_UNSUPPORTED, "head dim %d of a 4-bit cache must be a multiple of 16", s->d);
  if (s->blk % kPiece)
    return fail(SV_ERR_UNSUPPORTED, "pages of %d tokens of a 4-bit cache: need a multiple of %d", s->blk, kPiece);
  if (s->Hkv > 4096 || s->B > 65535)
    return fail(SV_ERR_UNSUPPORTED, "Hkv=%d heads or B=%d sequences of a 4-bit cache exceed 4096 and 65535", s->Hkv, s->B);
  return SV_OK;
}
sv_status check_kv4(const sv_shape* s, const sv_kv4* kv) {
  if (!kv) return fail(SV_ERR_INVALID_ARG, "kv is NULL");
  const sv_status r = check_pools(s, kv->k_pool, kv->v_pool, kv->num_pages);
  if (r != SV_OK) return r;
  return check_words4("k_exp and v_exp", {kv->k_exp, kv->v_exp});
}
// ... and of its sequences.
sv_status check_seqs4(const sv_shape* s, const sv_kv4* kv) {
  if (!kv->block_table || !kv->seq_ctx) return fail(SV_ERR_INVALID_ARG, "block_table/seq_ctx is NULL");
  if (kv->nb_max < 1) return fail(SV_ERR_INVALID_ARG, "nb_max=%d", kv->nb_max);
  if ((long long)(kv->nb_max + 1ll) * s->blk >= kInt - 1024 || (long long)s->B * kv->nb_max >= kInt)
    return fail(SV_ERR_UNSUPPORTED, "block table of %d x %d blocks of %d tokens is too large", s->B, kv->nb_max,
                s->blk);
  return check_words4("block_table and seq_ctx", {kv->block_table, kv->seq_ctx});
}

Rows4Args rows4(const sv_shape* s, const sv_kv4* kv, const int32_t* slots, int n, void* ws) {
  Rows4Args a{};
  a.k_pool = static_cast<uint8_t*>(kv->k_pool);
  a.v_pool = static_cast<uint8_t*>(kv->v_pool);
  a.slots = slots;
  a.k_exp = kv->k_exp;
  a.v_exp = kv->v_exp;
  a.status = static_cast<unsigned*>(ws);
  a.n = n;
  a.Hkv = s->Hkv;
  a.d = s->d;
  a.blk = s->blk;
  a.num_pages = kv->num_pages;
  return a;
}

// Warps of the row kernels: the grid's blocks have to fit 31 bits.
sv_status check_row_count(const sv_shape* s, int n) {
  if (n < 0) return fail(SV_ERR_INVALID_ARG, "n=%d is negative", n);
  if ((long long)n * (s->Hq + 2 * s->Hkv) * s->d >= (1ll << 40))
    return fail(SV_ERR_UNSUPPORTED, "n=%d rows are too many", n);
  return SV_OK;
}

// Workspace of the attention: status word, the pairs' slots, then the segments' (reference,
// sum) and sums of values, one slot per pair and CTA at most.
struct Layout4 {
  size_t slots, ml, o, total;
};
Layout4 layout4(const sv_shape& s) {
  size_t rows = 0;
  const long long stacked = (long long)s.T * (s.Hq / s.Hkv), pairs = (long long)s.B * s.Hkv;
  const int most[2] = {kSimt4Rows, kTc4Rows}, ctas[2] = {kMaxSimt4Ctas, kMaxTc4Ctas};
  for (int i = 0; i < 2; ++i) {
    const long long tiles = (stacked + most[i] - 1) / most[i], r = std::min<long long>(most[i], stacked);
    rows = std::max(rows, (size_t)((tiles * pairs + ctas[i]) * (i + 1) * r));  // (two streams on the tensor cores)
  }
  Layout4 L;
  L.slots = kStatusBytes;
  L.ml = L.slots + align256((stacked + kSimt4Rows - 1) / kSimt4Rows * pairs * sizeof(int2));
  L.o = L.ml + align256(rows * sizeof(float2));
  L.total = L.o + align256(rows * s.d * sizeof(float));
  return L;
}

}  // namespace
}  // namespace sva

using namespace sva;

extern "C" {

sv_status sv_norm_rope(const sv_shape* shape, const sv_rope* rope, const int32_t* positions, int n,
                       const void* q, long long q_stride, const void* k, long long k_stride, void* q_out,
                       long long q_out_stride, void* k_out, long long k_out_stride, void* workspace,
                       void* stream) {
  const CallRange range("sv_norm_rope");
  sv_status r = check_shape(shape);
  if (r != SV_OK) return r;
  if ((r = check_rope(shape, rope, positions)) != SV_OK) return r;
  if ((r = check_row_count(shape, n)) != SV_OK) return r;
  if (n == 0) return SV_OK;
  if (q && ((r = check_rows4(shape, "q", q, q_stride, shape->Hq)) != SV_OK ||
            (r = check_rows4(shape, "q_out", q_out, q_out_stride, shape->Hq)) != SV_OK))
    return r;
  if ((r = check_rows4(shape, "k", k, k_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_rows4(shape, "k_out", k_out, k_out_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_words4("the workspace", {workspace})) != SV_OK) return r;
  RopeArgs a{};
  fill_rope(&a, shape, rope, positions, n, workspace);
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.qo_stride = q_out_stride;
  a.ko_stride = k_out_stride;
  const cudaError_t e = launch_rope(a, shape->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "norm_rope launch");
}

sv_status sv_rope_write_kv(const sv_shape* shape, const sv_rope* rope, const int32_t* positions, int n,
                           const void* q, long long q_stride, void* q_out, long long q_out_stride,
                           const void* k, long long k_stride, const void* v, long long v_stride,
                           const int32_t* slot_map, void* k_pool, void* v_pool, int num_pages,
                           void* workspace, void* stream) {
  const CallRange range("sv_rope_write_kv");
  sv_status r = check_shape(shape);
  if (r != SV_OK) return r;
  if ((r = check_rope(shape, rope, positions)) != SV_OK) return r;
  if ((r = check_row_count(shape, n)) != SV_OK) return r;
  if ((r = check_pools(shape, k_pool, v_pool, num_pages)) != SV_OK) return r;
  if (n == 0) return SV_OK;
  if (!slot_map) return fail(SV_ERR_INVALID_ARG, "slot_map is NULL");
  if (q && ((r = check_rows4(shape, "q", q, q_stride, shape->Hq)) != SV_OK ||
            (r = check_rows4(shape, "q_out", q_out, q_out_stride, shape->Hq)) != SV_OK))
    return r;
  if ((r = check_rows4(shape, "k", k, k_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_rows4(shape, "v", v, v_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_words4("slot_map and the workspace", {slot_map, workspace})) != SV_OK) return r;
  RopeArgs a{};
  fill_rope(&a, shape, rope, positions, n, workspace);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.slots = slot_map;
  a.num_pages = num_pages;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.qo_stride = q_out_stride;
  const cudaError_t e = launch_rope(a, shape->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "rope_write_kv launch");
}

size_t sv_kv4_page_bytes(const sv_shape* shape) {
  if (check_shape4(shape) != SV_OK) return 0;
  return (size_t)shape->Hkv * (shape->blk / kPiece) * piece_bytes(shape->d);
}

sv_status sv_write_kv4(const sv_shape* shape, const void* k, long long k_stride, const void* v,
                       long long v_stride, const int32_t* slot_map, int n, const sv_kv4* kv,
                       void* workspace, void* stream) {
  const CallRange range("sv_write_kv4");
  sv_status r = check_shape4(shape);
  if (r != SV_OK) return r;
  if ((r = check_kv4(shape, kv)) != SV_OK) return r;
  if ((r = check_row_count(shape, n)) != SV_OK) return r;
  if (n == 0) return SV_OK;
  if (!slot_map) return fail(SV_ERR_INVALID_ARG, "slot_map is NULL");
  if ((r = check_rows4(shape, "k", k, k_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_rows4(shape, "v", v, v_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_words4("slot_map and the workspace", {slot_map, workspace})) != SV_OK) return r;
  Rows4Args a = rows4(shape, kv, slot_map, n, workspace);
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  const cudaError_t e = launch_write_kv4(a, shape->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "write_kv4 launch");
}

sv_status sv_read_kv4(const sv_shape* shape, const sv_kv4* kv, const int32_t* slot_map, int n,
                      void* k_out, long long k_stride, void* v_out, long long v_stride, void* workspace,
                      void* stream) {
  const CallRange range("sv_read_kv4");
  sv_status r = check_shape4(shape);
  if (r != SV_OK) return r;
  if ((r = check_kv4(shape, kv)) != SV_OK) return r;
  if ((r = check_row_count(shape, n)) != SV_OK) return r;
  if (n == 0) return SV_OK;
  if (!slot_map) return fail(SV_ERR_INVALID_ARG, "slot_map is NULL");
  if ((r = check_rows4(shape, "k_out", k_out, k_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_rows4(shape, "v_out", v_out, v_stride, shape->Hkv)) != SV_OK) return r;
  if ((r = check_words4("slot_map and the workspace", {slot_map, workspace})) != SV_OK) return r;
  Rows4Args a = rows4(shape, kv, slot_map, n, workspace);
  a.k_out = k_out;
  a.v_out = v_out;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  const cudaError_t e = launch_read_kv4(a, shape->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "read_kv4 launch");
}

sv_status sv_build_reps_kv4(const sv_shape* shape, const sv_kv4* kv, const int32_t* from_len,
                            int max_blocks, float* reps, void* workspace, void* stream) {
  const CallRange range("sv_build_reps_kv4");
  sv_status r = check_shape4(shape);
  if (r != SV_OK) return r;
  if ((r = check_kv4(shape, kv)) != SV_OK) return r;
  if ((r = check_seqs4(shape, kv)) != SV_OK) return r;
  if (max_blocks < 0 || max_blocks > kv->nb_max)
    return fail(SV_ERR_INVALID_ARG, "max_blocks=%d outside [0, nb_max=%d]", max_blocks, kv->nb_max);
  if ((long long)shape->B * shape->Hkv * max_blocks >= (1ll << 33))
    return fail(SV_ERR_UNSUPPORTED, "B=%d: the blocks are too many", shape->B);
  if ((r = check_words4("from_len and the workspace", {from_len, workspace})) != SV_OK) return r;
  if (max_blocks == 0) return SV_OK;
  if (!reps || !aligned(reps, 16)) return fail(SV_ERR_INVALID_ARG, "reps NULL or not 16-byte aligned");
  const Reps4Args a{static_cast<const uint8_t*>(kv->k_pool), kv->block_table, kv->seq_ctx, from_len,
                    kv->k_exp, reps, static_cast<unsigned*>(workspace), shape->B, shape->Hkv, shape->d,
                    shape->blk, kv->nb_max, kv->num_pages, max_blocks};
  const cudaError_t e = launch_reps_kv4(a, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "build_reps_kv4 launch");
}

size_t sv_kv4_workspace_bytes(const sv_shape* shape) {
  if (check_shape4(shape) != SV_OK || shape->B > kMaxB4) return 0;
  return layout4(*shape).total;
}

sv_status sv_attend_kv4(const sv_shape* shape, const void* q, const sv_kv4* kv, const int32_t* sel,
                        int n_sel, int sel_stride, const void* draft_k, const void* draft_v,
                        const int32_t* draft_parent, void* out, void* workspace, size_t ws_bytes,
                        void* stream) {
  const CallRange range("sv_attend_kv4");
  sv_status r = check_shape4(shape);
  if (r != SV_OK) return r;
  if (shape->B > kMaxB4) return fail(SV_ERR_UNSUPPORTED, "B=%d sequences exceeds %d", shape->B, kMaxB4);
  if ((r = check_kv4(shape, kv)) != SV_OK) return r;
  if ((r = check_seqs4(shape, kv)) != SV_OK) return r;
  if ((long long)shape->B * (kv->nb_max + 1ll) * shape->blk >= kInt * 16)
    return fail(SV_ERR_UNSUPPORTED, "B=%d: the batch's tokens are too many", shape->B);
  // the line of key tiles (64 tokens at least, 32 rows at least) is counted in 31 bits
  const long long row_tiles = (shape->T * (shape->Hq / shape->Hkv) + kSimt4Rows - 1) / kSimt4Rows;
  if (((long long)shape->B * (kv->nb_max + 1ll) * shape->blk >> 6) + shape->B * (1ll + kMaxPairCost) >= kInt / (shape->Hkv * row_tiles))
    return fail(SV_ERR_UNSUPPORTED, "B=%d, %d heads: the batch's tokens are too many", shape->B, shape->Hkv);
  if (sel && (n_sel < 0 || n_sel > sel_stride || n_sel > kv->nb_max))
    return fail(SV_ERR_INVALID_ARG, "n_sel=%d outside [0, sel_stride=%d] or beyond nb_max=%d", n_sel, sel_stride,
                kv->nb_max);
  if ((long long)shape->B * shape->T * shape->Hq * 4 >= kInt)
    return fail(SV_ERR_UNSUPPORTED, "B=%d: the batch's rows are too many", shape->B);
  if (!q || !draft_k || !draft_v || !out) return fail(SV_ERR_INVALID_ARG, "q/draft_k/draft_v/out is NULL");
  if (!aligned(q, 16) || !aligned(draft_k, 16) || !aligned(draft_v, 16) || !aligned(out, 16))
    return fail(SV_ERR_INVALID_ARG, "q/draft_k/draft_v/out must be 16-byte aligned");
  if ((r = check_words4("sel", {sel})) != SV_OK) return r;
  if ((r = check_parents(draft_parent, shape->T)) != SV_OK) return r;
  const Layout4 L = layout4(*shape);
  if (!workspace) return fail(SV_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(workspace, 256)) return fail(SV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (ws_bytes < L.total)
    return fail(SV_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, L.total);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  Attend4Args a{};
  a.q = q;
  a.draft_k = draft_k;
  a.draft_v = draft_v;
  a.out = out;
  a.k_pool = static_cast<const uint8_t*>(kv->k_pool);
  a.v_pool = static_cast<const uint8_t*>(kv->v_pool);
  a.block_table = kv->block_table;
  a.seq_ctx = kv->seq_ctx;
  a.sel = sel;
  a.k_exp = kv->k_exp;
  a.v_exp = kv->v_exp;
  a.status = reinterpret_cast<unsigned*>(w);
  a.slots = reinterpret_cast<int2*>(w + L.slots);
  a.part_ml = reinterpret_cast<float2*>(w + L.ml);
  a.part_o = reinterpret_cast<float*>(w + L.o);
  a.B = shape->B;
  a.T = shape->T;
  a.Hq = shape->Hq;
  a.Hkv = shape->Hkv;
  a.G = shape->Hq / shape->Hkv;
  a.d = shape->d;
  a.blk = shape->blk;
  a.nb_max = kv->nb_max;
  a.num_pages = kv->num_pages;
  a.n_sel = n_sel;
  a.sel_stride = sel_stride;
  a.ppb = shape->blk / kPiece;
  a.ppb_shift = a.ppb & (a.ppb - 1) ? -1 : __builtin_ctz(a.ppb);
  a.g_shift = a.G & (a.G - 1) ? -1 : __builtin_ctz(a.G);
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)shape->d));
  fill_ancestors(draft_parent, shape->T, a.anc);
  const cudaError_t e = attend4_tc_applies(a, shape->dtype) ? launch_attend4_tc(a, (cudaStream_t)stream)
                                                            : launch_attend4_simt(a, shape->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "attend_kv4 launch");
}

}  // extern "C"
