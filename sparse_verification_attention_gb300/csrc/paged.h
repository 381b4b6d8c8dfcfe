// Arguments of the paged-cache operators: block tables and slots from request
// lengths, packed K/V rows into pages, and attention of packed or stacked
// query rows over the pages.
#pragma once

#include "internal.h"

namespace sva {

// ---------------------------------------------------------------- tables
constexpr int kMaxRequests = 4096;  // requests of one sv_build_tables call

struct TablesArgs {
  const int32_t* old_len;     // [B]
  const int32_t* new_len;     // [B]
  const int32_t* pinned;      // [B] or null
  int32_t* block_table;       // [B, nb_max]
  int32_t* free_pages;        // [num_pages], a stack
  const int32_t* free_count;  // [1]
  int32_t* free_count_out;    // [1], may be free_count
  int32_t* cu_new;            // [B + 1]
  int32_t* slot_map;          // [n_max]
  int32_t* positions;         // [n_max] or null
  unsigned* status;           // may be null
  int B, blk, nb_max, num_pages, n_max;
  int blk_shift;              // log2(blk), -1 if blk is no power of two
};
cudaError_t launch_build_tables(const TablesArgs& a, cudaStream_t st);

struct WriteArgs {
  const void *k, *v;             // [N, Hkv, d], rows k_stride / v_stride apart
  const int32_t* slots;          // [N]
  void *k_pool, *v_pool;         // [num_pages, Hkv, blk, d]
  unsigned* status;              // may be null
  long long k_stride, v_stride;  // bytes
  int n, Hkv, blk, num_pages;
  int row_bytes;  // one head's row
};
cudaError_t launch_write_kv(const WriteArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- attention
constexpr int kMaxSegs = 1025;      // row segments of one call: sequences, and a shared prefix
constexpr int kMaxPlanCtas = 640;   // CTAs of a launch at most
constexpr int kOwnItemsPerCta = 2, kSharedItemsPerCta = 2;  // prefix form, see make_plan
constexpr int kStreamCost = 8;      // key tiles' time that joining cut units takes (make_plan)
constexpr int kSimtRows = 64;       // rows of an item on the CUDA cores
constexpr int kTcRows = 128;        // rows of a set on the tensor cores; an item has two
constexpr int kMaxTcCtas = 160;

// A unit that was cut behind its beginning: how many CTAs hold the rest of it
// (0: none was), and its rows.
struct PagedJoin {
  int more, tok0, ntok, head0, heads;
};

// One attention over the paged cache. Its query rows lie in segments: runs of
// consecutive rows ("tokens", Hq heads each) that attend to one sequence of
// keys. Prompt form: segment b = the rows cu_q[b]..cu_q[b+1], the last of
// seq_ctx[b] tokens, causal. Prefix form: segment 0 = every row of the batch
// over the shared pages of sequence 0's table row, segment 1 + b = the T
// drafts of sequence b over its own pages and then the drafts they see.
struct PagedArgs {
  const void* q;              // [n_rows, Hq, d], rows q_stride elements apart
  const void* k_pool;         // [num_pages, Hkv, blk, d]
  const void* v_pool;
  const void* draft_k;        // prefix form: [B, T, Hkv, d]
  const void* draft_v;
  void* out;                  // [n_rows, Hq, d]
  const int32_t* block_table; // [B, nb_max]
  const int32_t* seq_ctx;     // prompt form: device [B]
  const int32_t* cu_q;        // prompt form: device [B + 1]
  // workspace: status word, the scheduler's two words (zero between calls), what
  // the attention leaves to the merge launch, and the partial rows
  unsigned* status;
  unsigned* sched;
  PagedJoin* joins;           // prompt form: [CTAs]
  int2* segs;                 // prefix form: first partial row and runs of each segment
  float* part_o;              // [partial rows, d]
  float2* part_ml;            // [partial rows]: running maximum (log2 domain), sum
  long long q_stride;
  int B, Hq, Hkv, G, d, blk, nb_max, num_pages, n_rows;
  // a KV head's G query heads in hs groups of at most gs heads, so that the
  // gs rows of one token fit a row tile; hv = Hkv * hs
  int gs, hs, hv;
  // the launch's work split (make_plan): CTAs, the fewest key tiles that a run
  // is worth, tokens of a row tile, tokens above which its rows are two sets,
  // log2 of the keys of a key tile, key tiles' time that an item takes besides its own
  int ctas, min_run, tile, one_set, key_shift, item_cost;
  int elt;                    // bytes of an element
  int out_wide;               // rows of out lie on 32-byte boundaries
  float scale_log2;           // log2(e) / sqrt(d)
  int prefix;                 // 0: prompt form, 1: prefix form
  int T, n_shared;
  int ctx;                    // prefix form: uniform context ...
  int var;                    // ... or per sequence in seq_len
  int32_t seq_len[kMaxSegs - 1];
  unsigned long long anc[kMaxT];
};

// Cut every KV head's query heads into groups that fit a tile of `rows` rows.
inline void paged_heads(PagedArgs* a, int rows) {
  a->hs = (a->G + rows - 1) / rows;
  a->gs = (a->G + a->hs - 1) / a->hs;
  a->hs = (a->G + a->gs - 1) / a->gs;
  a->hv = a->Hkv * a->hs;
}

// Each launches the attention and the merge of its partial rows.
cudaError_t launch_paged_simt(PagedArgs a, int dtype, cudaStream_t st);
// bf16, head dims up to 128, pages that tile 128 keys (or 128 keys a page).
bool paged_tc_applies(const PagedArgs& a, int dtype);
cudaError_t launch_paged_tc(PagedArgs a, cudaStream_t st);
// Join the partial rows that the attention kernel launched just before left
// (the same arguments).
cudaError_t launch_paged_merge(const PagedArgs& a, int dtype, cudaStream_t st);

}  // namespace sva
