// Arguments of the operators between a fused projection and attention over a
// cache held in 4 bits: head norms with rotation, rows into 4-bit pages and
// back, representatives and verification attention over such pages.
#pragma once

#include "internal.h"

namespace sva {

// ---------------------------------------------------------------- norm and rotation
struct RopeArgs {
  const void *q, *k, *v;       // rows of heads; q may be null, v null without pools
  void *q_out, *k_out;         // rows; k_out null with pools
  void *k_pool, *v_pool;       // [num_pages, Hkv, blk, d] or null
  const int32_t* slots;        // with pools: [n]
  const int32_t* positions;    // [n] or null (no rotation)
  const float* table;          // [max_pos, rot]: cosines, sines
  const void *q_weight, *k_weight;  // [d] or null
  unsigned* status;            // may be null
  long long q_stride, k_stride, v_stride, qo_stride, ko_stride;  // elements
  int n, Hq, Hkv, d, blk, num_pages, rot, max_pos, interleaved;
  int parts_shift;             // log2 of the warps that share a token's heads
  float eps, inv_d;
};
cudaError_t launch_rope(RopeArgs a, int dtype, cudaStream_t st);

// ---------------------------------------------------------------- 4-bit pages
// A pool is [num_pages, Hkv, blk / 16] pieces of 16 tokens of one head, 9 d
// bytes each: 8 d bytes of E2M1 codes, then d bytes of E4M3 scales, one for
// every 16 dims of a token.
//   K codes [d / 16][16 tokens][8]: byte j holds dims 2 j (low bits) and 2 j + 1,
//     scales [16 tokens][d / 16]
//   V codes [d / 16][8][16 tokens]: byte c holds dims c (low bits) and c + 8,
//     scales [d / 16][16 tokens]
// A token's bytes are its own, so that a write never reads. K keeps a token's
// dims together and V a dim's tokens, as the two products take them: scores
// contract over dims, outputs over tokens.
constexpr int kPiece = 16;  // tokens of a piece
__host__ __device__ constexpr int piece_bytes(int d) { return 9 * d; }

struct Rows4Args {
  const void *k, *v;             // write: rows [n, Hkv, d]
  void *k_out, *v_out;           // read: rows
  uint8_t *k_pool, *v_pool;
  const int32_t* slots;          // [n]
  const int32_t *k_exp, *v_exp;  // [Hkv] or null
  unsigned* status;              // may be null
  long long k_stride, v_stride;  // elements
  int n, Hkv, d, blk, num_pages;
  int heads;                     // of a block (set by the launch)
  int wide;                      // rows lie on 32-byte boundaries (set by the launch)
};
cudaError_t launch_write_kv4(Rows4Args a, int dtype, cudaStream_t st);
cudaError_t launch_read_kv4(Rows4Args a, int dtype, cudaStream_t st);

struct Reps4Args {
  const uint8_t* k_pool;
  const int32_t* block_table;  // [B, nb_max]
  const int32_t* seq_ctx;      // [B]
  const int32_t* from_len;     // [B] or null
  const int32_t* k_exp;        // [Hkv] or null
  float* reps;                 // [B, Hkv, nb_max, d]
  unsigned* status;            // may be null
  int B, Hkv, d, blk, nb_max, num_pages, max_blocks;
  int heads, blk_shift;        // of a CTA; log2 of blk or -1 (both set by the launch)
};
cudaError_t launch_reps_kv4(Reps4Args a, cudaStream_t st);

// ---------------------------------------------------------------- attention
constexpr int kMaxB4 = 1024;         // sequences of a call
constexpr int kSimt4Rows = 32;       // row tile on the CUDA cores
constexpr int kTc4Rows = 64;         // ... and on the tensor cores, at most
constexpr int kMaxSimt4Ctas = 640;   // CTAs of a launch at most
constexpr int kMaxTc4Ctas = 160;
constexpr int kMaxPairCost = 8;      // of Attend4Args::pair_cost

// The T * G stacked rows of a (sequence, KV head) are cut into row tiles; a pair is one row
// tile of one (sequence, head). A pair's pieces (16 keys each) make key tiles of `ppt` pieces.
// The pairs' key tiles are laid end to end, with what beginning a pair costs ahead of them, and
// cut into equal shares, one per CTA; what a CTA has of a pair is a segment. (That cost left
// out: 16 sequences of 1 to 32768 tokens, 8 heads each, 82 us, as the CTAs whose share held
// several short pairs were last; counted as 2 tiles 64, as 4 to 8 tiles 58.) Segment (pair p,
// CTA c) leaves its rows' sums in slot p + c (p and c only grow along the line, so no two
// segments share one), once for each of its `streams`.
struct Attend4Args {
  const void *q, *draft_k, *draft_v;
  void* out;
  const uint8_t *k_pool, *v_pool;
  const int32_t* block_table;    // [B, nb_max]
  const int32_t* seq_ctx;        // [B]
  const int32_t* sel;            // [B, Hkv, sel_stride] or null: every full block
  const int32_t *k_exp, *v_exp;  // [Hkv] or null
  unsigned* status;
  int2* slots;    // workspace [pairs]: first slot of a pair and number of slots
  float2* part_ml;  // [slots, streams, rows]: reference (log2 domain) and sum
  float* part_o;    // [slots, streams, rows, d], in units of 2^v_exp
  int B, T, Hq, Hkv, G, d, blk, nb_max, num_pages, n_sel, sel_stride;
  int rows, row_tiles;  // rows of a row tile (of all but the last), row tiles of a (b, h)
  int streams;    // 2: a segment's even and odd tiles are summed apart
  int ppb, ppt, ppt_shift;  // pieces of a block and of a key tile (a power of two)
  int ppb_shift, g_shift;   // log2 of ppb and of G, -1 where it is no power of two
  int pair_cost;  // key tiles' time that beginning a pair takes
  int ctas;
  float scale_log2;  // log2(e) / sqrt(d)
  unsigned long long anc[kMaxT];
};
// Ends the copies of a CTA that gave up, when nobody waits on its barriers any more. A stage's
// barrier counts one arrival for K's copies and one for V's; the warps that issue them may have
// stopped some tiles apart, and a stage that only one of them armed would never complete:
// arrive(stage) stands in for the other. wait(stage, parity) then ends as the bytes land.
#ifdef __CUDACC__
#pragma nv_exec_check_disable
#endif
template <typename Arrive, typename Wait>
__host__ __device__ inline void end_copies(uint32_t k_tiles, uint32_t v_tiles, uint32_t stages, Arrive arrive, Wait wait) {
  const uint32_t some = k_tiles < v_tiles ? v_tiles : k_tiles, both = k_tiles + v_tiles - some;
  for (uint32_t i = both; i < some; ++i) arrive(i % stages);
  for (uint32_t i = some > stages ? some - stages : 0; i < some; ++i) wait(i % stages, i / stages & 1u);
}

// Each launches the attention over the cache and then the join with the drafts.
cudaError_t launch_attend4_simt(Attend4Args a, int dtype, cudaStream_t st);
// bf16, head dims up to 128.
bool attend4_tc_applies(const Attend4Args& a, int dtype);
cudaError_t launch_attend4_tc(Attend4Args a, cudaStream_t st);
// Adds the drafts to what the attention launched just before left (the same
// arguments) and writes out.
cudaError_t launch_join4(const Attend4Args& a, int dtype, cudaStream_t st);

}  // namespace sva
