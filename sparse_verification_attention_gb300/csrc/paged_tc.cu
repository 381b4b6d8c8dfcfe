// Attention of packed or stacked query rows over the paged cache on the
// 5th-generation tensor cores (tcgen05, TMEM accumulators): bf16, head dims up
// to 128 (64 and 128 exactly, others padded with zeros by the copies).
//
// One pass over the keys with a softmax's running maximum and sum: S = Q K^T
// for 128 rows x 128 keys into TMEM; two threads per row read it back, form
// P = 2^(s - m) in bf16 (fp32 sums) over S in TMEM, and O += P V accumulates in
// TMEM. O is rescaled only when some row's maximum grew by more than 2^8. P is
// rounded to bf16 because it is an operand of the second product; its sum is
// taken before the rounding.
//
// The gs query heads of a KV head are stacked with the tokens into the 128
// rows of a set (128 / gs tokens), so K and V are read once for all heads and a
// single token still fills gs rows. A CTA runs two sets:
//   pair:        an item's first and second 128 rows, each over all key tiles;
//   alternating: one set of rows, set 0 taking the even key tiles and set 1
//                the odd ones, folded at the end (items of few rows).
// Either way two independent softmax chains overlap with each other's products.
//
// Warps: 0-7 and 8-15 the softmax of set 0 and 1, 16 issues every MMA, 17 takes
// items off the plan, looks pages up and issues the TMA copies, 18-19 clear
// non-finite values out of V tiles that the mask cuts (below). Two threads share a
// row: each takes half of a tile's keys. They agree on the row's reference m from
// the tiles before, so neither waits for the other inside a tile (see softmax).
// Per set and key tile the MMA warp issues P V of one tile and then S of the
// next, so that the tensor cores work on the other set while this one's softmax
// runs; TMEM has no room for a second S, P and O of 128 x 128 per set.
//
// What bounds it, long prompts: the tensor cores and their hand-offs. A 32768-token
// prompt of 32/8 heads takes 5.6 to 6.0 ms, as the power limit allows: 1.47 to 1.56
// PFLOP/s, 0.77 to 0.82 of the measured bf16 burst rate and 0.86 to 0.91 of the
// sustained one; with the softmax cut down to a copy it took 5.36 ms beside 5.63.
// What the steps gave, at that size, in one session: one
// thread a row and an MMA warp issuing from a branch of one lane 7.64 ms;
// warp-uniform issue and two threads a row 6.86; waiters suspended instead of
// polling (the polls took issue slots from the softmax) 6.39; the halves agreeing a
// tile late 6.19; unmasked tiles in a copy of their own 6.04; the item's geometry in
// shared memory instead of registers 5.67. Halves of S as separate products of 64
// keys (four chains instead of two) were slower, 6.90: at N = 64 the operands'
// shared-memory reads bound the product.
// Few rows over long contexts: HBM, with the ring's 128 KB in flight per SM. A
// 16-sequence decoding step reads 645 MB in 121 to 124 us, 0.77 of the measured copy
// rate.
//
// Masked keys have P = 0, but 0 times a non-finite V is not 0: V tiles with a
// masked key (behind the diagonal, past the context, drafts another draft does
// not see, and the undefined rest of a last page) are scanned in shared memory,
// non-finite elements are zeroed and their keys noted, and a row that does see
// such a key gets the element added again at the end.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "host.h"
#include "internal.h"
#include "paged.cuh"
#include "ptx.h"
#include "tc.h"

namespace sva {
namespace {

using namespace paged;

constexpr int kKeys = 128;            // keys of a tile
constexpr int kRows = kTcRows;        // rows of a set
constexpr int kBox = 128 * 128;       // 128 rows of 64 columns, bytes
constexpr int kThreads = 640;
constexpr int kMmaWarp = 16, kLoadWarp = 17, kCleanWarp = 18;
constexpr int kItems = 4;             // item ring
constexpr int kItemReaders = 19;      // MMA, 16 softmax and 2 cleaning warps
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;   // O follows the maximum in steps of more than 2^8
// ... and never lies more than 2^kFixLog2 below a score of the tile: P stays under 2^32. A
// tile of 128 keys and the join of 640 runs then take sums of values up to 2^78 (with
// 2^64 up to 2^46).
constexpr float kFixLog2 = 32.0f;
constexpr int kMaxMasked = 4;         // masked key tiles of an item, at most 3 (see run_of)
// registers per thread of the softmax warps and of the others (the launch
// gives 96 to each of 640 threads: 512 * 104 + 128 * 64 = 640 * 96)
constexpr int kRegsSoftmax = 104, kRegsOther = 64;

// TMEM columns of set s: S (128 fp32; P, bf16 pairs, takes its place: 32 columns
// at the start of each half of 64 keys) and O (128 fp32)
__device__ constexpr uint32_t col_s(int s) { return s ? 128u : 0u; }
__device__ constexpr uint32_t col_o(int s) { return s ? 384u : 256u; }

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kBox;  // a K, V or Q tile, bytes
  static constexpr int kStages = 131072 / kTile;
  static constexpr int kSmem = 2 * kTile + kStages * kTile + 1024;
};

struct Control {
  uint64_t full[8], empty[8], vclean[8];
  uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2], o_done[2];
  uint64_t halves[2][4];  // the two warps of a set's lane quarter
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t meet, drained;
  uint32_t tmem;
  int abort;
  uint32_t nonfinite[kItems][kMaxMasked][4];  // keys of an item's masked tiles, from the last
  float mx[2][2][2][kRows];  // maxima of even and odd tiles by set and half
  float2 ml[2][2][kRows];  // maximum and sum by set and half
  unsigned long long anc[kMaxT];
  uint32_t place[kRows];   // token (high half) and head of a set's row
  Item items[kItems];
  Plan plan;
};

// What every role derives from an item.
struct Run {
  int pair;     // 1: two row sets over all tiles, 0: one over alternating tiles
  int n[2];     // key tiles of each set
  int masked;   // first key tile (of the run) with a masked key
};

struct Row {
  int tok, head;
  bool valid;  // the row is one of the item's
};

// Keys of the segment that token tok of an item sees.
__device__ __forceinline__ int keys_of(const Item& it, int tok) {
  return it.causal ? it.vis0 + tok : it.ctx;
}

__device__ __forceinline__ Run run_of(const Item& it, int tt) {
  Run r;
  r.pair = it.ntok > tt;
  if (r.pair) {
    r.n[0] = it.causal ? min(it.nk, max(0, ceil_div(max(0, it.vis0 + tt - 1), kKeys) - it.k0)) : it.nk;
    r.n[1] = it.nk;
  } else {
    r.n[0] = (it.nk + 1) / 2;
    r.n[1] = it.nk / 2;
  }
  // Tile j is cut by the mask when some row misses some of its keys: from the
  // tile that holds key vis0 on (causal), the context's end, and the drafts.
  // Those tiles span fewer than 256 + 128 keys: at most three.
  r.masked = max(0, max(0, it.causal ? it.vis0 : it.ctx) / kKeys - it.k0);
  if (it.draft) r.masked = min(r.masked, it.nk - 1);
  return r;
}

// Ring positions of the K and V tiles of an item of n key tiles, relative to
// its first: the order in which the MMA warp needs them (pair: K0 V0 K1 V1 ...;
// alternating: K0 K1 V0 K2 V1 ...).
__device__ __forceinline__ uint32_t pos_k(const Run& r, int j) {
  return r.pair ? 2 * j : (j == 0 ? 0 : 2 * j - 1);
}
__device__ __forceinline__ uint32_t pos_v(const Run& r, int j, int n) {
  return r.pair || j == n - 1 ? 2 * j + 1 : 2 * j + 2;
}

// The V tile at ring position pos, -1 where a K tile lies.
__device__ __forceinline__ int v_at(const Run& r, int pos, int n) {
  if (r.pair || pos == 2 * n - 1) return pos & 1 ? pos >> 1 : -1;
  return pos > 0 && !(pos & 1) ? (pos >> 1) - 1 : -1;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// MMA issue by a converged warp: the operands are computed by all lanes, so
// that descriptors stay in uniform registers, and one elected lane issues
// (lead != 0 there). Issued from a branch that only lane 0 takes, every MMA
// cost its thread about 100 cycles, which bounded the kernel.
__device__ __forceinline__ uint32_t elect_lead() {
  uint32_t lead;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(lead));
  return lead;
}
__device__ __forceinline__ void lead_mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void lead_mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void lead_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}

// 32 lanes x 32 (8) columns of TMEM into r[0..32) (r[0..8)).
__device__ __forceinline__ void ld32_at(uint32_t taddr, uint32_t* r) {
  tc::ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(r));
}
__device__ __forceinline__ void ld8_at(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

// The largest of 64 scores.
__device__ __forceinline__ float max64(const uint32_t (&v)[64]) {
  float mx[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    mx[c] = __uint_as_float(v[16 * c]);
#pragma unroll
    for (int i = 1; i < 15; i += 2)
      mx[c] = max3(mx[c], __uint_as_float(v[16 * c + i]), __uint_as_float(v[16 * c + i + 1]));
    mx[c] = fmaxf(mx[c], __uint_as_float(v[16 * c + 15]));
  }
  return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
}

// P = 2^(s - m) of 64 keys into 32 columns of TMEM at taddr, and its sum (even
// and odd keys apart).
__device__ __forceinline__ uint64_t exponentials(const uint32_t (&v)[64], uint32_t taddr, float m,
                                                 float scale) {
  const float nb = m == -INFINITY ? 0.f : -m;
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint64_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      e[i] = fma2(pack2(__uint_as_float(v[16 * c + 2 * i]), __uint_as_float(v[16 * c + 2 * i + 1])),
                  pack2(scale, scale), pack2(nb, nb));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = unpack2(e[i]);
      e[i] = pack2(ex2(x.x), ex2(x.y));
    }
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = unpack2(e[i]);
      p[i] = pack_bf16(x.x, x.y);
      sum[i & 1] = add2(sum[i & 1], e[i]);
    }
    tc::st8(taddr + 8 * c, p);
  }
  return add2(sum[0], sum[1]);
}

// n columns of a row's O times alpha (all products into O are complete).
__device__ __noinline__ void scale_o(uint32_t taddr, int n, float alpha) {
#pragma unroll 1
  for (int c = 0; c < n; c += 8) {
    uint32_t o[8];
    ld8_at(taddr + c, o);
    tc::wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
    tc::st8(taddr + c, o);
  }
}

// 64 keys of P in TMEM times alpha.
__device__ __noinline__ void scale_p(uint32_t taddr, float alpha) {
#pragma unroll 1
  for (int c = 0; c < 32; c += 8) {
    uint32_t p[8];
    ld8_at(taddr + c, p);
    tc::wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      p[e] = pack_bf16(__uint_as_float(p[e] << 16) * alpha, __uint_as_float(p[e] & 0xffff0000u) * alpha);
    tc::st8(taddr + c, p);
  }
}

// 32 bytes (a whole sector) to a 32-byte boundary.
__device__ __forceinline__ void store32(void* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]),
               "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

template <int N>
__device__ __forceinline__ void regs_grow() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_shrink() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Set the non-finite bf16 elements of four words to zero; true if there were any.
__device__ __forceinline__ bool clear_nonfinite(uint4* w) {
  uint32_t* x = reinterpret_cast<uint32_t*>(w);
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= ((x[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
  if (!bad) return false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = ((x[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    if (b & 0x8000u) x[i] &= 0xFFFF0000u;
    if (b & 0x80000000u) x[i] &= 0x0000FFFFu;
  }
  return true;
}

// Add the non-finite V elements that a row sees in the tiles that were
// cleared to columns [c0, c1) of its stored result (out, or the partial row).
__device__ __noinline__ void add_nonfinite(const PagedArgs& a, const Item& it,
                                           const uint32_t (*bits)[4], int nmasked, int vis,
                                           unsigned long long anc, int c0, int c1,
                                           __nv_bfloat16* out, float* part) {
  const __nv_bfloat16* pool = static_cast<const __nv_bfloat16*>(a.v_pool);
  const __nv_bfloat16* dv = static_cast<const __nv_bfloat16*>(a.draft_v);
  for (int e = 0; e < nmasked; ++e) {
    const bool drafts = it.draft && e == 0;
    const int base = (it.k0 + it.nk - 1 - e) * kKeys;
    for (int k = 0; k < kKeys; ++k) {
      if (!(bits[e][k >> 5] >> (k & 31) & 1u)) continue;
      const __nv_bfloat16* row;
      if (drafts) {
        if (k >= a.T || !(anc >> k & 1ull)) continue;
        row = dv + (((size_t)it.seq * a.T + k) * a.Hkv + it.kvh) * a.d;
      } else {
        const int key = base + k;
        if (key >= vis) continue;
        const int page = a.block_table[it.tab + key / a.blk];
        if (page < 0 || page >= a.num_pages) continue;
        row = pool + (((size_t)page * a.Hkv + it.kvh) * a.blk + key % a.blk) * a.d;
      }
      for (int c = c0; c < c1 && c < a.d; ++c) {
        const float x = __bfloat162float(row[c]);
        if (fabsf(x) < INFINITY) continue;
        if (out) out[c] = __float2bfloat16(__bfloat162float(out[c]) + x);
        else part[c] += x;
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_dk,
                    const __grid_constant__ CUtensorMap tm_dv, const __grid_constant__ PagedArgs a) {
  using C = Cfg<D>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t q_base = smem_u32(smem), ring = q_base + 2 * C::kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tt = kRows / a.gs;  // tokens of a set; an item's tile is two of them
  volatile int* abort = &sh.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 3);  // the MMAs that read it, and both cleaning warps
      mbar_init(smem_u32(&sh.vclean[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.q_full[i]), 1);
      mbar_init(smem_u32(&sh.q_empty[i]), 1);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_ready[i]), 8);
      for (int q = 0; q < 4; ++q) mbar_init(smem_u32(&sh.halves[i][q]), 2);
      mbar_init(smem_u32(&sh.o_done[i]), 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(smem_u32(&sh.item_full[i]), 1);
      mbar_init(smem_u32(&sh.item_empty[i]), kItemReaders);
    }
    mbar_init(smem_u32(&sh.meet), 16);
    mbar_init(smem_u32(&sh.drained), 1);
    sh.abort = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    prefetch_tensormap(&tm_q);
  }
  if (warp == kMmaWarp) {
    tc::alloc(smem_u32(&sh.tmem), kTmemCols);
    tc::relinquish();
  }
  if (threadIdx.x < kRows)
    sh.place[threadIdx.x] = threadIdx.x / a.gs << 16 | threadIdx.x % a.gs;
  if (a.prefix)
    for (int t = threadIdx.x; t < a.T; t += kThreads) sh.anc[t] = a.anc[t];
  pdl_wait();
  pdl_trigger();
  tc::fence_before();
  make_plan(a, &sh.plan, reinterpret_cast<int*>(smem));
  save_plan(a, &sh.plan);
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned site) {
    return mbar_wait_abortable(smem_u32(bar), parity, abort, a.status, site);
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity, unsigned site) {
    return __all_sync(0xffffffffu, wait(bar, parity, site)) != 0;
  };
  // the seq-th item of this CTA; read in place until done_item
  auto take_item = [&](uint32_t seq) {
    const int s = seq % kItems;
    return wait_all(&sh.item_full[s], (seq / kItems) & 1, 20u) &&
           sh.items[s].valid != 0;
  };
  auto done_item = [&](uint32_t seq) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.item_empty[seq % kItems]));
  };

  if (warp >= kMmaWarp) regs_shrink<kRegsOther>();
  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ items, copies
    // earlier kernels' plain stores to the pools come before this one's bulk copies
    asm volatile("fence.proxy.async.global;" ::: "memory");
    const int box_rows = min(a.blk, kKeys), ppt = kKeys / box_rows;
    const int oob = a.num_pages * a.Hkv * a.blk;  // past the pool: TMA fills zeros
    // lane -> (page of the tile, column half) of one box
    const int pg = lane / C::kHalves, half = lane % C::kHalves;
    const bool mine = lane < ppt * C::kHalves;
    uint32_t at = 0, alt = 0;
    uint32_t q_used = 0, q_phase = 0;  // bit s: slot s has been used; the phase of its release
    bool ok = true;
    Cursor cursor{};  // lane 0's
    if (lane == 0) cursor = start_cursor(a, &sh.plan);
    // decode item `seq` into the ring (the number of the item after it, asked for
    // on the way, is there by the next call)
    auto prepare = [&](uint32_t seq) {
      const int slot = seq % kItems;
      if (seq >= kItems &&
          !wait_all(&sh.item_empty[slot], ((seq / kItems) & 1) ^ 1, 1u))
        return false;
      if (lane == 0) sh.items[slot] = next_item(a, &sh.plan, &cursor);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.item_full[slot]));
      return true;
    };
    ok = prepare(0);
    for (uint32_t seq = 0; ok; ++seq) {
      const Item& it = sh.items[seq % kItems];
      if (!it.valid) break;
      const Run r = run_of(it, tt);
      // the pool row of this lane's box of key tile j
      auto lookup = [&](int j) {
        int row = oob;
        if (mine && j < it.nk && !(it.draft && j == it.nk - 1)) {
          const int key = (it.k0 + j) * kKeys + pg * box_rows;
          if (key < it.ctx) {
            const int page = __ldcg(a.block_table + it.tab + key / a.blk);
            if (page >= 0 && page < a.num_pages)
              row = (page * a.Hkv + it.kvh) * a.blk + key % a.blk;
            else if (half == 0)
              atomicOr(a.status, SV_FLAG_BAD_PAGE);
          }
        }
        return row;
      };
      auto load = [&](bool v, int j, int row) {
        const uint32_t x = at + (v ? pos_v(r, j, it.nk) : pos_k(r, j));
        const int s = x % NS;
        if (x >= NS && !wait_all(&sh.empty[s], ((x / NS) & 1) ^ 1, 2u)) return false;
        const uint32_t bar = smem_u32(&sh.full[s]), dst = ring + s * C::kTile;
        const bool drafts = it.draft && j == it.nk - 1;
        if (lane == 0) mbar_arrive_expect_tx(bar, drafts ? C::kTile / 2 : C::kTile);
        __syncwarp();
        if (drafts) {
          if (lane < C::kHalves)
            tma_load_4d(dst + lane * kBox, v ? &tm_dv : &tm_dk, 64 * lane, it.kvh, 0, it.seq, bar);
        } else if (mine) {
          tma_load_2d(dst + half * kBox + pg * box_rows * 128, v ? &tm_v : &tm_k, 64 * half, row, bar);
        }
        return true;
      };
      int row0 = lookup(0), row1 = lookup(1);
      if (it.nk > 0) {
        // Q: both slots (pair), or the slots in turn
        for (int s = 0; s < 2 && ok; ++s) {
          if (!r.pair && s != (int)(alt & 1)) continue;
          if (q_used >> s & 1) {
            if (!(ok = wait_all(&sh.q_empty[s], q_phase >> s & 1, 3u))) break;
            q_phase ^= 1u << s;
          }
          q_used |= 1u << s;
          const uint32_t bar = smem_u32(&sh.q_full[s]);
          if (lane == 0) mbar_arrive_expect_tx(bar, C::kHalves * tt * a.gs * 128);
          __syncwarp();
          if (lane < C::kHalves)
            tma_load_3d(q_base + s * C::kTile + lane * kBox, &tm_q, 64 * lane, it.head0,
                        it.tok0 + (r.pair ? s * tt : 0), bar);
        }
        if (!r.pair) ++alt;
        if (ok && !r.pair) ok = load(false, 0, row0);
        for (int j = 0; j < it.nk && ok; ++j) {
          // the next item is decoded while the ring is full of this one's tiles
          if (j == 2 && !(ok = prepare(seq + 1))) break;
          const int row2 = lookup(j + 2);
          ok = r.pair ? load(false, j, row0) : j + 1 >= it.nk || load(false, j + 1, row1);
          ok = ok && load(true, j, row0);
          row0 = row1;
          row1 = row2;
        }
        at += 2 * it.nk;
      }
      if (ok && it.nk <= 2) ok = prepare(seq + 1);
    }
    // never leave with a copy still in flight
    __syncwarp();
    if (*abort) {
      for (uint32_t s = 0; s < NS; ++s)
        for (int ph = 0; ph < 2; ++ph) mbar_wait_drain(smem_u32(&sh.full[s]), ph);
      for (int s = 0; s < 2; ++s)
        for (int ph = 0; ph < 2; ++ph) mbar_wait_drain(smem_u32(&sh.q_full[s]), ph);
    }
    if (lane == 0) leave(a);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t id_s = tc::idesc_bf16(128, kKeys, false, false);
    constexpr uint32_t id_o = tc::idesc_bf16(128, D, false, true);
    const uint64_t dq0 = tc::smem_desc(q_base, 16, 1024);
    const uint64_t dk0 = tc::smem_desc(ring, 16, 1024);
    const uint64_t dv0 = tc::smem_desc(ring, kBox, 1024);
    uint32_t at = 0, alt = 0;
    uint32_t q_phase = 0, p_phase = 0;  // bit s: the next phase of slot (set) s
    const uint32_t lead = elect_lead();
    bool ok = true;
    for (uint32_t seq = 0; ok && take_item(seq); ++seq) {
      const Item& it = sh.items[seq % kItems];
      const Run r = run_of(it, tt);
      const int nk = it.nk;
      if (nk > 0) {
        auto stage = [&](uint32_t pos) { return (at + pos) % NS; };
        auto phase = [&](uint32_t pos) { return ((at + pos) / NS) & 1; };
        auto k_wait = [&](int j) { return wait_all(&sh.full[stage(pos_k(r, j))], phase(pos_k(r, j)), 4u); };
        auto v_wait = [&](int j) {
          const uint32_t p = pos_v(r, j, nk);
          return wait_all(&sh.vclean[stage(p)], phase(p), 5u);
        };
        auto issue_s = [&](int s, int qs, int j) {
          tc::fence_after();
          const uint64_t dq = dq0 + (uint64_t)(qs * (C::kTile >> 4));
          const uint64_t dk = dk0 + (uint64_t)(stage(pos_k(r, j)) * (C::kTile >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
            lead_mma_ss(lead, tmem + col_s(s), dq + off, dk + off, id_s, kk > 0 ? 1u : 0u);
          }
          lead_commit(lead, smem_u32(&sh.s_full[s]));
        };
        // O += P V, once both halves of P (and of O, if it was rescaled) are ready
        auto issue_o = [&](int s, int j, bool first) {
          if (!wait_all(&sh.p_ready[s], p_phase >> s & 1, 6u)) return false;
          p_phase ^= 1u << s;
          tc::fence_after();
          const uint64_t dv = dv0 + (uint64_t)(stage(pos_v(r, j, nk)) * (C::kTile >> 4));
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            lead_mma_ts(lead, tmem + col_o(s), tmem + col_s(s) + (kk >> 2) * 64 + (kk & 3) * 8,
                        dv + (uint64_t)((kk * 2048) >> 4), id_o, !first || kk > 0 ? 1u : 0u);
          return true;
        };
        auto free_k = [&](int j) { lead_commit(lead, smem_u32(&sh.empty[stage(pos_k(r, j))])); };
        auto free_v = [&](int j) { lead_commit(lead, smem_u32(&sh.empty[stage(pos_v(r, j, nk))])); };
        if (r.pair) {
          ok = wait_all(&sh.q_full[0], q_phase & 1, 7u) && wait_all(&sh.q_full[1], q_phase >> 1 & 1, 7u) &&
               k_wait(0);
          q_phase ^= 3u;
          if (ok) {
            if (r.n[0] > 0) issue_s(0, 0, 0);
            issue_s(1, 1, 0);
            free_k(0);
          }
          for (int j = 0; ok && j < nk; ++j) {
            const bool more = j + 1 < nk;
            // what the two products need is waited for ahead of P
            if (!(ok = v_wait(j) && (!more || k_wait(j + 1)))) break;
            if (j < r.n[0]) {
              if (!(ok = issue_o(0, j, j == 0))) break;
              if (j + 1 < r.n[0]) {
                issue_s(0, 0, j + 1);
              } else {
                lead_commit(lead, smem_u32(&sh.o_done[0]));
              }
            }
            if (!(ok = issue_o(1, j, j == 0))) break;
            free_v(j);
            if (more) {
              issue_s(1, 1, j + 1);
              free_k(j + 1);
            } else {
              lead_commit(lead, smem_u32(&sh.o_done[1]));
            }
            if (j + 2 == nk || nk == 1) {  // the item's last S is out
              lead_commit(lead, smem_u32(&sh.q_empty[0]));
              lead_commit(lead, smem_u32(&sh.q_empty[1]));
            }
          }
        } else {
          const int qs = alt++ & 1;
          ok = wait_all(&sh.q_full[qs], q_phase >> qs & 1, 7u) && k_wait(0);
          q_phase ^= 1u << qs;
          if (ok) {
            issue_s(0, qs, 0);
            free_k(0);
            if (nk > 1 && (ok = k_wait(1))) {
              issue_s(1, qs, 1);
              free_k(1);
            }
            if (nk <= 2) lead_commit(lead, smem_u32(&sh.q_empty[qs]));
          }
          for (int j = 0; ok && j < nk; ++j) {
            const int s = j & 1;
            if (!(ok = v_wait(j) && (j + 2 >= nk || k_wait(j + 2)))) break;
            if (!(ok = issue_o(s, j, j < 2))) break;
            free_v(j);
            if (j + 2 < nk) {
              issue_s(s, qs, j + 2);
              free_k(j + 2);
              if (j + 3 == nk) lead_commit(lead, smem_u32(&sh.q_empty[qs]));
            } else {
              lead_commit(lead, smem_u32(&sh.o_done[s]));
            }
          }
        }
      }
      at += 2 * nk;
      done_item(seq);
    }
    lead_commit(lead, smem_u32(&sh.drained));  // TMEM is given back after every MMA
    mbar_wait_drain(smem_u32(&sh.drained), 0);
    __syncwarp();
  } else if (warp >= kCleanWarp) {
    // ------------------------------------------------------------ V tiles
    const int w = warp - kCleanWarp;  // keys [64 w, 64 w + 64)
    uint32_t at = 0;
    bool ok = true;
    for (uint32_t seq = 0; ok && take_item(seq); ++seq) {
      const Item& it = sh.items[seq % kItems];
      const Run r = run_of(it, tt);
      const int nk = it.nk;
      // every ring position in order: a V tile that needs it is cleared, and the
      // stage's barrier advances once per use whatever the stage holds
      for (int pos = 0; pos < 2 * nk; ++pos) {
        const uint32_t x = at + pos;
        const int s = x % NS;
        if (!(ok = wait_all(&sh.full[s], (x / NS) & 1, 8u))) break;
        const int j = v_at(r, pos, nk);
        if (j >= r.masked) {
          uint8_t* v = smem + 2 * C::kTile + s * C::kTile;
          uint32_t bits[2] = {0, 0};
#pragma unroll 4
          for (int i = 0; i < 16 * C::kHalves; ++i) {
            // 16-byte chunks of a 128-byte row of 64 columns; the swizzle
            // moves chunks within their row only
            const int row = 64 * w + (i & 15) * 4 + (lane >> 3);
            uint4* p = reinterpret_cast<uint4*>(v + (i >> 4) * kBox + row * 128 + (lane & 7) * 16);
            uint4 x4 = *p;
            if (clear_nonfinite(&x4)) {
              *p = x4;
              bits[(row >> 5) & 1] |= 1u << (row & 31);
            }
          }
          bits[0] = __reduce_or_sync(0xffffffffu, bits[0]);
          bits[1] = __reduce_or_sync(0xffffffffu, bits[1]);
          if (bits[0] | bits[1]) fence_proxy_async_shared();
          if (lane < 2)
            sh.nonfinite[seq % kItems][min(kMaxMasked - 1, nk - 1 - j)][2 * w + lane] = bits[lane];
        }
        __syncwarp();
        // The stage is not filled again before this warp has seen it: a warp that
        // came late to a K tile (which nothing else makes it hurry for) could
        // otherwise find its barrier two phases on, and wait for ever.
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh.vclean[s]));
          mbar_arrive(smem_u32(&sh.empty[s]));
        }
      }
      at += 2 * nk;
      done_item(seq);
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_grow<kRegsSoftmax>();
    const int X = warp >> 3, H = warp >> 2 & 1, q4 = warp & 3, r = 32 * q4 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q4) << 16);
    const uint32_t tS = lane_base + col_s(X) + 64 * H;
    const uint32_t tO = lane_base + col_o(X);
    uint32_t s_uses = 0, o_uses = 0, h_uses = 0, meets = 0;
    bool ok = true;
    // all softmax warps meet
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.meet));
      return wait_all(&sh.meet, meets++ & 1, 9u);
    };
    // the two warps of this set's rows meet
    auto half_arrive = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.halves[X][q4]));
    };
    auto half_wait = [&]() {
      return wait_all(&sh.halves[X][q4], h_uses++ & 1, 13u);
    };
    auto meet_half = [&]() {
      half_arrive();
      return half_wait();
    };
    // token (of the item) and head (of the group) of row r of set s
    auto row_of = [&](const Item& it, const Run& run, int s, int r) {
      const uint32_t place = sh.place[r];
      Row row{(int)(place >> 16), (int)(place & 0xffff), false};
      row.valid = row.tok < tt;
      if (run.pair && s) row.tok += tt;
      row.valid = row.valid && row.tok < it.ntok && row.head < it.heads;
      return row;
    };
    for (uint32_t seq = 0; ok && take_item(seq); ++seq) {
      const Item& it = sh.items[seq % kItems];
      // Little of an item is kept in registers over its key tiles (the inner
      // loop needs them all): what the mask and the results need is read again
      // from shared memory.
      bool mine_valid, live;  // a warp without rows only keeps step
      int kt, kt_end, stride, plain;
      {
        const Run run = run_of(it, tt);
        mine_valid = row_of(it, run, X, r).valid;
        live = __any_sync(0xffffffffu, mine_valid);
        kt = run.pair ? 0 : X;
        kt_end = run.pair ? run.n[X] : it.nk;
        stride = run.pair ? 1 : 2;
        // key tiles before `plain` show all their keys to all rows of the set
        const int least = keys_of(it, run.pair && X ? tt : 0) - (it.k0 * kKeys + 64 * H);
        plain = least < 64 ? 0 : (least + 64) / kKeys;
        if (it.draft) plain = min(plain, it.nk - 1);
      }
      const bool empty = kt >= kt_end;
      float m_run = -INFINITY, l_run = 0.f, mine = -INFINITY;
      // Move the row's reference to m or up to one above it, by a whole number: alpha, by
      // which its sum, its O and, where they are there already, its weights are
      // multiplied, is a power of two, and weights in bf16 are not rounded a second time.
      // (The first reference is the maximum itself: a single key has the weight 1.)
      auto move_ref = [&](float m) {
        const bool first = m_run == -INFINITY;  // nothing is summed yet
        const float step = ceilf(m - m_run), alpha = first ? (m == -INFINITY ? 1.f : 0.f) : ex2(-step);
        l_run *= alpha;
        m_run = first ? m : m_run + step;
        return alpha;
      };
      // This half's maximum of a row that is not one of the item's is -inf: such a row
      // (another sequence's queries, padding, or what the slot held before) must not
      // move the references of the rows beside it, whose rounding goes with them.
      auto top_score = [&](const uint32_t(&v)[64]) {
        return mine_valid ? max64(v) * a.scale_log2 : -INFINITY;
      };
      // The two threads of a row agree on its reference without waiting for each
      // other: exponentials take what both knew of the tiles before (their maxima
      // lie in sh.mx), so P may exceed 1, but what it exceeds by only moves
      // exponents. When one of them finds a maximum more than 2^kFixLog2 above the
      // reference, its warp moves it at once for both halves; the other half
      // recognises that in the next tile, by the same comparison.
      auto catch_up = [&](float other) {  // the other half's maximum of the last tile
        if (__any_sync(0xffffffffu, other > m_run + kFixLog2)) move_ref(fmaxf(m_run, fmaxf(mine, other)));
      };
      // One key tile of the set. General: the set's first tile of the item and those
      // with a masked key; the others run a copy without that code.
      auto softmax_tile = [&](bool start, auto tag) {
        constexpr bool general = decltype(tag)::value;
        const uint32_t odd = s_uses & 1;
        if (!wait_all(&sh.s_full[X], s_uses++ & 1, 10u)) return false;
        if (live) {
          tc::fence_after();
          const float other = general && start ? -INFINITY : sh.mx[odd ^ 1][X][H ^ 1][r];
          uint32_t v[64];
          ld32_at(tS, v);  // (nothing may touch v before the wait)
          ld32_at(tS + 32, v + 32);
          tc::wait_ld();
          // O follows the maximum in steps of more than 2^kRescaleLog2, each half its
          // columns: S of this tile was issued behind the P V of the last
          if (__any_sync(0xffffffffu, fmaxf(mine, other) > m_run + kRescaleLog2) && !(general && start)) {
            catch_up(other);
            const float both = fmaxf(mine, other);
            if (__any_sync(0xffffffffu, both > m_run + kRescaleLog2))
              scale_o(tO + D / 2 * H, D / 2, move_ref(fmaxf(m_run, both)));
          }
          if (general && kt >= plain) {
            uint32_t keep[2];  // keys of this half that the row sees
            const Row row = row_of(it, run_of(it, tt), X, r);
            if (it.draft && kt == it.nk - 1) {  // drafts 0..63: all in the first half
              const unsigned long long see = row.valid && H == 0 ? sh.anc[it.draft0 + row.tok] : 0ull;
              keep[0] = (uint32_t)see;
              keep[1] = (uint32_t)(see >> 32);
            } else {
              const int lim = keys_of(it, row.tok) - (it.k0 + kt) * kKeys - 64 * H;
              keep[0] = lim >= 32 ? 0xffffffffu : lim <= 0 ? 0u : (1u << lim) - 1u;
              keep[1] = lim >= 64 ? 0xffffffffu : lim <= 32 ? 0u : (1u << (lim - 32)) - 1u;
            }
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (!(keep[i >> 5] >> (i & 31) & 1u)) v[i] = 0xff800000u;  // -inf
          }
          if (general && start) {
            mine = top_score(v);
            sh.mx[odd][X][H][r] = mine;
            if (!meet_half()) return false;
            m_run = fmaxf(mine, sh.mx[odd][X][H ^ 1][r]);
          }
          uint64_t sum = exponentials(v, tS, m_run, a.scale_log2);
          if (!(general && start)) {
            mine = top_score(v);
            sh.mx[odd][X][H][r] = mine;
            const bool fix = __any_sync(0xffffffffu, mine > m_run + kFixLog2);
            tc::wait_st();
            tc::fence_before();
            half_arrive();  // P is written; or, on a fix, it will be
            ++h_uses;
            if (fix) {
              --h_uses;
              if (!half_wait()) return false;
              tc::fence_after();
              const float now = sh.mx[odd][X][H ^ 1][r];
              const bool alone = !__any_sync(0xffffffffu, now > m_run + kFixLog2);
              const float alpha = move_ref(fmaxf(m_run, fmaxf(mine, now)));
              // alone: the other half's P is written, against the old reference
              scale_o(tO + (alone ? 0 : D / 2 * H), alone ? D : D / 2, alpha);
              if (alone) scale_p(lane_base + col_s(X) + 64 * (H ^ 1), alpha);
              sum = exponentials(v, tS, m_run, a.scale_log2);
            }
          }
          const float2 s2 = unpack2(sum);
          l_run += s2.x + s2.y;
          tc::wait_st();
          tc::fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_ready[X]));
        return true;
      };
      for (bool start = true; ok && kt < kt_end; kt += stride, start = false)
        ok = start || kt >= plain ? softmax_tile(start, std::true_type{})
                                  : softmax_tile(false, std::false_type{});
      if (!ok) break;
      // ---------------------------------------------------------- results
      const Run run = run_of(it, tt);
      const Row row = row_of(it, run, X, r);
      if (!empty) {
        if (!(ok = wait_all(&sh.o_done[X], o_uses++ & 1, 11u))) break;
        tc::fence_after();
        if (live) catch_up(sh.mx[(s_uses & 1) ^ 1][X][H ^ 1][r]);
      }
      // the row's maximum and sum over both halves (and, alternating, both sets)
      float w[2] = {X ? 0.f : 1.f, X ? 1.f : 0.f}, m_out = m_run, l_out = l_run;
      sh.ml[X][H][r] = make_float2(m_run, l_run);
      if (run.pair) {
        if (!(ok = meet_half())) break;
        l_out += sh.ml[X][H ^ 1][r].y;
      } else {
        if (!(ok = meet())) break;
        tc::fence_after();
        const float2 m0 = sh.ml[0][0][r], m1 = sh.ml[1][0][r];
        m_out = fmaxf(m0.x, m1.x);
        w[0] = m0.x == -INFINITY ? 0.f : exp2f(m0.x - m_out);
        w[1] = m1.x == -INFINITY ? 0.f : exp2f(m1.x - m_out);
        l_out = w[0] * (m0.y + sh.ml[0][1][r].y) + w[1] * (m1.y + sh.ml[1][1][r].y);
      }
      if (live) {
        // non-finite V in a cleared tile
        const int nmasked = min(kMaxMasked, max(0, it.nk - run.masked));
        const uint32_t(*nf)[4] = sh.nonfinite[seq % kItems];
        uint32_t any_nf = 0;
        for (int e = 0; e < nmasked; ++e) any_nf |= nf[e][0] | nf[e][1] | nf[e][2] | nf[e][3];
        const float inv = l_out == 0.f ? 0.f : 1.0f / l_out;
        const bool use0 = (run.pair ? X == 0 : true) && run.n[0] > 0;
        const bool use1 = (run.pair ? X == 1 : true) && run.n[1] > 0;
        const size_t prow = (size_t)max(it.part, 0) + row.tok * a.gs + row.head;
        // 16 columns at a time: this thread's share of the row's D is its half
        // (pair), or a quarter of both sets' sums (alternating)
        const int c0 = run.pair ? D / 2 * H : D / 4 * (2 * X + H), c1 = c0 + (run.pair ? D / 2 : D / 4);
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          __syncwarp();
          float f[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) f[e] = 0.f;
          uint32_t o[16];
          if (use0) {
            tc::ld16(lane_base + col_o(0) + c, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = w[0] != 0.f ? w[0] * __uint_as_float(o[e]) : 0.f;
          }
          if (use1) {
            tc::ld16(lane_base + col_o(1) + c, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] += w[1] != 0.f ? w[1] * __uint_as_float(o[e]) : 0.f;
          }
          if (!row.valid) continue;
          uint32_t x[16];
          if (it.part < 0) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) +
                                 ((size_t)(it.tok0 + row.tok) * a.Hq + it.head0 + row.head) * a.d + c;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = pack_bf16(f[2 * e] * inv, f[2 * e + 1] * inv);
            if (a.out_wide) {  // d is a multiple of 16
              if (c < a.d) store32(dst, x);
            } else {
              if (c < a.d) *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
              if (c + 8 < a.d) *reinterpret_cast<uint4*>(dst + 8) = make_uint4(x[4], x[5], x[6], x[7]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(f[e]);
            float* dst = a.part_o + prow * a.d + c;
            if (c < a.d) store32(dst, x);
            if (c + 8 < a.d) store32(dst + 8, x + 8);
          }
        }
        if (any_nf && row.valid)
          add_nonfinite(a, it, nf, nmasked, keys_of(it, row.tok),
                        it.draft ? sh.anc[it.draft0 + row.tok] : 0ull, c0, c1,
                        it.part < 0 ? static_cast<__nv_bfloat16*>(a.out) +
                                          ((size_t)(it.tok0 + row.tok) * a.Hq + it.head0 + row.head) * a.d
                                    : nullptr,
                        a.part_o + prow * a.d);
        if (row.valid && it.part >= 0 && H == 0 && (run.pair || X == 0)) a.part_ml[prow] = make_float2(m_out, l_out);
      }
      tc::fence_before();  // O is read: the next item's products may overwrite it
      // both halves (pair) or all warps (alternating) have read sums and O
      if (!(ok = run.pair ? meet_half() : meet())) break;
      done_item(seq);
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, kTmemCols);
  }
}

bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const auto enc = get_encode();
  if (!enc) return false;
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box,
             step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_cfg(PagedArgs a, const CUtensorMap* m, cudaStream_t st) {
  const int dev = current_device();
  static std::atomic<int> ready[kMaxDevices];
  if (!ready[dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(
        paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    ready[dev].store(1);
  }
  a.ctas = std::min(sm_count(), kMaxTcCtas);
  const cudaError_t e = launch_pdl(paged_tc_kernel<D>, dim3(a.ctas), dim3(kThreads), Cfg<D>::kSmem, st,
                                   m[0], m[1], m[2], m[3], m[4], a);
  return e == cudaSuccess ? launch_paged_merge(a, SV_BF16, st) : e;
}

}  // namespace

bool paged_tc_applies(const PagedArgs& a, int dtype) {
  // a key tile is whole pages, or part of one; boxes of 8 rows or more keep
  // the swizzle's pattern
  return dtype == SV_BF16 && a.d <= 128 && a.blk >= 8 &&
         (a.blk % kKeys == 0 || kKeys % a.blk == 0);
}

cudaError_t launch_paged_tc(PagedArgs a, cudaStream_t st) {
  paged_heads(&a, kRows);
  a.min_run = 2;
  a.one_set = kRows / a.gs;
  a.tile = 2 * a.one_set;
  a.key_shift = 7;
  a.item_cost = 4;
  a.out_wide = a.d % 16 == 0 && aligned(a.out, 32);
  CUtensorMap m[5];
  const cuuint64_t d = a.d, hd = (cuuint64_t)a.Hkv * a.d;
  {
    const cuuint64_t dims[3] = {d, (cuuint64_t)a.Hq, (cuuint64_t)a.n_rows};
    const cuuint64_t strides[2] = {d * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.gs, (cuuint32_t)(kRows / a.gs)};
    if (!encode(&m[2], a.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  m[0] = m[1] = m[3] = m[4] = m[2];  // (a map that no copy uses has to be one all the same)
  if (a.num_pages > 0) {
    const cuuint64_t dims[2] = {d, (cuuint64_t)a.num_pages * a.Hkv * a.blk}, strides[1] = {d * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)std::min(a.blk, kKeys)};
    if (!encode(&m[0], a.k_pool, 2, dims, strides, box) || !encode(&m[1], a.v_pool, 2, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  if (a.prefix) {
    const cuuint64_t dims[4] = {d, (cuuint64_t)a.Hkv, (cuuint64_t)a.T, (cuuint64_t)a.B};
    const cuuint64_t strides[3] = {d * 2, hd * 2, hd * 2 * a.T};
    const cuuint32_t box[4] = {64, 1, 64, 1};
    if (!encode(&m[3], a.draft_k, 4, dims, strides, box) || !encode(&m[4], a.draft_v, 4, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  return a.d <= 64 ? launch_cfg<64>(a, m, st) : launch_cfg<128>(a, m, st);
}

}  // namespace sva
