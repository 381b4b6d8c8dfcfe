// Attention over a 4-bit cache on the 5th-generation tensor cores (tcgen05, TMEM):
// bf16 queries, head dims up to 128, pages of any multiple of 16 tokens.
//
// Rows are few (T drafts x G heads of a KV head) and the cache is long, so the
// products are taken transposed: S^T = K Q^T with the 128 keys of a tile as the
// M rows and up to 64 rows as the N columns, O^T += V^T P^T with the head's dims as M.
// K goes from the ring of pages through a thread's registers, where codes become halves,
// into TMEM and is the A operand from there; V goes into shared memory as halves, a key a
// row. (V^T in TMEM as well: 190 us instead of 188 in the case below, as an MMA of 128 x N x 16
// takes 65 cycles with A in TMEM, for any N up to 128, and 47 with A in shared memory, N up
// to 64.)
// Code times scale has at most six significant bits and is exact in f16. Q is
// scaled by a power of two per row so that its largest element lies in [2^14, 2^15):
// exact for elements down to 2^-24 of it, below within 2^-39 of it (half of f16's smallest
// step); factor and exponents go into the softmax's scale.
//
// Twenty warps: four for K and four for V (codes to halves), eight of softmax, and four that
// copy K, copy V and lay out Q of later segments, issue the MMAs of the scores, issue those of
// the outputs. Even and odd tiles are two streams with a softmax warpgroup, references, sums
// and an O of their own, joined with the segments: a tile's chain from scores to weights is
// as long as its products.
// A softmax thread has 4 keys and every fourth pair of columns. It does not look for
// a tile's maxima: references stand until some row's weights, summed over a thread's
// 4 keys, pass 2^15, which the warps tell each other by a vote; only then (and in a
// segment's first tile) maxima are taken across lanes and O is rescaled.
// Weights are held 2^7 times their size, so that f16's range covers 2^-31 .. 2^8 of the
// reference. As an operand of the products a weight has f16's 11 bits (2^-11, an eighth of the
// output's own rounding to bf16), which is what lets V be halves; its sum is fp32's.
//
// What bounds it. Four sequences of 131072 tokens, 8 heads of 128, 32 rows: 154 us, 3.9 TB/s
// of pages, 0.58 of the copy rate. A tile of 128 keys takes about 1400 cycles, of which the MMA
// pipe needs 900 (8 x 65 + 8 x 47), shared memory about 900 (bytes in, V as halves in
// and out, P) and the issue slots about 900. (When it was 161 us: without the products 145,
// without the conversions 129, without softmax 147, without any of them 108.) More
// warps for K and V gained nothing (768 threads 166 us, 896 171: fewer registers each). Two MMA
// warps instead of one: 197 instead of 216; softmax with a key a thread and factors in shared
// memory: 188; pages past L2's reach evict-first 164, before 170.
// Short calls: everything that runs once is fetched from a cold instruction cache at 12 to 30
// cycles an instruction, so it is rolled, short and split among the warps. Eight
// sequences of 64 selected blocks, trees of 16, 128 rows a head: 34 us, of which a CTA spends
// 10 until its first scores (lengths, pages and first copies one after the other), 2 a tile and 2 at a
// segment's end; 63 when one warp laid out Q, all threads tracked all references, and the
// weights of a tile waited in registers that spilled.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "host.h"
#include "kv4.cuh"
#include "tc.h"
#include "tc_issue.cuh"

namespace sva {
namespace {

using namespace kv4;

// Key tiles' time that beginning a pair takes. 3, 5 and 8 of them: 16 ragged sequences of 1 to
// 32768 tokens 59, 55 and 56 us (8 heads of 128, one token), 37, 34 and 34 (4 heads of 64), 117,
// 101 and 97 (4 heads of 128, 128 rows); 64 sequences of 50 to 3000 36, 37 and 39 (one token) and
// 129, 119 and 119 (128 rows).
constexpr int kPairCost = 5;
static_assert(kPairCost <= kMaxPairCost, "the calls' limits count this many");
constexpr int kKeys = 128, kPieces = kKeys / kPiece;
// Rings. Copies run at most kMaxStages tiles ahead of V, V two ahead of its products, so the
// infos of 11 tiles, and of as many segments, are in use at most. Q, with its factors, runs
// at most two segments ahead of the scores and those two ahead of the weights.
constexpr int kInfo = 16, kSegs = 16, kF = 8;
constexpr int kMaxStages = 8;
constexpr int kThreads = 640;
constexpr int kSoftmaxWarp = 8, kKLoadWarp = 16, kVLoadWarp = 17, kScoreWarp = 18, kOutWarp = 19;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 128, kColK = 256;  // two of at most 64 columns each
constexpr float kLift = 7.f;    // weights are 2^kLift times their size ...
constexpr float kTop = 32768.f; // ... and below this, so that f16 (65504) holds them
// References move when a row's weights of a thread's 4 keys sum up to more than kTop: one
// of them is above 2^13 then, its score more than 6 (log2) above its reference. kSlack lies
// below that, so that the move always ends the cause. (Rows vote one by one: in a sum over
// several, a row that is not finite would hide those that have to move.)
constexpr float kSlack = 1.9f;

// What the loading warp tells the others of a tile: tokens that count of each piece
// (a byte each), its place in the segment, and the segment.
struct alignas(16) TileInfo {
  uint64_t valid;
  uint32_t flags, seg;
};
constexpr uint32_t kBegin = 1, kEnd = 2;          // the segment's first and last tile
constexpr uint32_t kFirst = 4, kLast = 8;         // ... the stream's
constexpr uint32_t kOnly = 16;                    // the other stream has none
constexpr uint64_t kAllValid = 0x1010101010101010ull;

struct SegInfo {
  int slot, rows;
};

struct Control {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t s_ready[2], k_empty[2], s_full[2];  // K (and room for S) is there; S = K Q^T is done
  uint64_t o_ready[2], pv_done[2], o_empty[2]; // V and P are there; O += V P is done; O has been read
  uint64_t q_first, q_full[2], q_empty[2], drained[2], meet[2];
  uint32_t tmem;
  int abort;
  uint32_t over[2][2];                    // by warpgroup and turn: 1 + the tile whose references move
  TileInfo info[kInfo];
  SegInfo seg[kSegs];
  alignas(16) float f[kF][kTc4Rows];   // factor of a row's scores
  // both streams' columns: minus (reference - kLift), what O and the sums shrink by as it
  // moves, and by warp of a warpgroup the maxima and sums
  alignas(16) float nm[2 * kTc4Rows], corr[2 * kTc4Rows], mx[4][2 * kTc4Rows], sum[4][2 * kTc4Rows];
  int tiles;                              // of the CTA's share
  uint32_t copied[2];                     // ... of which K's and V's copies were issued, once both warps are done
  Segment first;                          // its first
  Line line;
};

template <int N>
struct Cfg {
  static constexpr int kQBytes = 2 * N * 128;       // two blocks of 64 dims
  static constexpr int kPBytes = kKeys * 128;       // a key's 64 columns
  static constexpr int kVBytes = 2 * kKeys * 128;   // two blocks of 64 dims
  static constexpr int kFixed = 2 * (kQBytes + kPBytes + kVBytes) + (int)sizeof(Control);
};

__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
// Bytes at .. at + 3 of a row whose last index is `last`.
__device__ __forceinline__ uint32_t lds8x4(uint32_t row, int at, int last) {
  uint32_t r = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) r |= lds8(row + min(at + j, last)) << (8 * j);
  return r;
}
__device__ __forceinline__ uint32_t first_bytes(int n) {  // a mask of the first n bytes of a word
  return n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}
template <int H>
__device__ __forceinline__ uint32_t mul_by_half(uint32_t x, uint32_t s) {
  const __half2 ss = *reinterpret_cast<const __half2*>(&s);
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x), H ? __high2half2(ss) : __low2half2(ss));
  return *reinterpret_cast<const uint32_t*>(&y);
}
// The dim of a head that row m of V^T in shared memory holds.
__device__ __forceinline__ int dim_of(int m) {
  const int g = m >> 4;
  return g * 16 + (m >> 3 & 1) * 4 + (((m >> 1) + g) & 3) + (m & 1) * 8;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Instruction descriptor of kind::f16 with f16 operands and fp32 sums, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// 32 lanes x 8 columns of TMEM.
__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
// 16 lanes x 8 N columns of TMEM into 4 N registers: of eight columns, a lane has those at
// 2 (lane % 4) and behind it in row lane / 4, and the same in row lane / 4 + 8.
template <int N>
__device__ __forceinline__ void ld_16x256b(uint32_t taddr, uint32_t* r) {
  if constexpr (N == 1) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
  } else if constexpr (N == 2) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  } else {
    static_assert(N == 4, "columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
}
__device__ __forceinline__ void st_16x256b_x1(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
// bulk_load under an L2 policy.
__device__ __forceinline__ void bulk_load_once(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}
// Four 8 x 8 blocks of halves, a row of block b at the address in lane 8 b + row.
__device__ __forceinline__ void put(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2),
               "r"(r3)
               : "memory");
}

// A wait that may suspend the warp for up to a millisecond: without the hint it comes back
// after a fraction of a tile, and the polls of the twenty warps took issue slots from those
// that had work.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
// The rest of a wait, out of line (a wait's clock and limit inline would fill the
// instruction cache).
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, unsigned* status,
                                     unsigned site) {
  return __all_sync(0xffffffffu, mbar_wait_abortable(bar, parity, abort, status, site));
}

// The first segment with key tiles at position x of the line or behind it (without: the
// CTA's share ends first).
__device__ __noinline__ Segment segment_from(const Attend4Args& a, const Line& line, int x, int end) {
  Segment s;
  s.tiles = 0;
  while (x < end && s.tiles == 0) {
    s = segment_at(a, line, x, end, blockIdx.x);
    x = s.next;
  }
  return s;
}

// Q of a segment into shared memory as halves, K-major with the 128-byte swizzle, and the
// factors of its rows' scores: warp `part` of `parts`, a row by 4 lanes, 32 dims each, the next
// row's loads under way meanwhile. (It takes its arguments by value: read through a
// reference to the kernel's parameters, 64 rows took a warp 39000 cycles.)
struct QRows {
  const __nv_bfloat16* q;  // the (sequence, head)'s first row
  float scale;
  int row0, rows, d, G, g_shift, skip;  // skip: from a token's last row of the head to the next token's first
};
__device__ __forceinline__ QRows q_rows(const Attend4Args& a, const Segment& s) {
  QRows x;
  x.q = static_cast<const __nv_bfloat16*>(a.q) + row_at(a, s.b, s.h, 0) * a.d;
  x.scale = a.scale_log2 * exp2i(head_exp(a.k_exp, s.h));
  x.row0 = s.rt * a.rows;
  x.rows = min(a.rows, a.T * a.G - x.row0);
  x.d = a.d, x.G = a.G, x.g_shift = a.g_shift, x.skip = a.Hq - a.G;
  return x;
}
__device__ __noinline__ void lay_out_q(const QRows x, int n, uint32_t to, float* f, int part, int parts) {
  const int lane = threadIdx.x & 31, c = lane & 3;
  auto load = [&](int r, uint4 (&w)[4]) {
    const int at = x.row0 + r, t = x.g_shift >= 0 ? at >> x.g_shift : quotient(at, x.G);
    const __nv_bfloat16* from = x.q + (long long)(at + t * x.skip) * x.d;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = make_uint4(0, 0, 0, 0);
      if (r < x.rows && 8 * (c + 4 * k) < x.d) w[k] = __ldcg(reinterpret_cast<const uint4*>(from) + c + 4 * k);
    }
  };
  int r = part * 8 + (lane >> 2);
  uint4 next[4];
  load(r, next);
#pragma unroll 1
  for (; part * 8 < n; part += parts, r += 8 * parts) {
    uint32_t w[16], m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[4 * k] = next[k].x, w[4 * k + 1] = next[k].y, w[4 * k + 2] = next[k].z, w[4 * k + 3] = next[k].w;
    }
    if ((part + parts) * 8 < n) load(r + 8 * parts, next);
    // the largest element's bits (of positive floats they compare as integers; a NaN's are
    // the largest and leave the row as it is)
#pragma unroll
    for (int i = 0; i < 16; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    uint32_t top = max(m & 0xffffu, m >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the power of two that takes it into [2^14, 2^15)
    const int e = (int)(top >> 7), up = e == 0 || e == 255 ? 0 : min(100, 127 + 14 - e);
    const float k2 = exp2i(up);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_f16(__uint_as_float(w[i] << 16) * k2, __uint_as_float(w[i] & 0xffff0000u) * k2);
    const uint32_t row = to + r * 128, chunk = (uint32_t)(c ^ (r & 7)) << 4;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      sts128(row + (k >> 1) * (n * 128) + (chunk ^ (k & 1) << 6), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    // (the factor stays finite, as scores of zero have to stay zero: where it would not, others
    // are beyond 2^90 either way)
    if (c == 0) f[r] = fminf(x.scale * exp2i(-up), FLT_MAX);
  }
  fence_proxy_async_shared();
  __syncwarp();
}

// DG: groups of 16 dims (8: d = 128), 0: any number up to 8.
template <int N, int DG>
__global__ void __launch_bounds__(kThreads, 1) attend4_tc_kernel(const __grid_constant__ Attend4Args a, int stages) {
  using C = Cfg<N>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_base = base, p_base = q_base + 2 * C::kQBytes, v_base = p_base + 2 * C::kPBytes;
  const uint32_t ctl = v_base + 2 * C::kVBytes;
  Control& sh = *reinterpret_cast<Control*>(smem_raw + (ctl - smem_u32(smem_raw)));
  const uint32_t ring = ctl + (uint32_t)((sizeof(Control) + 127) / 128 * 128);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = DG ? DG : a.d / 16;
  const uint32_t pb = (uint32_t)piece_bytes(groups * 16), side = kPieces * pb, stage_bytes = 2 * side;

  if (warp == kScoreWarp) {
    tc::alloc(smem_u32(&sh.tmem), kTmemCols);
    tc::relinquish();
  }
  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 2);
      mbar_init(smem_u32(&sh.empty[i]), 8);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_ready[i]), 8);
      mbar_init(smem_u32(&sh.k_empty[i]), 1);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.o_ready[i]), 8);
      mbar_init(smem_u32(&sh.pv_done[i]), 1);
      mbar_init(smem_u32(&sh.o_empty[i]), 4);
      mbar_init(smem_u32(&sh.q_full[i]), 2);
      mbar_init(smem_u32(&sh.drained[i]), 1);
      mbar_init(smem_u32(&sh.q_empty[i]), 1);
      mbar_init(smem_u32(&sh.meet[i]), 4);
      sh.over[i][0] = sh.over[i][1] = 0;
    }
    mbar_init(smem_u32(&sh.q_first), kKLoadWarp);
    sh.abort = 0;
    fence_barrier_init();
  }
  pdl_wait();
  pdl_trigger();
  if (warp == kOutWarp) {
    if (make_line(a, &sh.line)) atomicOr(a.status, SV_FLAG_BAD_LENGTH);
    __syncwarp();
    const int x = sh.line.begin(blockIdx.x), end = sh.line.begin(blockIdx.x + 1);
    int tiles = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) tiles = tiles_before(a, sh.line, i ? end : x) - tiles;
    if (lane == 0) sh.tiles = tiles;
    const Segment s = segment_from(a, sh.line, x, end);
    if (lane == 0) sh.first = s;
  } else if (warp == kKLoadWarp || warp == kVLoadWarp) {
    // earlier kernels' plain stores to the pools come before this one's bulk copies
    asm volatile("fence.proxy.async.global;" ::: "memory");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t tiles = (uint32_t)sh.tiles;
  auto wait = [&](uint64_t& bar, uint32_t parity, unsigned site) {
    const uint32_t addr = smem_u32(&bar);
    return __all_sync(0xffffffffu, try_wait_long(addr, parity & 1u)) ||
           wait_on(addr, parity & 1u, &sh.abort, a.status, site);
  };
  auto arrive = [&](uint64_t& bar) {  // once for the warp
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar));
  };

  if (warp < kKLoadWarp && tiles) {
    // the first segment's Q, which everybody waits for (later ones: the loading warps, ahead)
    lay_out_q(q_rows(a, sh.first), N, q_base, sh.f[0], warp, kKLoadWarp);
    arrive(sh.q_first);
  }
  if (warp < 4) {
    // ------------------------------------------------------------ K: lane = key
    const uint32_t piece = (uint32_t)tid / kPiece, tok = (uint32_t)tid % kPiece;
    const uint32_t tlane = (uint32_t)(warp * 32) << 16;
    for (uint32_t i = 0, st = 0, ph = 0; i < tiles; ++i) {
      if (!wait(sh.full[st], ph, 1u)) break;
      if (!wait(sh.k_empty[i & 1], (i >> 1) ^ 1u, 2u)) break;
      tc::fence_after();
      const uint32_t at = ring + st * stage_bytes + piece * pb;
      const uint32_t codes = at + tok * 8, scales = at + groups * 128 + tok * groups;
      const uint32_t to = tmem + tlane + kColK + (i & 1) * 64;
#pragma unroll 1
      for (int g = 0; g < groups; g += 4) {  // (behind the last group: columns that no product reads)
        uint32_t r[32];
        uint2 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = lds64(codes + (DG ? g + j : min(g + j, groups - 1)) * 128);
        uint32_t s01, s23;
        e4m3x4_to_f16(DG ? lds32(scales + g) : lds8x4(scales, g, groups - 1), s01, s23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e2m1x8_to_f16(w[j].x, r + 8 * j);
          e2m1x8_to_f16(w[j].y, r + 8 * j + 4);
        }
        scale_f16x2<0>(r, s01);
        scale_f16x2<1>(r + 8, s01);
        scale_f16x2<0>(r + 16, s23);
        scale_f16x2<1>(r + 24, s23);
        tc::st32(to + g * 8, r);
      }
      arrive(sh.empty[st]);
      tc::wait_st();
      tc::fence_before();
      arrive(sh.s_ready[i & 1]);
      if (++st == (uint32_t)stages) st = 0, ph ^= 1u;
    }
  } else if (warp < kSoftmaxWarp) {
    // ------------------------------------------------------------ V: halves into shared memory
    const int w = warp & 3;
    for (uint32_t i = 0, st = 0, ph = 0; i < tiles; ++i) {
      if (!wait(sh.full[st], ph, 3u)) break;
      if (!wait(sh.pv_done[i & 1], (i >> 1) ^ 1u, 4u)) break;
      tc::fence_after();
      const uint64_t valid = sh.info[i % kInfo].valid;
      const uint32_t from = ring + st * stage_bytes + side;
      // A thread has 4 code rows (8 dims: rows c .. c + 3 hold them and those 8 behind) of a
      // piece's 16 tokens: row = key, 128 bytes of 64 dims, 128-byte swizzle. The rows are taken
      // in an order that differs from group to group, so that the loads of 8 lanes fall
      // into different banks; dim_of() undoes it.
      const uint32_t cb = lane & 1, gq = lane >> 1 & 3, half = lane >> 3 & 1, p = 2 * w + (lane >> 4), g = half * 4 + gq;
      if (DG || (int)g < groups) {
        const uint32_t at = from + p * pb;
        uint4 c[4], sc = lds128(at + groups * 128 + g * 16);
#pragma unroll
        for (int r = 0; r < 4; ++r) c[r] = lds128(at + g * 128 + (4 * cb + ((r + gq) & 3)) * 16);
        if (valid != kAllValid) {  // tokens that do not count: a scale of zero, whatever the bytes hold
          const int n = (int)(valid >> (8 * p) & 0xff);
          sc.x &= first_bytes(n), sc.y &= first_bytes(n - 4), sc.z &= first_bytes(n - 8), sc.w &= first_bytes(n - 12);
        }
        const uint32_t to = v_base + (i & 1) * C::kVBytes + half * (kKeys * 128) + p * kPiece * 128;
        auto four = [&](int k, uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t s4) {  // tokens 4 k ..
          uint32_t f[4][4], s01, s23;
          e4m3x4_to_f16(s4, s01, s23);
          e2m1x8_to_f16(c0, f[0]);
          e2m1x8_to_f16(c1, f[1]);
          e2m1x8_to_f16(c2, f[2]);
          e2m1x8_to_f16(c3, f[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t s1 = j < 2 ? s01 : s23;
            uint32_t h[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = j & 1 ? mul_by_half<1>(f[r][j], s1) : mul_by_half<0>(f[r][j], s1);
            const uint32_t tok = 4 * k + j;
            sts128(to + tok * 128 + (((2 * gq + cb) ^ (tok & 7)) << 4), h[0], h[1], h[2], h[3]);
          }
        };
        four(0, c[0].x, c[1].x, c[2].x, c[3].x, sc.x);
        four(1, c[0].y, c[1].y, c[2].y, c[3].y, sc.y);
        four(2, c[0].z, c[1].z, c[2].z, c[3].z, sc.z);
        four(3, c[0].w, c[1].w, c[2].w, c[3].w, sc.w);
      }
      arrive(sh.empty[st]);
      fence_proxy_async_shared();
      arrive(sh.o_ready[i & 1]);
      if (++st == (uint32_t)stages) st = 0, ph ^= 1u;
    }
  } else if (warp < kKLoadWarp) {
    // ------------------------------------------------------------ softmax
    // TMEM gives a thread the scores of 4 keys (lane / 4 and those 8, 16 and 24 behind) and of
    // two neighbouring columns in every eight: the factors, references and sums of NC / 4
    // columns stay in registers. (With a key a thread and all columns they came from shared
    // memory, 16 loads of 16 bytes a tile that the other roles' traffic held up: 800 to
    // 1200 cycles for 80 instructions.)
    constexpr int NC = N, CH = 16, NCH = NC / CH, J = NC / 8;  // (in runs of 32 columns the registers spilled)
    const int wg = (warp - kSoftmaxWarp) >> 2, quad = warp & 3, in_wg = (warp - kSoftmaxWarp) & 3;
    // the stream's columns of O and of the exchange arrays
    const int own0 = wg * NC;
    const int g = lane >> 2, t2 = (lane & 3) * 2;  // key in eight, column in eight
    const uint32_t tlane = (uint32_t)(quad * 32) << 16, tmem_o = tmem + tlane + kColO + own0;
    // this lane's row of the 8 x 8 blocks that it addresses for P's stores (see put)
    const int prow = quad * 32 + (lane >> 4) * 8 + (lane & 7), pchunk = lane >> 3 & 1;
    arrive(sh.s_ready[wg]);  // S is free
    uint64_t f[J], nm[J], l[J];  // factor, minus (reference - kLift), sum: two columns each
    bool first = true;           // no key of the stream has counted yet
    uint32_t met = 0;
    // the warpgroup's four warps wait for each other (no named barrier: that wait has no limit)
    auto meet = [&] {
      arrive(sh.meet[wg]);
      return wait(sh.meet[wg], met++, 17u);
    };
    // What `op` makes of the warp's values of each pair of columns, x[j] in lane (g, t2) that of
    // columns 8 j + t2: to row[own0 + ..]. Lanes halve their columns with every exchange.
    auto fold = [&](float2* x, float* row, auto op) {
#pragma unroll
      for (int o = 16, n = J / 2; o >= 4; o >>= 1, n >>= 1) {
        const bool up = lane & o;
        if (n) {
#pragma unroll
          for (int j = 0; j < n; ++j) {
            const float2 keep = up ? x[j + n] : x[j], give = up ? x[j] : x[j + n];
            x[j].x = op(keep.x, __shfl_xor_sync(0xffffffffu, give.x, o));
            x[j].y = op(keep.y, __shfl_xor_sync(0xffffffffu, give.y, o));
          }
        } else {
          x[0].x = op(x[0].x, __shfl_xor_sync(0xffffffffu, x[0].x, o));
          x[0].y = op(x[0].y, __shfl_xor_sync(0xffffffffu, x[0].y, o));
        }
      }
      if (g % (8 / J) == 0) *reinterpret_cast<float2*>(row + own0 + g / (8 / J) * 8 + t2) = x[0];
    };
    const int mine = own0 + in_wg * 32 + lane;  // the column whose reference the thread keeps
    const bool keeps = in_wg * 32 + lane < NC;
    for (uint32_t i = wg; i < tiles; i += 2) {  // (i & 1 = wg: the buffers of S, P and O)
      const uint32_t turn = i >> 1;
      if (!wait(sh.s_full[wg], turn, 5u)) break;
      tc::fence_after();
      const TileInfo info = sh.info[i % kInfo];
      if (info.flags & kFirst) {
        first = true;
        const float* ff = sh.f[info.seg % kF] + t2;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          f[j] = *reinterpret_cast<const uint64_t*>(ff + 8 * j);
          nm[j] = l[j] = 0;
        }
      }
      const bool any = info.valid != 0, partial = info.valid != kAllValid;  // keys of the tile that count
      bool on[4] = {true, true, true, true};  // keys g, g + 8, g + 16, g + 24 count
      if (partial) {
        const int v0 = (int)(info.valid >> (16 * quad) & 0xff), v1 = (int)(info.valid >> (16 * quad + 8) & 0xff);
        on[0] = g < v0, on[1] = g + 8 < v0, on[2] = g < v1, on[3] = g + 8 < v1;
      }
      const uint32_t tmem_s = tmem + tlane + kColS + wg * 64;
      uint32_t s[2][CH / 2];
      uint64_t sums[J];
      // scores of keys 0 .. 15 and 16 .. 31 of the warp's: columns 8 j + t2 (+ 1) of key g in
      // s[.][4 j] (4 j + 1), of key g + 8 in 4 j + 2 (4 j + 3)
      auto load = [&](int ch) {
        ld_16x256b<CH / 8>(tmem_s + ch * CH, s[0]);
        ld_16x256b<CH / 8>(tmem_s + ch * CH + (16u << 16), s[1]);
        tc::wait_ld();
      };
      // Weights of a run of columns, their sums over the thread's keys, and P^T into shared
      // memory: row = key, 128 bytes of 64 columns, 128-byte swizzle; 8 x 8 blocks of halves as
      // they lie in the registers.
      const uint32_t row = p_base + wg * C::kPBytes + (uint32_t)prow * 128;
      auto weigh = [&](int ch, auto masked) {
        uint32_t p[2][CH / 4];
#pragma unroll
        for (int j = 0; j < CH / 8; ++j) {
          const int col = ch * (CH / 8) + j;
          uint64_t sum = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t* v = &s[k >> 1][4 * j + 2 * (k & 1)];
            const float2 x = unpack2(fma2(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])), f[col], nm[col]));
            float2 e = make_float2(ex2(x.x), ex2(x.y));
            if (decltype(masked)::value && !on[k]) e = make_float2(0.f, 0.f);
            sum = add2(sum, pack2(e.x, e.y));
            p[k >> 1][2 * j + (k & 1)] = pack_f16(e.x, e.y);
          }
          sums[col] = sum;
        }
        const uint32_t at = row + (uint32_t)(((ch * (CH / 8) + pchunk) ^ (lane & 7)) << 4);
#pragma unroll
        for (int h = 0; h < 2; ++h)  // (columns 0 and 8 of keys 0 .., then of keys 8 ..)
          put(at + h * 16 * 128, p[h][0], p[h][2], p[h][1], p[h][3]);
      };
      // References move when the stream begins and when the vote says so: maxima over the
      // tile's keys, then O and the sums follow.
      // The products of the stream's tile before, which read P and write O, are complete.
      bool ok = wait(sh.pv_done[wg], turn ^ 1u, 6u);
      if (!ok) break;
      tc::fence_after();
#pragma unroll 1
      for (bool over = first && any;; over = true) {
        if (over) {
          float2 m[J];
#pragma unroll
          for (int ch = 0; ch < NCH; ++ch) {
            load(ch);
#pragma unroll
            for (int j = 0; j < CH / 8; ++j) {
              const float2 ff = unpack2(f[ch * (CH / 8) + j]);
              float2 x = make_float2(-INFINITY, -INFINITY);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t* v = &s[k >> 1][4 * j + 2 * (k & 1)];
                if (on[k]) x = make_float2(fmaxf(x.x, __uint_as_float(v[0]) * ff.x), fmaxf(x.y, __uint_as_float(v[1]) * ff.y));
              }
              m[ch * (CH / 8) + j] = x;
            }
          }
          fold(m, sh.mx[in_wg], [](float x, float y) { return fmaxf(x, y); });
          if (!(ok = meet())) break;
          if (keeps) {
            const float top = fmaxf(fmaxf(sh.mx[0][mine], sh.mx[1][mine]), fmaxf(sh.mx[2][mine], sh.mx[3][mine]));
            const float old = kLift - sh.nm[mine];
            const bool up = first || top > old + kSlack;
            if (up) sh.nm[mine] = kLift - top;
            sh.corr[mine] = up ? ex2(old - top) : 1.f;  // (not read for a stream's first)
          }
          if (!(ok = meet())) break;
#pragma unroll
          for (int j = 0; j < J; ++j) nm[j] = *reinterpret_cast<const uint64_t*>(&sh.nm[own0 + 8 * j + t2]);
          if (!first) {
            float2 corr[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
              corr[j] = *reinterpret_cast<const float2*>(&sh.corr[own0 + 8 * j + t2]);
              const float2 x = unpack2(l[j]);
              l[j] = pack2(x.x * corr[j].x, x.y * corr[j].y);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < J; ++j) {
                uint32_t o[4];
                const uint32_t at = tmem_o + (h ? 16u << 16 : 0u) + 8 * j;
                ld_16x256b<1>(at, o);
                tc::wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  o[k] = __float_as_uint(__uint_as_float(o[k]) * (k & 1 ? corr[j].y : corr[j].x));
                st_16x256b_x1(at, o);
              }
            tc::wait_st();
          }
          first = false;
        }
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          load(ch);
          if (partial) weigh(ch, std::true_type());
          else weigh(ch, std::false_type());
        }
        if (over) break;  // weights are 2^kLift at most now
        float most = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float2 x = unpack2(sums[j]);
          most = max3(most, x.x, x.y);  // (leaves NaNs out)
        }
        if (__any_sync(0xffffffffu, !first && most > kTop) && lane == 0) sh.over[wg][turn & 1] = i + 1;
        if (!(ok = meet()) || *(volatile uint32_t*)&sh.over[wg][turn & 1] != i + 1) break;
      }
      if (!ok) break;
      tc::fence_before();
      arrive(sh.s_ready[wg]);  // S has been read: room for the next in its place
#pragma unroll
      for (int j = 0; j < J; ++j) l[j] = add2(l[j], sums[j]);
      fence_proxy_async_shared();
      tc::fence_before();
      arrive(sh.o_ready[wg]);
      if (info.flags & kLast) {
        // the stream's sums: O from TMEM (lane = dim), l over the 128 keys' threads
        if (!wait(sh.pv_done[wg], turn, 8u)) break;
        tc::fence_after();
        const SegInfo si = sh.seg[info.seg % kSegs];
        const long long out = (2ll * si.slot + wg) * a.rows;
        const int m = quad * 32 + lane;
        float* to = a.part_o + out * (groups * 16) + dim_of(m);
        const int cols = m < groups * 16 ? si.rows : 0;
#pragma unroll 1
        for (int c0 = 0; c0 < NC; c0 += 8, to += 8 * groups * 16) {
          uint32_t o[8];
          ld8(tmem_o + c0, o);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c0 + e < cols) to[e * groups * 16] = __uint_as_float(o[e]);
        }
        tc::fence_before();
        arrive(sh.o_empty[wg]);
        float2 x[J];
#pragma unroll
        for (int j = 0; j < J; ++j) x[j] = unpack2(l[j]);
        fold(x, sh.sum[in_wg], [](float x, float y) { return x + y; });
        if (!meet()) break;
        // (the sums' next writer comes behind a vote of the next tile's, and with it all these reads)
        const int r = in_wg * 32 + lane;
        if (r < si.rows) {
          const float sum = (sh.sum[0][mine] + sh.sum[1][mine]) + (sh.sum[2][mine] + sh.sum[3][mine]);
          a.part_ml[out + r] = first ? make_float2(-INFINITY, 0.f) : make_float2(-sh.nm[mine], sum);
          if (info.flags & kOnly) a.part_ml[out + r + (wg ? -a.rows : a.rows)] = make_float2(-INFINITY, 0.f);
        }
      }
    }
  } else {
    if (warp == kKLoadWarp || warp == kVLoadWarp) {
      // ------------------------------------------------------------ segments, pages, copies
      // One warp copies K and tells the others of a tile, one copies V (a copy takes its warp
      // 110 cycles, and a tile of two pages is four); both lay out Q of the segments behind
      // the first.
      const bool is_v = warp == kVLoadWarp;
      const uint8_t* pool = is_v ? a.v_pool : a.k_pool;
      unsigned flags = 0;
      const uint64_t once = l2_evict_first_policy();
      const int unit_shift = a.ppb_shift < 0 ? 0 : min(a.ppb_shift, 3);  // log2 of a unit's pieces
      uint32_t i = 0, st = 0, ph = 0, seg = 0;
      bool ok = true;
      const int end = sh.line.begin(blockIdx.x + 1);
      for (Segment s = sh.first; ok && s.tiles; s = segment_from(a, sh.line, s.next, end)) {
        if (seg > 0) {
          // (its buffer's segment before, the first one too, has been multiplied)
          if (seg > 1 && !(ok = wait(sh.q_empty[seg & 1], (seg >> 1) - 1, 10u))) break;
          lay_out_q(q_rows(a, s), N, q_base + (seg & 1) * C::kQBytes, sh.f[seg % kF], is_v, 2);
          arrive(sh.q_full[seg & 1]);
        }
        if (!is_v && lane == 0) {
          sh.seg[seg % kSegs].slot = s.slot;
          sh.seg[seg % kSegs].rows = min(a.rows, a.T * a.G - s.rt * a.rows);
        }
        // Lane = unit, the pieces of a tile that lie in one page: one copy. 32 units (16 tiles for
        // pages of 64 tokens) are a batch. A selected block is read two batches ahead, its
        // page one, and neither is looked at before it is due, so that a batch's copies wait
        // for no load of their own (when they did, the loading warp took 1000 cycles a tile).
        const int32_t* sel = a.sel ? a.sel + ((long long)s.b * a.Hkv + s.h) * a.sel_stride : nullptr;
        const int32_t* row = a.block_table + (long long)s.b * a.nb_max;
        const int slots = sel ? a.n_sel : s.full, p0 = s.tile0 * kPieces + (lane << unit_shift);
        const int last = min((s.tile0 + s.tiles) * kPieces, s.pieces), batch = 32 << unit_shift;
        auto slot_of = [&](int p) { return a.ppb_shift >= 0 ? p >> a.ppb_shift : quotient(p, a.ppb); };
        auto entry_of = [&](int p) {
          const int at = sel && p < last ? slot_of(p) : slots;
          return at < slots ? __ldcg(sel + at) : -1;
        };
        struct Look {
          int valid, sub, page;  // tokens that count, first piece within its block, page (not checked)
        };
        auto look = [&](int p, int entry) {
          Look k = {0, 0, 0};
          if (p >= last) return k;
          const int at = slot_of(p);
          int block = sel ? entry : at;
          k.sub = p - at * a.ppb;
          k.valid = kPiece << unit_shift;
          if (at >= slots) {  // the partial last block
            block = s.full;
            k.sub = p - slots * a.ppb;
            k.valid = min(k.valid, s.ctx - s.full * a.blk - k.sub * kPiece);
          } else if (block < 0 || block >= s.full) {
            if (block != -1) flags |= SV_FLAG_BAD_BLOCK_INDEX;
            k.valid = 0;
            return k;
          }
          k.page = __ldcg(row + block);
          return k;
        };
        int entry = entry_of(p0);
        Look next = look(p0, entry);
        entry = entry_of(p0 + batch);
#pragma unroll 1
        for (int t0 = 0, p = p0; ok && t0 < s.tiles; t0 += batch / kPieces, p += batch) {
          Look now = next;
          next = look(p + batch, entry);
          entry = entry_of(p + 2 * batch);
          if (now.valid && (now.page < 0 || now.page >= a.num_pages)) {
            flags |= SV_FLAG_BAD_PAGE;
            now.valid = 0;
          }
          const uint8_t* from = pool + ((long long)now.page * a.Hkv * a.ppb + s.h * a.ppb + now.sub) * pb;
          const uint32_t bytes = (uint32_t)(now.valid + kPiece - 1) / kPiece * pb;
          const uint32_t to = (is_v ? side : 0u) + ((uint32_t)(lane << unit_shift) % kPieces) * pb;
          const bool full = __all_sync(0xffffffffu, now.valid == kPiece << unit_shift);
          const int tile = (lane << unit_shift) / kPieces, n = min(batch / kPieces, s.tiles - t0);
#pragma unroll 1
          for (int t = 0; t < n; ++t, ++i) {
            if (!(ok = wait(sh.empty[st], ph ^ 1u, 9u))) break;
            const uint32_t bar = smem_u32(&sh.full[st]);
            uint32_t all = kPieces * pb;
            uint64_t valid = kAllValid;
            if (!full) {
              uint32_t lo = 0, hi = 0;
              if (tile == t) {
#pragma unroll 1
                for (int j = 0; j < 1 << unit_shift; ++j) {
                  const uint32_t v = (uint32_t)min(max(now.valid - j * kPiece, 0), kPiece);
                  const int at = (lane << unit_shift) % kPieces + j;
                  if (at < 4) lo |= v << (8 * at);
                  else hi |= v << (8 * (at - 4));
                }
              }
              lo = __reduce_or_sync(0xffffffffu, lo);
              hi = __reduce_or_sync(0xffffffffu, hi);
              valid = (uint64_t)hi << 32 | lo;
              all = __reduce_add_sync(0xffffffffu, tile == t ? bytes : 0u);
            }
            if (lane == 0) {
              if (!is_v) {
                const int at = t0 + t, left = s.tiles - at;
                const uint32_t place = (at == 0 ? kBegin : 0u) | (left == 1 ? kEnd : 0u) | (at < 2 ? kFirst : 0u) |
                                       (left <= 2 ? kLast : 0u) | (s.tiles == 1 ? kOnly : 0u);
                sh.info[i % kInfo] = {valid, place, seg};
              }
              mbar_arrive_expect_tx(bar, all);
            }
            __syncwarp();
            if (tile == t && bytes) bulk_load_once(ring + st * stage_bytes + to, from, bytes, bar, once);
            if (++st == (uint32_t)stages) st = 0, ph ^= 1u;
          }
        }
        ++seg;
      }
      if (flags) atomicOr(a.status, flags);
      if (lane == 0) sh.copied[is_v] = i;
    } else if (warp == kScoreWarp) {
      // ------------------------------------------------------------ S^T = K Q^T
      constexpr uint32_t id_s = idesc_f16(N, false, false);
      const uint64_t dq = tc::smem_desc(q_base, 16, 1024);
      const uint32_t lead = elect_lead();
      for (uint32_t i = 0; i < tiles; ++i) {
        if (!wait(sh.s_ready[i & 1], i >> 1, 11u)) break;
        const TileInfo info = sh.info[i % kInfo];
        const uint32_t sb = i & 1, qb = info.seg & 1;
        // (the first segment's Q has a barrier of its own: buffer 0 completes once less)
        if ((info.flags & kBegin) &&
            !(info.seg ? wait(sh.q_full[qb], (info.seg >> 1) - (qb ^ 1u), 12u) : wait(sh.q_first, 0, 12u)))
          break;
        tc::fence_after();
        const uint64_t q = dq + (uint64_t)(qb * (C::kQBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < (DG ? DG : 8); ++kk)
          if (DG || kk < groups)
            lead_mma_ts(lead, tmem + kColS + sb * 64, tmem + kColK + (i & 1) * 64 + kk * 8,
                        q + (uint64_t)(((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4), id_s, kk > 0 ? 1u : 0u);
        lead_commit(lead, smem_u32(&sh.s_full[sb]));
        lead_commit(lead, smem_u32(&sh.k_empty[i & 1]));
        if (info.flags & kEnd) lead_commit(lead, smem_u32(&sh.q_empty[qb]));
      }
      if (sh.abort) {  // products in flight end before TMEM is given back
        lead_commit(lead, smem_u32(&sh.drained[0]));
        mbar_wait_drain(smem_u32(&sh.drained[0]), 0);
      }
    } else {
      // ------------------------------------------------------------ O^T += V^T P^T
      const int pairs = a.B * a.Hkv * a.row_tiles;
      for (int p = blockIdx.x * 32 + lane; p < pairs; p += gridDim.x * 32) a.slots[p] = slots_of(a, sh.line, p);
      __syncwarp();
      constexpr uint32_t id_o = idesc_f16(N, true, true);
      const uint64_t dp = tc::smem_desc(p_base, kKeys * 128, 1024), dv = tc::smem_desc(v_base, kKeys * 128, 1024);
      const uint32_t lead = elect_lead();
      uint32_t begun[2] = {0, 0};  // segments that O's streams have begun
      for (uint32_t i = 0; i < tiles; ++i) {
        if (!wait(sh.o_ready[i & 1], i >> 1, 14u)) break;
        const bool first = sh.info[i % kInfo].flags & kFirst;
        const uint32_t ob = i & 1;
        if (first && !wait(sh.o_empty[ob], begun[ob]++ ^ 1u, 15u)) break;
        tc::fence_after();
        const uint64_t p = dp + (uint64_t)((i & 1) * (C::kPBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          lead_mma_ss(lead, tmem + kColO + ob * N, dv + (uint64_t)((ob * C::kVBytes + kk * 2048) >> 4),
                      p + (uint64_t)((kk * 2048) >> 4), id_o, first && kk == 0 ? 0u : 1u);
        lead_commit(lead, smem_u32(&sh.pv_done[i & 1]));
      }
      if (sh.abort) {
        lead_commit(lead, smem_u32(&sh.drained[1]));
        mbar_wait_drain(smem_u32(&sh.drained[1]), 0);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kScoreWarp) tc::dealloc(tmem, kTmemCols);
  if (sh.abort && warp == kKLoadWarp && lane == 0)  // copies in flight end before the CTA does
    end_copies(
        sh.copied[0], sh.copied[1], (uint32_t)stages, [&](uint32_t st) { mbar_arrive(smem_u32(&sh.full[st])); },
        [&](uint32_t st, uint32_t parity) { mbar_wait_drain(smem_u32(&sh.full[st]), parity); });
}

template <int N, int DG>
cudaError_t launch(const Attend4Args& a, cudaStream_t st) {
  using C = Cfg<N>;
  constexpr int kMost = 227 * 1024;
  static std::atomic<int> ready[kMaxDevices];
  const int dev = current_device();
  if (!ready[dev].load()) {
    const cudaError_t e =
        cudaFuncSetAttribute(attend4_tc_kernel<N, DG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    ready[dev].store(1);
  }
  const int stage = 2 * kPieces * piece_bytes(a.d), fixed = 1024 + C::kFixed + 128;
  const int stages = std::min(kMaxStages, (kMost - fixed) / stage);
  return launch_pdl(attend4_tc_kernel<N, DG>, dim3(a.ctas), dim3(kThreads), (size_t)kMost, st, a, stages);
}

template <int N>
cudaError_t launch_n(const Attend4Args& a, cudaStream_t st) {
  return a.d == 128 ? launch<N, 8>(a, st) : launch<N, 0>(a, st);
}

}  // namespace

bool attend4_tc_applies(const Attend4Args& a, int dtype) { return dtype == SV_BF16 && a.d <= 128; }

cudaError_t launch_attend4_tc(Attend4Args a, cudaStream_t st) {
  const int stacked = a.T * a.G;
  a.row_tiles = (stacked + kTc4Rows - 1) / kTc4Rows;
  a.rows = (stacked + a.row_tiles - 1) / a.row_tiles;
  a.streams = 2;
  a.pair_cost = kPairCost;
  a.ppt = kPieces;
  a.ppt_shift = 3;
  a.ctas = std::min(kMaxTc4Ctas, sm_count());
  const cudaError_t e = a.rows <= 16   ? launch_n<16>(a, st)
                        : a.rows <= 32 ? launch_n<32>(a, st)
                                       : launch_n<64>(a, st);
  return e == cudaSuccess ? launch_join4(a, SV_BF16, st) : e;
}

}  // namespace sva
