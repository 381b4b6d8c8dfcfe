// Attention over a 4-bit cache on the 5th-generation tensor cores (tcgen05, TMEM):
// bf16 queries, head dims up to 128, pages of any multiple of 16 tokens.
//
// Rows are few (T drafts x G heads of a KV head) and the cache is long, so the
// products are taken transposed: S^T = K Q^T with the 128 keys of a tile as the
// M rows and the rows as the N columns, O^T += V^T P^T with the head's dims as M.
// The cost of a product then follows the rows (N = 16 .. 128), not a padded 128,
// and K and V^T are the A operands, which tcgen05 takes from TMEM: a code goes
// from the ring of pages through a thread's registers, where it becomes a half, into
// TMEM, and never back into shared memory. That is why V's pages keep a dim's tokens
// together: a TMEM lane of V^T is one dim.
// Code times scale has at most five significant bits and is exact in f16. Q is
// scaled by a power of two per row so that its largest element lies in [2^14, 2^15),
// exact as well; factor and exponents go into the softmax's scale.
//
// Warps: 0-3 K, 4-7 V (codes to halves), then the softmax (one warpgroup for up to
// 32 rows, else two that share the columns), one that takes the CTA's segments off
// the line, looks pages up, copies them and lays out Q, one that issues the MMAs.
// A softmax thread has one key and a run of rows (columns). It does not look for
// a tile's maxima: a row's reference stands until some score exceeds it by 2^8, which
// the warps find out with a vote at the tile's barrier; only then (and in a segment's first
// tile) maxima are taken across lanes and O is rescaled. Weights are held 2^7 times
// their size, so that f16's range covers 2^-31 .. 2^8 of the reference.
#include <algorithm>
#include <atomic>

#include "host.h"
#include "kv4.cuh"
#include "tc.h"
#include "tc_issue.cuh"

namespace sva {
namespace {

using namespace kv4;

constexpr int kKeys = 128, kPieces = kKeys / kPiece;
constexpr int kInfo = 16;   // ring of tile infos: more than tiles in flight (stages, and two behind them)
constexpr int kSegs = 8;    // ring of segment infos: more than the segments that Q and S run ahead
constexpr int kMaxStages = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 128, kColK = 256, kColV = 384;  // K and V: two of 64 columns
constexpr float kLift = 7.f;    // weights are 2^kLift times their size ...
constexpr float kSlack = 8.f;   // ... and at most 2^kSlack above the reference's

// What the loading warp tells the others of a tile: tokens that count of each piece
// (a byte each), and whether a segment begins or ends with it.
struct TileInfo {
  uint64_t valid;
  uint32_t flags;
};
constexpr uint32_t kFirst = 1, kLast = 2;
constexpr uint64_t kAllValid = 0x1010101010101010ull;

struct SegInfo {
  long long slot;
  int rows;
};

struct Control {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t k_full[2], k_empty[2], v_full[2], s_full[2], s_empty[2], p_full[2], pv_done[2];
  uint64_t q_full[2], q_empty[2], o_empty, drained, meet[2];
  uint32_t tmem;
  int abort;
  uint32_t over[2][2];                   // by warpgroup and tile parity: 1 + the tile whose references move
  TileInfo info[kInfo];
  SegInfo seg[kSegs];
  alignas(16) float f[kSegs][kTc4Rows];  // factor of a row's scores
  alignas(16) float nm[kTc4Rows];        // minus (reference - kLift) of a row, log2 domain
  float corr[kTc4Rows];
  float mx[4][kTc4Rows];                 // by warp of a softmax warpgroup (also: sums)
  int cu[kMaxB4 + 1];
};

template <int N>
struct Cfg {
  static constexpr int kGroups = N <= 32 ? 1 : 2;    // softmax warpgroups
  static constexpr int kCols = N / kGroups;          // rows (columns) of a warpgroup
  static constexpr int kThreads = 256 + 128 * kGroups + 64;
  static constexpr int kLoadWarp = 8 + 4 * kGroups, kMmaWarp = kLoadWarp + 1;
  static constexpr int kS = N <= 64 ? 2 : 1;         // S buffers
  static constexpr int kQ = N <= 64 ? 2 : 1;         // Q buffers
  static constexpr int kQBytes = 2 * N * 128;        // two blocks of 64 dims
  static constexpr int kPBytes = (N > 64 ? 2 : 1) * kKeys * 128;
  static constexpr int kFixed = kQ * kQBytes + 2 * kPBytes + (int)sizeof(Control);
};

__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
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
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// 16 lanes x 32 columns of TMEM: four blocks of 8 columns; of a block, the lane's
// registers are row lane / 4 (columns 2 (lane % 4), + 1) and row lane / 4 + 8.
__device__ __forceinline__ void st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Instruction descriptor of kind::f16 with f16 operands and fp32 sums, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// The rest of a wait, out of line: four roles' loops share an SM quarter's instruction
// cache, and with every wait's clock and limit inline (and the loops unrolled) they did
// not fit. 128 K tokens x 4 took 495 us, most of it waiting for instructions.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, unsigned* status,
                                     unsigned site) {
  return mbar_wait_abortable(bar, parity, abort, status, site);
}

// DG: groups of 16 dims (8: d = 128), 0: any number up to 8.
template <int N, int DG>
__global__ void __launch_bounds__(Cfg<N>::kThreads, 1) attend4_tc_kernel(const __grid_constant__ Attend4Args a, int stages) {
  using C = Cfg<N>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_base = base, p_base = q_base + C::kQ * C::kQBytes;
  const uint32_t ctl = p_base + 2 * C::kPBytes;
  Control& sh = *reinterpret_cast<Control*>(smem_raw + (ctl - smem_u32(smem_raw)));
  const uint32_t ring = ctl + (uint32_t)((sizeof(Control) + 127) / 128 * 128);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = DG ? DG : a.d / 16;
  const uint32_t pb = (uint32_t)piece_bytes(groups * 16), side = kPieces * pb, stage_bytes = 2 * side;

  if (warp == C::kMmaWarp) tc::alloc(smem_u32(&sh.tmem), kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), 4);
      mbar_init(smem_u32(&sh.k_empty[i]), 1);
      mbar_init(smem_u32(&sh.v_full[i]), 4);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.s_empty[i]), 4 * C::kGroups);
      mbar_init(smem_u32(&sh.p_full[i]), 4 * C::kGroups);
      mbar_init(smem_u32(&sh.pv_done[i]), 1);
      mbar_init(smem_u32(&sh.q_full[i]), 1);
      mbar_init(smem_u32(&sh.q_empty[i]), 1);
    }
    mbar_init(smem_u32(&sh.o_empty), 4 * C::kGroups);
    mbar_init(smem_u32(&sh.drained), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.meet[i]), 4);
      sh.over[i][0] = sh.over[i][1] = 0;
    }
    sh.abort = 0;
    fence_barrier_init();
  }
  pdl_wait();
  pdl_trigger();
  bool bad = false;
  if (warp == C::kLoadWarp) {
    bad = scan_tiles(a, sh.cu);
    __syncwarp();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  if (blockIdx.x == 0)
    for (int b = tid; b <= a.B; b += C::kThreads) a.cu[b] = sh.cu[b];
  const Line line = line_of(a, sh.cu[a.B]);
  const int cta = blockIdx.x;
  const long long begin = cta < line.ctas ? line.first(cta) : 0, end = cta < line.ctas ? line.first(cta + 1) : 0;
  const uint32_t tiles = (uint32_t)(end - begin);
  auto wait = [&](uint64_t& bar, uint32_t parity, unsigned site) {
    const uint32_t addr = smem_u32(&bar);
    return mbar_try_wait(addr, parity & 1u) || wait_on(addr, parity & 1u, &sh.abort, a.status, site);
  };

  if (warp < 4) {
    // ------------------------------------------------------------ K: lane = key
    const uint32_t piece = (uint32_t)tid / kPiece, tok = (uint32_t)tid % kPiece;
    const uint32_t tlane = (uint32_t)(warp * 32) << 16;
    for (uint32_t i = 0, st = 0, ph = 0; i < tiles; ++i) {
      if (!wait(sh.full[st], ph, 1u)) break;
      if (!wait(sh.k_empty[i & 1], (i >> 1) ^ 1u, 2u)) break;
      tc::fence_after();
      const uint32_t codes = ring + st * stage_bytes + piece * pb, scales = codes + groups * 128 + tok * groups;
      const uint32_t to = tmem + tlane + kColK + (i & 1) * 64;
#pragma unroll 1
      for (int g = 0; g < groups; g += 2) {
        uint32_t r[16];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (!DG && g + j >= groups) {  // the second half of the last pair
#pragma unroll
            for (int e = 0; e < 8; ++e) r[8 * j + e] = 0;
            continue;
          }
          const uint32_t two = __byte_perm(e4m3x2_to_f16x2(lds8(scales + g + j)), 0, 0x1010);
          const uint2 w = lds64(codes + (g + j) * 128 + tok * 8);
          e2m1x8_to_f16(w.x, r + 8 * j);
          e2m1x8_to_f16(w.y, r + 8 * j + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) r[8 * j + e] = mul_f16x2(r[8 * j + e], two);
        }
        tc::st16(to + g * 8, r);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.empty[st]));
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.k_full[i & 1]));
      if (++st == (uint32_t)stages) st = 0, ph ^= 1u;
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ V: lane = dim
    const int w = warp - 4;
    const uint32_t t4 = lane & 3;  // code row lane / 4 (that dim and the one 8 behind), tokens 4 t4 ..
    for (uint32_t i = 0, st = 0, ph = 0; i < tiles; ++i) {
      if (!wait(sh.full[st], ph, 3u)) break;
      if (!wait(sh.pv_done[i & 1], (i >> 1) ^ 1u, 4u)) break;
      tc::fence_after();
      const uint64_t valid = sh.info[i % kInfo].valid;
      const uint32_t from = ring + st * stage_bytes + side;
      if (valid != kAllValid) {
        // tokens that do not count get a scale of zero, whatever their bytes hold: the
        // warp's two groups x 128 tokens, 4 tokens at a time
        for (int e = lane; e < 64; e += 32) {
          const int g = 2 * w + (e >> 5), p = e >> 2 & 7, n = (int)(valid >> (8 * p) & 0xff) - (e & 3) * 4;
          const uint32_t at = from + p * pb + groups * 128 + g * 16 + (e & 3) * 4;
          if (g < groups && n < 4) sts32(at, n <= 0 ? 0u : lds32(at) & ((1u << (8 * n)) - 1u));
        }
        fence_proxy_async_shared();  // ahead of the next copy into the stage
        __syncwarp();
      }
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {  // group q / 2 of the warp's two, half q % 2 of the keys
        const int g = 2 * w + (q >> 1);
        if (!DG && g >= groups) break;
        const uint32_t code = from + (q & 1) * 4 * pb + g * 128 + lane * 4;
        const uint32_t scale = from + (q & 1) * 4 * pb + groups * 128 + g * 16 + t4 * 4;
        uint32_t r[16];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t c = lds32(code + p * pb), s = lds32(scale + p * pb), c4 = c >> 4, c8 = c >> 8;
          const uint32_t lo = (c & 0x000f000fu) | (c4 & 0xfff0fff0u);   // bytes 0, 2: tokens (0, 1), (2, 3)
          const uint32_t hi = (c4 & 0x000f000fu) | (c8 & 0xfff0fff0u);  // ... of the dim 8 behind
          uint32_t s01, s23;
          e4m3x4_to_f16(s, s01, s23);
          e2m1x4_to_f16(lo, r[4 * p], r[4 * p + 1]);
          e2m1x4_to_f16(hi, r[4 * p + 2], r[4 * p + 3]);
          r[4 * p] = mul_f16x2(r[4 * p], s01);
          r[4 * p + 1] = mul_f16x2(r[4 * p + 1], s23);
          r[4 * p + 2] = mul_f16x2(r[4 * p + 2], s01);
          r[4 * p + 3] = mul_f16x2(r[4 * p + 3], s23);
        }
        st_16x256b_x4(tmem + ((uint32_t)(w * 32 + (q >> 1) * 16) << 16) + kColV + (i & 1) * 64 + (q & 1) * 32, r);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.empty[st]));
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.v_full[i & 1]));
      if (++st == (uint32_t)stages) st = 0, ph ^= 1u;
    }
  } else if (warp < C::kLoadWarp) {
    // ------------------------------------------------------------ softmax: lane = key
    constexpr int CH = C::kCols <= 32 ? C::kCols : 16;  // columns in registers at a time
    constexpr int NCH = C::kCols / CH;
    const int wg = (warp - 8) >> 2, quad = warp & 3, col0 = wg * C::kCols;
    const int key = quad * 32 + lane;
    const uint32_t tlane = (uint32_t)(quad * 32) << 16;
    float l[C::kCols];
    bool first = true;  // no key of the segment has counted yet
    uint32_t seg = 0, met = 0;
    bool ok = true;
    // the warpgroup's four warps wait for each other (no named barrier: that wait has no limit)
    auto meet = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.meet[wg]));
      return wait(sh.meet[wg], met++, 17u);
    };
    for (uint32_t i = 0; i < tiles; ++i) {
      const uint32_t sb = i % C::kS;
      if (!(ok = wait(sh.s_full[sb], i / C::kS, 5u))) break;
      tc::fence_after();
      const TileInfo info = sh.info[i % kInfo];
      const uint32_t flags = info.flags;
      const float* f = sh.f[seg % kSegs] + col0;
      if (flags & kFirst) {
        first = true;
#pragma unroll
        for (int c = 0; c < C::kCols; ++c) l[c] = 0.f;
      }
      const bool counts = key % kPiece < (int)(info.valid >> (8 * (key / kPiece)) & 0xff);
      const bool any = info.valid != 0;  // a key of the tile counts
      uint32_t s[CH];
      auto load = [&](int ch) {
        const uint32_t at = tmem + tlane + kColS + sb * 64 + col0 + ch * CH;
        if constexpr (CH == 32) tc::ld32(at, s);
        else if constexpr (CH == 16) tc::ld16(at, s);
        else {
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]), "=r"(s[7])
                       : "r"(at)
                       : "memory");
        }
        tc::wait_ld();
        if (!counts) {
#pragma unroll
          for (int c = 0; c < CH; ++c) s[c] = 0xff800000u;
        }
      };
      // x = s f - (m - kLift), in place
      auto relative = [&](int ch) {
#pragma unroll
        for (int c = 0; c < CH; c += 4) {
          const float4 ff = *reinterpret_cast<const float4*>(f + ch * CH + c);
          const float4 nn = *reinterpret_cast<const float4*>(sh.nm + col0 + ch * CH + c);
          s[c] = __float_as_uint(__fmaf_rn(__uint_as_float(s[c]), ff.x, nn.x));
          s[c + 1] = __float_as_uint(__fmaf_rn(__uint_as_float(s[c + 1]), ff.y, nn.y));
          s[c + 2] = __float_as_uint(__fmaf_rn(__uint_as_float(s[c + 2]), ff.z, nn.z));
          s[c + 3] = __float_as_uint(__fmaf_rn(__uint_as_float(s[c + 3]), ff.w, nn.w));
        }
      };
      bool over = first && any;
      if (!over) {
        float top = -INFINITY;
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          load(ch);
          relative(ch);
#pragma unroll
          for (int c = 0; c < CH; ++c) top = fmaxf(top, __uint_as_float(s[c]));
        }
        if (__any_sync(0xffffffffu, !first && counts && top > kLift + kSlack) && lane == 0) sh.over[wg][i & 1] = i + 1;
        if (!(ok = meet())) break;
        over = *(volatile uint32_t*)&sh.over[wg][i & 1] == i + 1;
      }
      if (over) {
        // the references move: maxima over the tile's keys, then O and the sums follow
#pragma unroll 1
        for (int ch = 0; ch < NCH; ++ch) {
          load(ch);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const float m = redux_max(counts ? __uint_as_float(s[c]) * f[ch * CH + c] : -INFINITY);
            if (lane == 0) sh.mx[quad][col0 + ch * CH + c] = m;
          }
        }
        if (!(ok = meet())) break;
        const int c = (warp - 8 - 4 * wg) * 32 + lane;
        if (c < C::kCols) {
          const int col = col0 + c;
          const float top = fmaxf(fmaxf(sh.mx[0][col], sh.mx[1][col]), fmaxf(sh.mx[2][col], sh.mx[3][col]));
          const float old = kLift - sh.nm[col];
          const bool move = first || top > old + kSlack;
          sh.corr[col] = move && !first ? ex2(old - top) : 1.f;
          if (move) sh.nm[col] = kLift - top;
        }
        if (!(ok = meet())) break;
        if (!first) {
          if (!(ok = wait(sh.pv_done[(i - 1) & 1], (i - 1) >> 1, 6u))) break;
          tc::fence_after();
#pragma unroll
          for (int c0 = 0; c0 < C::kCols; c0 += 8) {
            uint32_t o[8];
            const uint32_t at = tmem + tlane + kColO + col0 + c0;
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7])
                         : "r"(at)
                         : "memory");
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float k = sh.corr[col0 + c0 + c];
              o[c] = __float_as_uint(__uint_as_float(o[c]) * k);
              l[c0 + c] *= k;
            }
            tc::st8(at, o);
          }
          tc::wait_st();
        }
        first = false;
      }
      // weights, their sums, and P^T into shared memory (row = key, 128 bytes of 64 columns)
      if (!(ok = wait(sh.pv_done[i & 1], (i >> 1) ^ 1u, 7u))) break;
      const uint32_t row = p_base + (i & 1) * C::kPBytes + (uint32_t)key * 128;
#pragma unroll
      for (int ch = 0; ch < NCH; ++ch) {
        if (NCH > 1 || over) {
          load(ch);
          relative(ch);
        }
        if (ch == NCH - 1) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.s_empty[sb]));
        }
#pragma unroll
        for (int c = 0; c < CH; c += 8) {
          uint32_t p[4] = {0, 0, 0, 0};
          if (counts) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = ex2(__uint_as_float(s[c + 2 * e])), y = ex2(__uint_as_float(s[c + 2 * e + 1]));
              l[ch * CH + c + 2 * e] += x;
              l[ch * CH + c + 2 * e + 1] += y;
              p[e] = pack_f16(x, y);
            }
          }
          const uint32_t col = (uint32_t)(col0 + ch * CH + c);
          sts128(row + (col >> 6) * (kKeys * 128) + ((((col & 63) >> 3) ^ (key & 7)) << 4), p[0], p[1], p[2], p[3]);
        }
      }
      fence_proxy_async_shared();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[i & 1]));
      if (flags & kLast) {
        // the segment's sums: l over the 128 keys' threads, O from TMEM (lane = dim)
        const SegInfo info2 = sh.seg[seg % kSegs];
#pragma unroll
        for (int c = 0; c < C::kCols; ++c) {
          float x = l[c];
#pragma unroll
          for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (lane == 0) sh.mx[quad][col0 + c] = x;
        }
        if (!(ok = meet())) break;
        const int c = (warp - 8 - 4 * wg) * 32 + lane, r = col0 + c;
        const long long out = info2.slot * a.rows;
        if (c < C::kCols && r < info2.rows) {
          const float x = (sh.mx[0][r] + sh.mx[1][r]) + (sh.mx[2][r] + sh.mx[3][r]);
          a.part_ml[out + r] = first ? make_float2(-INFINITY, 0.f) : make_float2(-sh.nm[r], x);
        }
        if (!(ok = wait(sh.pv_done[i & 1], i >> 1, 8u))) break;
        tc::fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < C::kCols && col0 + c0 < info2.rows; c0 += 8) {
          uint32_t o[8];
          const uint32_t at = tmem + tlane + kColO + col0 + c0;
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7])
                       : "r"(at)
                       : "memory");
          tc::wait_ld();
          if (key < groups * 16) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (col0 + c0 + e < info2.rows) a.part_o[(out + col0 + c0 + e) * (groups * 16) + key] = __uint_as_float(o[e]);
          }
        }
        tc::fence_before();
        if (!(ok = meet())) break;  // the exchange arrays are free again, and O has been read
        if (lane == 0) mbar_arrive(smem_u32(&sh.o_empty));
        ++seg;
      }
    }
    (void)ok;
  } else if (warp == C::kLoadWarp) {
    // ------------------------------------------------------------ segments, pages, copies, Q
    unsigned flags = bad ? SV_FLAG_BAD_LENGTH : 0u;
    uint32_t i = 0, st = 0, ph = 0, seg = 0;
    bool ok = true;
    for (long long x = begin; ok && x < end; ++seg) {
      const Segment s = segment_at(a, sh.cu, x, end, cta);
      x += s.tiles;
      const int row0 = s.rt * a.rows, rows = min(a.rows, a.T * a.G - row0);
      if (lane == 0) {
        sh.seg[seg % kSegs].slot = s.slot;
        sh.seg[seg % kSegs].rows = rows;
      }
      // four tiles' pages at a time: lane = piece
      int valid;
      long long at = piece_at(a, s, s.tile0 * kPieces + lane, &valid, &flags);
      if (s.tiles * kPieces <= lane) at = -1, valid = 0;
      for (int t0 = 0; ok && t0 < s.tiles; t0 += 4) {
        const long long now = at;
        const int v = valid;
        if (t0 + 4 < s.tiles) {
          at = piece_at(a, s, (s.tile0 + t0 + 4) * kPieces + lane, &valid, &flags);
          if ((s.tiles - t0 - 4) * kPieces <= lane) at = -1, valid = 0;
        }
        const long long prev = __shfl_up_sync(0xffffffffu, now, 1);
        const bool there = now >= 0;
        // a run of pieces that follow each other in the pool is one copy
        const uint32_t heads = __ballot_sync(0xffffffffu, there && ((lane & 7) == 0 || prev < 0 || now != prev + 1));
        const uint32_t have = __ballot_sync(0xffffffffu, there);
        const uint32_t stop = (heads | ~have | 0x01010101u) & ~((2u << lane) - 1u);  // where a run of this lane ends
        const int run = (stop ? __ffs(stop) - 1 : 32) - lane;
        for (int t = 0; t < 4 && t0 + t < s.tiles; ++t, ++i) {
          if (!(ok = wait(sh.empty[st], ph ^ 1u, 9u))) break;
          const uint32_t nibble = (lane >> 3) == t ? (uint32_t)v : 0u;
          uint32_t lo = __reduce_or_sync(0xffffffffu, (lane & 4) == 0 ? nibble << (8 * (lane & 3)) : 0u);
          uint32_t hi = __reduce_or_sync(0xffffffffu, (lane & 4) != 0 ? nibble << (8 * (lane & 3)) : 0u);
          if (lane == 0) {
            TileInfo& ti = sh.info[i % kInfo];
            ti.valid = (uint64_t)hi << 32 | lo;
            ti.flags = (t0 + t == 0 ? kFirst : 0u) | (t0 + t == s.tiles - 1 ? kLast : 0u);
            mbar_arrive_expect_tx(smem_u32(&sh.full[st]), 2u * pb * __popc(have >> (8 * t) & 0xffu));
          }
          __syncwarp();
          if ((lane >> 3) == t && (heads >> lane & 1u)) {
            const uint32_t dst = ring + st * stage_bytes + (lane & 7) * pb;
            bulk_load(dst, a.k_pool + now * pb, run * pb, smem_u32(&sh.full[st]));
            bulk_load(dst + side, a.v_pool + now * pb, run * pb, smem_u32(&sh.full[st]));
          }
          if (++st == (uint32_t)stages) st = 0, ph ^= 1u;
        }
        if (t0 == 0 && ok) {
          // Q of the segment: rows of 16 lanes, 8 dims each, as halves (128-byte swizzle)
          const uint32_t qb = seg % C::kQ;
          if (!(ok = wait(sh.q_empty[qb], (seg / C::kQ) ^ 1u, 10u))) break;
          const int c = lane & 15, half = lane >> 4;
          const float scale = a.scale_log2 * exp2i(head_exp(a.k_exp, s.h));
#pragma unroll 1
          for (int r0 = 0; r0 < N; r0 += 16) {
            uint4 w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int r = r0 + 2 * u + half;
              w[u] = make_uint4(0, 0, 0, 0);
              if (r < rows && c < 2 * groups)
                w[u] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                             row_at(a, s.b, s.h, row0 + r) * a.d) + c);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int r = r0 + 2 * u + half;
              const uint32_t ww[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
              float y[8], top = 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[2 * e] = __uint_as_float(ww[e] << 16);
                y[2 * e + 1] = __uint_as_float(ww[e] & 0xffff0000u);
                top = fmaxf(top, fmaxf(fabsf(y[2 * e]), fabsf(y[2 * e + 1])));
              }
#pragma unroll
              for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              // the power of two that takes top into [2^14, 2^15)
              const int e2 = (int)(__float_as_uint(top) >> 23);
              const int up = e2 == 0 || e2 == 255 ? 0 : min(100, 127 + 14 - e2);
              const float k = exp2i(up);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] *= k;
              sts128(q_base + qb * C::kQBytes + (c >> 3) * (N * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                     pack_f16(y[0], y[1]), pack_f16(y[2], y[3]), pack_f16(y[4], y[5]), pack_f16(y[6], y[7]));
              if (c == 0) sh.f[seg % kSegs][r] = scale * exp2i(-up);
            }
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.q_full[qb]));
        }
      }
    }
    if (flags) atomicOr(a.status, flags);
    if (sh.abort) {  // copies in flight end before the CTA does
      for (uint32_t k = 0; k < (uint32_t)stages && k < i; ++k) {
        const uint32_t j = i - 1 - k;
        mbar_wait_drain(smem_u32(&sh.full[j % stages]), (j / stages) & 1u);
      }
    }
  } else {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t id_s = idesc_f16(N, false), id_o = idesc_f16(N, true);
    const uint64_t dq = tc::smem_desc(q_base, 16, 1024);
    const uint64_t dp = tc::smem_desc(p_base, kKeys * 128, 1024);
    const uint32_t lead = elect_lead();
    uint32_t seg_s = 0, seg_o = 0;  // segments begun by S and by O
    bool ok = true;
    auto issue_s = [&](uint32_t i) {
      if (!wait(sh.k_full[i & 1], i >> 1, 11u)) return false;
      const uint32_t flags = sh.info[i % kInfo].flags;
      const uint32_t sb = i % C::kS, qb = seg_s % C::kQ;
      if ((flags & kFirst) && !wait(sh.q_full[qb], seg_s / C::kQ, 12u)) return false;
      if (!wait(sh.s_empty[sb], (i / C::kS) ^ 1u, 13u)) return false;
      tc::fence_after();
      const uint64_t q = dq + (uint64_t)(qb * (C::kQBytes >> 4));
#pragma unroll
      for (int kk = 0; kk < (DG ? DG : 8); ++kk)
        if (DG || kk < groups)
          lead_mma_ts(lead, tmem + kColS + sb * 64, tmem + kColK + (i & 1) * 64 + kk * 8,
                      q + (uint64_t)(((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4), id_s, kk > 0 ? 1u : 0u);
      lead_commit(lead, smem_u32(&sh.s_full[sb]));
      lead_commit(lead, smem_u32(&sh.k_empty[i & 1]));
      if (flags & kLast) {
        lead_commit(lead, smem_u32(&sh.q_empty[qb]));
        ++seg_s;
      }
      return true;
    };
    auto issue_o = [&](uint32_t i) {
      if (!wait(sh.v_full[i & 1], i >> 1, 14u)) return false;
      const bool first = sh.info[i % kInfo].flags & kFirst;
      if (first) {
        if (!wait(sh.o_empty, seg_o ^ 1u, 15u)) return false;
        ++seg_o;
      }
      if (!wait(sh.p_full[i & 1], i >> 1, 16u)) return false;
      tc::fence_after();
      const uint64_t p = dp + (uint64_t)((i & 1) * (C::kPBytes >> 4));
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk)
        lead_mma_ts(lead, tmem + kColO, tmem + kColV + (i & 1) * 64 + kk * 8, p + (uint64_t)((kk * 2048) >> 4),
                    id_o, first && kk == 0 ? 0u : 1u);
      lead_commit(lead, smem_u32(&sh.pv_done[i & 1]));
      return true;
    };
    if (tiles > 0) ok = issue_s(0);
    for (uint32_t i = 0; ok && i < tiles; ++i) {
      // with one S buffer the next S waits for this tile's weights, else it goes ahead of them
      if (i + 1 < tiles && !(ok = issue_s(i + 1))) break;
      ok = issue_o(i);
    }
    if (!ok) {  // products in flight end before TMEM is given back
      lead_commit(lead, smem_u32(&sh.drained));
      mbar_wait_drain(smem_u32(&sh.drained), 0);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == C::kMmaWarp) {
    tc::relinquish();
    tc::dealloc(tmem, kTmemCols);
  }
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
  return launch_pdl(attend4_tc_kernel<N, DG>, dim3(a.ctas), dim3(C::kThreads), (size_t)kMost, st, a, stages);
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
  a.ppt = kPieces;
  a.ctas = std::min(kMaxTc4Ctas, sm_count());
  const cudaError_t e = a.rows <= 16   ? launch_n<16>(a, st)
                        : a.rows <= 32 ? launch_n<32>(a, st)
                        : a.rows <= 64 ? launch_n<64>(a, st)
                                       : launch_n<128>(a, st);
  return e == cudaSuccess ? launch_join4(a, SV_BF16, st) : e;
}

}  // namespace sva
