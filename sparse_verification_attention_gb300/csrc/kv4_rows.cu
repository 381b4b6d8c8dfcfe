// Rows into the pages of a 4-bit cache and back, and the representatives of
// its blocks.
#include "kv4.cuh"

namespace sva {
namespace {

using namespace kv4;

constexpr int kThreads = 256;  // of the representatives
constexpr int kRowThreads = 64;
constexpr int kGroup = 16;  // dims that share a scale

// 16 elements of bf16 or fp32, in 32-byte accesses where the rows allow it (`wide`): in two
// halves every sector is asked for, or written, twice. (Loads past L1, as with __ldcg.)
template <typename T>
__device__ __forceinline__ void load16(const T* p, bool wide, float (&x)[16]) {
  uint32_t w[4 * sizeof(T)];
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); i += 2) {
    uint32_t* v = w + 4 * i;
    const uint4* q = reinterpret_cast<const uint4*>(p) + i;
    if (wide) {
      asm volatile("ld.relaxed.gpu.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                   : "l"(q));
    } else {
      const uint4 a = __ldcg(q), b = __ldcg(q + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
    else x[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}
template <typename T>
__device__ __forceinline__ void store16(T* p, bool wide, const float (&x)[16]) {
  uint32_t w[4 * sizeof(T)];
#pragma unroll
  for (int i = 0; i < (int)(4 * sizeof(T)); ++i)
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
    else w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); i += 2) {
    const uint32_t* v = w + 4 * i;
    uint4* q = reinterpret_cast<uint4*>(p) + i;
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                   "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                   : "memory");
    } else {
      q[0] = make_uint4(v[0], v[1], v[2], v[3]);
      q[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
}

// A lane has one group of one token, in `heads` heads one after the other; a warp 16
// tokens and two neighbouring groups, so that rows are read in runs of 64 bytes, K codes
// written in runs of 128 and the bytes of a V code row in runs of 16 when the tokens'
// slots follow each other (nothing depends on it). Blocks: 16 tokens (x), a pair of groups
// of K in one warp and of V in the other (y), heads (z). Places are worked out once for all heads:
// one head a lane, with its divisions, took 347 instructions a group. 13,343 rows of 8 heads
// of 128 in bf16: 18 us written and 13 read back, 4.5 TB/s. (All heads and four pairs of groups in a
// block, whose last wave is a fifth: 31.7 us for both; two heads at a time, in more registers, 34.4.)
struct Place {
  int token, g, is_v, tok, h0, h1;
  long long step;  // from a head's piece to the next head's
  uint8_t* piece;  // of head h0; null: nothing to do
};
__device__ __forceinline__ Place place_of(const Rows4Args& a) {
  const int lane = threadIdx.x & 31, groups = a.d / kGroup;
  Place p;
  p.token = blockIdx.x * 16 + (lane >> 1);
  p.is_v = threadIdx.x >= 32;
  p.g = blockIdx.y * 2 + (lane & 1);
  p.h0 = blockIdx.z * a.heads;
  p.h1 = min(p.h0 + a.heads, a.Hkv);
  p.piece = nullptr;
  p.tok = 0;
  p.step = (long long)(a.blk / kPiece) * piece_bytes(a.d);
  pdl_wait();
  pdl_trigger();
  if (p.token >= a.n || p.g >= groups) return p;
  const int slot = a.slots[p.token];
  const int page = slot < 0 ? -1 : (int)((unsigned)slot / (unsigned)a.blk);
  if (page < 0 || page >= a.num_pages) {
    if (slot != -1 && p.h0 == 0 && p.g == 0 && a.status) atomicOr(a.status, SV_FLAG_BAD_PAGE);
    return p;
  }
  const int in = slot - page * a.blk;
  p.tok = in % kPiece;
  p.piece = (p.is_v ? a.v_pool : a.k_pool) + ((long long)page * a.Hkv + p.h0) * p.step +
            (in / kPiece) * piece_bytes(a.d);
  return p;
}

// Rounding: the scale of a group is amax / 6 to the nearest E4M3 value, a code the
// nearest E2M1 value of x / (scale 2^exp). Quotients in 32 bits never move one onto a
// border between two codes or over it: a border times a scale has at most seven
// significant bits, so an x that is not on the border differs from it by a unit in its last
// place at least, 2^-23 / 1.875 relatively, and the quotient by more than half a unit. x times
// the reciprocal is off by up to two units; one step of Newton's on the quotient, whose
// remainder x - q s the fma gives exactly, leaves 2^-45 before the last rounding.
// (With a division each a group took 550 instructions, and 13,343 rows of 8 heads 33 us.)
template <typename T, bool IS_V>
__device__ __forceinline__ void write_groups(const Rows4Args& a, const Place& p) {
  const T* from = static_cast<const T*>(IS_V ? a.v : a.k) + p.token * (IS_V ? a.v_stride : a.k_stride) +
                  (long long)p.h0 * a.d + p.g * kGroup;
  uint8_t *codes = p.piece + p.g * 128 + (IS_V ? p.tok : p.tok * 8),
          *scale = p.piece + 8 * a.d + (IS_V ? p.g * 16 + p.tok : p.tok * (a.d / kGroup) + p.g);
#pragma unroll 1
  for (int h = p.h0; h < p.h1; ++h, from += a.d, codes += p.step, scale += p.step) {
    float x[16];
    load16(from, a.wide, x);
    const int e = head_exp(IS_V ? a.v_exp : a.k_exp, h);
    uint32_t top = 0;  // magnitudes compare as integers, a NaN's above all
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    const float amax = __uint_as_float(top) * exp2i(-e);
    const uint32_t sb = top > 0x7f800000u ? 0x7fu : f32_to_e4m3(__fdiv_rn(amax, 6.f));
    const float s = e4m3_to_f32(sb) * exp2i(e);
    if (amax > 6.5f * 448.f) {  // beyond the largest code: no infinities below
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = fminf(fmaxf(x[i], -8.f * s), 8.f * s);
    }
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float q = x[i] * r;
      x[i] = __fmaf_rn(__fmaf_rn(-q, s, x[i]), r, q);
    }
    if (IS_V) {
#pragma unroll
      for (int j = 0; j < 8; ++j) codes[j * 16] = (uint8_t)f32x2_to_e2m1x2(x[j], x[j + 8]);
    } else {
      uint32_t c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = f32x2_to_e2m1x2(x[2 * j], x[2 * j + 1]);
      const uint32_t lo = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, hi = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
      *reinterpret_cast<uint2*>(codes) = make_uint2(lo, hi);
    }
    *scale = (uint8_t)sb;
  }
}
template <typename T>
__global__ void __launch_bounds__(kRowThreads) write_kv4_kernel(const __grid_constant__ Rows4Args a) {
  const Place p = place_of(a);
  if (!p.piece) return;
  if (p.is_v) write_groups<T, true>(a, p);
  else write_groups<T, false>(a, p);
}

template <typename T, bool IS_V>
__device__ __forceinline__ void read_groups(const Rows4Args& a, const Place& p) {
  T* to = static_cast<T*>(IS_V ? a.v_out : a.k_out) + p.token * (IS_V ? a.v_stride : a.k_stride) +
          (long long)p.h0 * a.d + p.g * kGroup;
  const uint8_t *codes = p.piece + p.g * 128 + (IS_V ? p.tok : p.tok * 8),
                *scale = p.piece + 8 * a.d + (IS_V ? p.g * 16 + p.tok : p.tok * (a.d / kGroup) + p.g);
#pragma unroll 1
  for (int h = p.h0; h < p.h1; ++h, to += a.d, codes += p.step, scale += p.step) {
    uint32_t w[2], f16[8];
    const float s = e4m3_to_f32(__ldcg(scale)) * exp2i(head_exp(IS_V ? a.v_exp : a.k_exp, h));
    if (IS_V) {
      uint32_t c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = __ldcg(codes + j * 16);
      w[0] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
      w[1] = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
    } else {
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(codes));
      w[0] = v.x;
      w[1] = v.y;
    }
    e2m1x8_to_f16(w[0], f16);
    e2m1x8_to_f16(w[1], f16 + 4);
    float x[16];  // (V: byte j holds dims j and j + 8)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = f16x2_to_f32(f16[j]);
      x[IS_V ? j : 2 * j] = f.x * s;
      x[IS_V ? j + 8 : 2 * j + 1] = f.y * s;
    }
    store16(to, a.wide, x);
  }
}
template <typename T>
__global__ void __launch_bounds__(kRowThreads) read_kv4_kernel(const __grid_constant__ Rows4Args a) {
  const Place p = place_of(a);
  if (!p.piece) return;
  if (p.is_v) read_groups<T, true>(a, p);
  else read_groups<T, false>(a, p);
}

// One warp per (sequence, block) and a few of its heads: a lane has a group of 4 tokens of
// every piece (so 16 sums), 8 groups side by side (those of d > 128 in two rounds). The four
// token subsets are folded at the end, always in the same order.
//
// Code times scale is exact in f16. What costs is to sum halves in fp32: a conversion each
// and an addition, 62 us for 5,102 blocks of 8 heads. A product with the identity does it
// instead: in m16n8k16 a lane's A registers lie at the rows and columns of its four sums and
// at those 8 columns behind, so S += A (I above I) adds two tokens' halves to the lane's own
// sums. (A NaN reaches the sums in its row of 4 lanes, which are the same dims of the group's
// other tokens. The tensor cores' fp32 sums may be cut off where an addition rounds: a step, not
// half of one, of each of the blk / 4 sums that a lane adds up.)
// The same blocks: 51 us with one head a warp, whose lengths, page and places took as many
// instructions as a third of its sums (72% of the issue slots, HBM at 0.6 of its rate); 41.7 us
// now, 5.0 TB/s. Five CTAs an SM; six spill (44.7), four 42.8.
constexpr int kSlot = 4608;  // bytes of a block that a warp has under way together, at most
// DG: groups of 16 dims (8: d = 128), 0: any number.
template <int DG>
__global__ void __launch_bounds__(kThreads, 5) reps_kv4_kernel(const __grid_constant__ Reps4Args a) {
  __shared__ __align__(16) uint8_t slots[kThreads / 32][kSlot];
  const uint32_t slot = smem_u32(slots[threadIdx.x >> 5]);
  const int lane = threadIdx.x & 31, sub = lane & 3;
  const int jb = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.Hkv), b = blockIdx.z;
  pdl_wait();
  pdl_trigger();
  const int most = a.nb_max * a.blk, len0 = a.seq_ctx[b], from0 = a.from_len ? a.from_len[b] : 0;
  const int len = min(max(len0, 0), most), from = min(max(from0, 0), most);
  if (threadIdx.x == 0 && h0 == 0 && blockIdx.x == 0 && a.status && (len != len0 || from != from0))
    atomicOr(a.status, SV_FLAG_BAD_LENGTH);
  const int j = (a.blk_shift >= 0 ? from >> a.blk_shift : quotient(from, a.blk)) + jb;
  if (jb >= a.max_blocks || j >= (a.blk_shift >= 0 ? len >> a.blk_shift : quotient(len, a.blk))) return;
  const int page = a.block_table[(long long)b * a.nb_max + j];
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0 && a.status) atomicOr(a.status, SV_FLAG_BAD_PAGE);
    return;
  }
  const int groups = DG ? DG : a.d / kGroup, pb = piece_bytes(groups * kGroup), pieces = a.blk / kPiece;
  const int chunk = DG ? kSlot / piece_bytes(DG * kGroup) : quotient(kSlot, pb);  // pieces
  const uint8_t* p = a.k_pool + ((long long)page * a.Hkv + h0) * pieces * pb + lane * 16;
  float* to = a.reps + (((long long)b * a.Hkv + h0) * a.nb_max + j) * (groups * kGroup) + sub * 4;
  const float inv = __fdiv_rn(1.f, (float)a.blk);
  // B: rows 2 sub and 2 sub + 1 of column lane / 4, and the same 8 rows below
  const uint32_t identity = (lane >> 2 == 2 * sub ? 0x3c00u : 0u) | (lane >> 2 == 2 * sub + 1 ? 0x3c000000u : 0u);
#pragma unroll 1
  for (int h = h0; h < h1; ++h, p += pieces * pb, to += (long long)a.nb_max * (groups * kGroup)) {
    const int e = head_exp(a.k_exp, h);
#pragma unroll 1
    for (int g0 = 0; g0 < groups; g0 += 8) {
      const int g = DG ? lane >> 2 : min(g0 + (lane >> 2), groups - 1);  // (behind the last: not stored)
      float sum[4][4] = {};  // dims 4 i .. 4 i + 3
#pragma unroll 1
      for (int t0 = 0; t0 < pieces; t0 += chunk) {
        const int n = min(chunk, pieces - t0);
        if (pieces > chunk || g0 == 0) {
          __syncwarp();
          const uint8_t* src = p + (long long)t0 * pb;
          const int bytes = n * pb;
          for (int i = lane * 16; i < bytes; i += 512, src += 512)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + i), "l"(src) : "memory");
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
        }
        // (groups with odd numbers take their tokens the other way round: 8 lanes' loads fall
        // into different banks)
        const uint32_t odd = (uint32_t)g & 1u;
        uint32_t c0 = slot + g * 128 + sub * 32 + odd * 16, c1 = c0 + 16 - odd * 32;
        uint32_t s0 = slot + groups * 128 + sub * 4 * groups + g + odd * 2 * groups, s1 = s0 + 2 * groups - odd * 4 * groups;
#pragma unroll 1
        for (int t = 0; t < n; ++t, c0 += pb, c1 += pb, s0 += pb, s1 += pb) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // two tokens
            const uint4 c = lds128(k ? c1 : c0);
            uint32_t f[2][8], s, unused;
            e4m3x4_to_f16(lds8(k ? s1 : s0) | lds8((k ? s1 : s0) + groups) << 8, s, unused);
            e2m1x8_to_f16(c.x, f[0]);
            e2m1x8_to_f16(c.y, f[0] + 4);
            e2m1x8_to_f16(c.z, f[1]);
            e2m1x8_to_f16(c.w, f[1] + 4);
            scale_f16x2<0>(f[0], s);
            scale_f16x2<1>(f[1], s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile(
                  "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%8}, {%0,%1,%2,%3};"
                  : "+f"(sum[i][0]), "+f"(sum[i][1]), "+f"(sum[i][2]), "+f"(sum[i][3])
                  : "r"(f[0][2 * i]), "r"(f[0][2 * i + 1]), "r"(f[1][2 * i]), "r"(f[1][2 * i + 1]), "r"(identity));
          }
        }
      }
      // fold: the lane keeps 4 of the 16 sums of its group
      float x[8], y[4];
      const bool up2 = sub & 2, up1 = sub & 1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float lo = sum[i / 4][i % 4], hi = sum[2 + i / 4][i % 4];
        x[i] = (up2 ? hi : lo) + __shfl_xor_sync(0xffffffffu, up2 ? lo : hi, 2);
      }
      const float unit = inv * exp2i(e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[i] = ((up1 ? x[4 + i] : x[i]) + __shfl_xor_sync(0xffffffffu, up1 ? x[i] : x[4 + i], 1)) * unit;
      if (DG || g0 + (lane >> 2) < groups) *reinterpret_cast<float4*>(to + g * kGroup) = make_float4(y[0], y[1], y[2], y[3]);
    }
  }
}

bool wide_rows(const void* p, long long stride, int elt) {
  return reinterpret_cast<uintptr_t>(p) % 32 == 0 && stride * elt % 32 == 0;
}

// Heads in as many blocks as keep the GPU busy to the end (eight times as many lose more by
// working out places than the last wave costs; one pair of groups a block and not four:
// 64 tokens of 8 heads written and read 4.0 us, not 5.2).
template <typename F>
cudaError_t launch_rows(Rows4Args a, cudaStream_t st, F kernel) {
  const unsigned x = (unsigned)((a.n + 15ll) / 16), y = (unsigned)(a.d / kGroup + 1) / 2;
  int z = 1;
  while (z < a.Hkv && (long long)x * y * z < 32 * 152) z *= 2;
  a.heads = (a.Hkv + z - 1) / z;
  const dim3 grid(x, y, (unsigned)((a.Hkv + a.heads - 1) / a.heads));
  return launch_pdl(kernel, grid, dim3(kRowThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_write_kv4(Rows4Args a, int dtype, cudaStream_t st) {
  const int elt = dtype == SV_BF16 ? 2 : 4;
  a.wide = wide_rows(a.k, a.k_stride, elt) && wide_rows(a.v, a.v_stride, elt);
  return dtype == SV_BF16 ? launch_rows(a, st, write_kv4_kernel<__nv_bfloat16>) : launch_rows(a, st, write_kv4_kernel<float>);
}

cudaError_t launch_read_kv4(Rows4Args a, int dtype, cudaStream_t st) {
  const int elt = dtype == SV_BF16 ? 2 : 4;
  a.wide = wide_rows(a.k_out, a.k_stride, elt) && wide_rows(a.v_out, a.v_stride, elt);
  return dtype == SV_BF16 ? launch_rows(a, st, read_kv4_kernel<__nv_bfloat16>) : launch_rows(a, st, read_kv4_kernel<float>);
}

cudaError_t launch_reps_kv4(Reps4Args a, cudaStream_t st) {
  const unsigned x = (unsigned)((a.max_blocks + kThreads / 32 - 1) / (kThreads / 32));
  a.blk_shift = a.blk & (a.blk - 1) ? -1 : __builtin_ctz(a.blk);
  // a block's heads one after the other (what is worked out for the block counts once), in as
  // many CTAs as the GPU takes
  int y = 1;
  while (y < a.Hkv && (long long)x * y * a.B < 8 * 152) y *= 2;
  a.heads = (a.Hkv + y - 1) / y;
  const dim3 grid(x, (unsigned)((a.Hkv + a.heads - 1) / a.heads), (unsigned)a.B);
  return launch_pdl(a.d == 128 ? reps_kv4_kernel<8> : reps_kv4_kernel<0>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace sva
