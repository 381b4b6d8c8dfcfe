// Rows into the pages of a 4-bit cache and back, and the representatives of
// its blocks.
#include "kv4.cuh"

namespace sva {
namespace {

using namespace kv4;

constexpr int kThreads = 256;
constexpr int kGroup = 16;  // dims that share a scale

// 16 elements of bf16 or fp32.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]) {
  constexpr int kVecs = (int)sizeof(T);  // 16-byte vectors
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if constexpr (sizeof(T) == 4) {
        x[4 * i + j] = __uint_as_float(w[j]);
      } else {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
  }
}
template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(x[4 * i + j]);
      else w[j] = pack_bf16(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
    reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A lane has one group of one token's head; a warp 16 tokens and two neighbouring
// groups, so that rows are read in runs of 64 bytes, K codes written in runs of 128
// and the bytes of a V code row in runs of 16 when the tokens' slots follow each
// other (nothing depends on it). Blocks: 16 tokens (x), eight pairs of groups (y): those
// of K, then those of V.
struct Place {
  int token, h, g, is_v, tok;
  uint8_t* piece;  // null: nothing to do
};
__device__ __forceinline__ Place place_of(const Rows4Args& a) {
  const int lane = threadIdx.x & 31;
  const int groups = a.d / kGroup, cols = a.Hkv * groups;
  int col = (blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5)) * 2 + (lane & 1);
  Place p;
  p.token = blockIdx.x * 16 + (lane >> 1);
  p.is_v = col >= cols;
  col -= p.is_v ? cols : 0;
  p.h = (unsigned)col / (unsigned)groups;
  p.g = col - p.h * groups;
  p.piece = nullptr;
  p.tok = 0;
  pdl_wait();
  pdl_trigger();
  if (p.token >= a.n || col >= cols) return p;
  const int slot = a.slots[p.token];
  const int page = slot < 0 ? -1 : (int)((unsigned)slot / (unsigned)a.blk);
  if (page < 0 || page >= a.num_pages) {
    if (slot != -1 && p.h == 0 && p.g == 0 && a.status) atomicOr(a.status, SV_FLAG_BAD_PAGE);
    return p;
  }
  const int in = slot - page * a.blk;
  p.tok = in % kPiece;
  p.piece = (p.is_v ? a.v_pool : a.k_pool) +
            (((long long)page * a.Hkv + p.h) * (a.blk / kPiece) + in / kPiece) * piece_bytes(a.d);
  return p;
}

// Rounding: the scale of a group is amax / 6 to the nearest E4M3 value, a code the
// nearest E2M1 value of x / (scale 2^exp). Quotients in 32 bits never move one onto a
// border between two codes or over it: a border times a scale has at most seven
// significant bits, so an x that is not on the border differs from it by a unit in its last
// place at least, 2^-23 / 1.875 relatively, and the quotient by more than half a unit. x times
// the reciprocal is off by up to two units; one step of Newton's on the quotient, whose
// remainder x - q s the fma gives exactly, leaves 2^-45 before the last rounding.
// (A division each took 550 instructions a group, 33 us for 13,343 rows of 8 heads.)
template <typename T>
__global__ void __launch_bounds__(kThreads) write_kv4_kernel(const __grid_constant__ Rows4Args a) {
  const Place p = place_of(a);
  if (!p.piece) return;
  float x[16];
  load16(static_cast<const T*>(p.is_v ? a.v : a.k) + p.token * (p.is_v ? a.v_stride : a.k_stride) +
             (long long)p.h * a.d + p.g * kGroup,
         x);
  const int e = head_exp(p.is_v ? a.v_exp : a.k_exp, p.h);
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
  uint32_t c[8];  // dims 2 j, 2 j + 1 of K, j, j + 8 of V
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float q = x[i] * r;
    x[i] = __fmaf_rn(__fmaf_rn(-q, s, x[i]), r, q);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) c[j] = p.is_v ? f32x2_to_e2m1x2(x[j], x[j + 8]) : f32x2_to_e2m1x2(x[2 * j], x[2 * j + 1]);
  uint8_t* codes = p.piece + p.g * 128;
  if (p.is_v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) codes[j * 16 + p.tok] = (uint8_t)c[j];
    p.piece[8 * a.d + p.g * 16 + p.tok] = (uint8_t)sb;
  } else {
    const uint32_t lo = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, hi = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
    *reinterpret_cast<uint2*>(codes + p.tok * 8) = make_uint2(lo, hi);
    p.piece[8 * a.d + p.tok * (a.d / kGroup) + p.g] = (uint8_t)sb;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) read_kv4_kernel(const __grid_constant__ Rows4Args a) {
  const Place p = place_of(a);
  if (!p.piece) return;
  const uint8_t* codes = p.piece + p.g * 128;
  uint32_t w[2], h[8];
  const uint32_t sb = __ldcg(p.piece + 8 * a.d + (p.is_v ? p.g * 16 + p.tok : p.tok * (a.d / kGroup) + p.g));
  if (p.is_v) {
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = __ldcg(codes + j * 16 + p.tok);
    w[0] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
    w[1] = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
  } else {
    const uint2 v = __ldcg(reinterpret_cast<const uint2*>(codes + p.tok * 8));
    w[0] = v.x;
    w[1] = v.y;
  }
  e2m1x8_to_f16(w[0], h);
  e2m1x8_to_f16(w[1], h + 4);
  const float s = e4m3_to_f32(sb) * exp2i(head_exp(p.is_v ? a.v_exp : a.k_exp, p.h));
  float x[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = f16x2_to_f32(h[j]);
    x[2 * j] = f.x * s;
    x[2 * j + 1] = f.y * s;
  }
  if (p.is_v) {  // dims j, j + 8 stand side by side
    float y[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[2 * j], y[j + 8] = x[2 * j + 1];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = y[j];
  }
  store16(static_cast<T*>(p.is_v ? a.v_out : a.k_out) + p.token * (p.is_v ? a.v_stride : a.k_stride) +
              (long long)p.h * a.d + p.g * kGroup,
          x);
}

// x += the halves of h (low, high) times the half s, in fp32.
__device__ __forceinline__ void fma_f32_f16x2(float& x, float& y, uint32_t h, uint16_t s) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "fma.rn.f32.f16 %0, a, %3, %0;\n\t"
      "fma.rn.f32.f16 %1, b, %3, %1;\n\t}"
      : "+f"(x), "+f"(y)
      : "r"(h), "h"(s));
}

// One warp per (sequence, head, block): a lane has a group of 4 tokens of every piece (so
// 16 sums), `gp` lanes side by side the groups (those of d > 128 in two rounds). The four
// token subsets are folded at the end, always in the same order.
// Bound by HBM, and nearly as much by issue: the products are fp32 sums of halves.
__global__ void __launch_bounds__(kThreads) reps_kv4_kernel(const __grid_constant__ Reps4Args a) {
  const int lane = threadIdx.x & 31, sub = lane & 3;
  const int jb = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int h = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  pdl_trigger();
  const int most = a.nb_max * a.blk, len0 = a.seq_ctx[b], from0 = a.from_len ? a.from_len[b] : 0;
  const int len = min(max(len0, 0), most), from = min(max(from0, 0), most);
  if (threadIdx.x == 0 && h == 0 && blockIdx.x == 0 && a.status && (len != len0 || from != from0))
    atomicOr(a.status, SV_FLAG_BAD_LENGTH);
  const int j = from / a.blk + jb;
  if (jb >= a.max_blocks || j >= len / a.blk) return;
  const int page = a.block_table[(long long)b * a.nb_max + j];
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0 && a.status) atomicOr(a.status, SV_FLAG_BAD_PAGE);
    return;
  }
  const int groups = a.d / kGroup, pb = piece_bytes(a.d), pieces = a.blk / kPiece;
  const uint8_t* p = a.k_pool + ((long long)page * a.Hkv + h) * pieces * pb;
  const float unit = __fdiv_rn(exp2i(head_exp(a.k_exp, h)), (float)a.blk);
  float* to = a.reps + (((long long)b * a.Hkv + h) * a.nb_max + j) * a.d;
#pragma unroll 1
  for (int g0 = 0; g0 < groups; g0 += 8) {
    const int g = g0 + (lane >> 2);
    const bool on = g < groups;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    if (on) {
      const uint8_t *codes = p + g * 128 + sub * 32, *scales = p + 8 * a.d + sub * 4 * groups + g;
#pragma unroll 2
      for (int t = 0; t < pieces; ++t, codes += pb, scales += pb) {
        const uint4 c[2] = {__ldcg(reinterpret_cast<const uint4*>(codes)), __ldcg(reinterpret_cast<const uint4*>(codes) + 1)};
        const uint32_t sc = __ldcg(scales) | __ldcg(scales + groups) << 8 | __ldcg(scales + 2 * groups) << 16 |
                            (uint32_t)__ldcg(scales + 3 * groups) << 24;
        uint32_t s[2];
        e4m3x4_to_f16(sc, s[0], s[1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w0 = k % 2 ? c[k / 2].z : c[k / 2].x, w1 = k % 2 ? c[k / 2].w : c[k / 2].y;
          uint32_t f[8];
          e2m1x8_to_f16(w0, f);
          e2m1x8_to_f16(w1, f + 4);
          const uint16_t sk = (uint16_t)(k % 2 ? s[k / 2] >> 16 : s[k / 2]);
#pragma unroll
          for (int i = 0; i < 8; ++i) fma_f32_f16x2(x[2 * i], x[2 * i + 1], f[i], sk);
        }
      }
    }
    // fold: the lane keeps 4 of the 16 sums of its group
    float y[4];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] += __shfl_xor_sync(0xffffffffu, x[i], 1);
      x[i] += __shfl_xor_sync(0xffffffffu, x[i], 2);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = (sub == 0 ? x[i] : sub == 1 ? x[4 + i] : sub == 2 ? x[8 + i] : x[12 + i]) * unit;
    if (on) *reinterpret_cast<float4*>(to + g * kGroup + sub * 4) = make_float4(y[0], y[1], y[2], y[3]);
  }
}

dim3 row_grid(const Rows4Args& a) {
  const int pairs = a.Hkv * (a.d / kGroup);  // K and V: two groups each
  return dim3((unsigned)((a.n + 15ll) / 16), (unsigned)((pairs + kThreads / 32 - 1) / (kThreads / 32)));
}

}  // namespace

cudaError_t launch_write_kv4(const Rows4Args& a, int dtype, cudaStream_t st) {
  const dim3 block(kThreads);
  return dtype == SV_BF16 ? launch_pdl(write_kv4_kernel<__nv_bfloat16>, row_grid(a), block, 0, st, a)
                          : launch_pdl(write_kv4_kernel<float>, row_grid(a), block, 0, st, a);
}

cudaError_t launch_read_kv4(const Rows4Args& a, int dtype, cudaStream_t st) {
  const dim3 block(kThreads);
  return dtype == SV_BF16 ? launch_pdl(read_kv4_kernel<__nv_bfloat16>, row_grid(a), block, 0, st, a)
                          : launch_pdl(read_kv4_kernel<float>, row_grid(a), block, 0, st, a);
}

cudaError_t launch_reps_kv4(const Reps4Args& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.max_blocks + kThreads / 32 - 1) / (kThreads / 32)), (unsigned)a.Hkv, (unsigned)a.B);
  return launch_pdl(reps_kv4_kernel, grid, dim3(kThreads), 0, st, a);
}

}  // namespace sva
