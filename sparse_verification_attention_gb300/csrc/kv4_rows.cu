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
// other (nothing depends on it).
struct Place {
  const int32_t* slot;
  long long token;
  int h, g, is_v;
  bool ok;
};
__device__ __forceinline__ Place place_of(const Rows4Args& a) {
  const int lane = threadIdx.x & 31;
  const int groups = a.d / kGroup, cols = a.Hkv * groups * 2;  // K groups, then V groups
  const int pairs = (cols + 1) / 2;                            // pairs of groups
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long tb = w / pairs;
  int col = (int)(w - tb * pairs) * 2 + (lane & 1);
  Place p;
  p.token = tb * 16 + (lane >> 1);
  p.ok = p.token < a.n && col < cols;
  p.is_v = col >= a.Hkv * groups;
  col -= p.is_v ? a.Hkv * groups : 0;
  p.h = col / groups;
  p.g = col - p.h * groups;
  return p;
}
// The piece and token within it of a slot, or null.
__device__ __forceinline__ uint8_t* piece_of(const Rows4Args& a, const Place& p, int* tok) {
  const int slot = a.slots[p.token];
  const int page = slot < 0 ? -1 : slot / a.blk;
  if (page < 0 || page >= a.num_pages) {
    if (slot != -1 && p.h == 0 && p.g == 0 && a.status) atomicOr(a.status, SV_FLAG_BAD_PAGE);
    return nullptr;
  }
  const int in = slot - page * a.blk;
  *tok = in & (kPiece - 1);
  return (p.is_v ? a.v_pool : a.k_pool) +
         (((long long)page * a.Hkv + p.h) * (a.blk / kPiece) + in / kPiece) * piece_bytes(a.d);
}

// Rounding: the scale of a group is amax / 6 to the nearest E4M3 value, a code the
// nearest E2M1 value of element / scale. Both quotients are rounded correctly in 32
// bits, and that never moves one onto a border between two codes: a border times a
// scale has at most seven significant bits, so a 24-bit element differs from it by
// a unit in its last place at least, which is more than half a unit of the quotient.
template <typename T>
__global__ void __launch_bounds__(kThreads) write_kv4_kernel(const __grid_constant__ Rows4Args a) {
  const Place p = place_of(a);
  pdl_wait();
  pdl_trigger();
  if (!p.ok) return;
  int tok;
  uint8_t* piece = piece_of(a, p, &tok);
  if (!piece) return;
  float x[16];
  load16(static_cast<const T*>(p.is_v ? a.v : a.k) + p.token * (p.is_v ? a.v_stride : a.k_stride) +
             (long long)p.h * a.d + p.g * kGroup,
         x);
  const float unit = exp2i(-head_exp(p.is_v ? a.v_exp : a.k_exp, p.h));
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] *= unit;
    nan |= x[i] != x[i];
    amax = fmaxf(amax, fabsf(x[i]));
  }
  const uint32_t sb = nan ? 0x7fu : f32_to_e4m3(__fdiv_rn(amax, 6.f));
  const float s = e4m3_to_f32(sb);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = s > 0.f ? __fdiv_rn(x[i], s) : 0.f;
  uint8_t* codes = piece + p.g * 128;
  if (p.is_v) {
#pragma unroll
    for (int c = 0; c < 8; ++c) codes[c * 16 + tok] = (uint8_t)f32x2_to_e2m1x2(x[c], x[c + 8]);
    piece[8 * a.d + p.g * 16 + tok] = (uint8_t)sb;
  } else {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j / 4] |= f32x2_to_e2m1x2(x[2 * j], x[2 * j + 1]) << (j % 4 * 8);
    *reinterpret_cast<uint2*>(codes + tok * 8) = make_uint2(w[0], w[1]);
    piece[8 * a.d + tok * (a.d / kGroup) + p.g] = (uint8_t)sb;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) read_kv4_kernel(const __grid_constant__ Rows4Args a) {
  const Place p = place_of(a);
  pdl_wait();
  pdl_trigger();
  if (!p.ok) return;
  int tok;
  const uint8_t* piece = piece_of(a, p, &tok);
  if (!piece) return;
  const uint8_t* codes = piece + p.g * 128;
  float x[16];
  const float unit = exp2i(head_exp(p.is_v ? a.v_exp : a.k_exp, p.h));
  const float s =
      e4m3_to_f32(__ldcg(piece + 8 * a.d + (p.is_v ? p.g * 16 + tok : tok * (a.d / kGroup) + p.g))) * unit;
  if (p.is_v) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float2 f = f16x2_to_f32(e2m1x2_to_f16x2(__ldcg(codes + c * 16 + tok)));
      x[c] = f.x * s;
      x[c + 8] = f.y * s;
    }
  } else {
    const uint2 v = __ldcg(reinterpret_cast<const uint2*>(codes + tok * 8));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = f16x2_to_f32(e2m1x2_to_f16x2((j < 4 ? v.x : v.y) >> (j % 4 * 8) & 0xffu));
      x[2 * j] = f.x * s;
      x[2 * j + 1] = f.y * s;
    }
  }
  store16(static_cast<T*>(p.is_v ? a.v_out : a.k_out) + p.token * (p.is_v ? a.v_stride : a.k_stride) +
              (long long)p.h * a.d + p.g * kGroup,
          x);
}

// One warp per (sequence, head, block): lanes are groups x token subsets, 16 sums a
// lane, the subsets folded at the end (always in the same order).
__global__ void __launch_bounds__(kThreads) reps_kv4_kernel(const __grid_constant__ Reps4Args a, int gp) {
  const int lane = threadIdx.x & 31, g = lane & (gp - 1), sub = lane / gp, subs = 32 / gp;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  const long long bh = w / a.max_blocks;
  const int b = (int)(bh / a.Hkv), h = (int)(bh - (long long)b * a.Hkv);
  if (b >= a.B) return;
  const int most = a.nb_max * a.blk;
  const int len = min(max(a.seq_ctx[b], 0), most), from = a.from_len ? min(max(a.from_len[b], 0), most) : 0;
  if (lane == 0 && h == 0 && w == bh * a.max_blocks && a.status &&
      (len != a.seq_ctx[b] || (a.from_len && from != a.from_len[b])))
    atomicOr(a.status, SV_FLAG_BAD_LENGTH);
  const int j = from / a.blk + (int)(w - bh * a.max_blocks);
  if (j >= len / a.blk) return;
  const int page = a.block_table[(long long)b * a.nb_max + j];
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0 && a.status) atomicOr(a.status, SV_FLAG_BAD_PAGE);
    return;
  }
  const int groups = a.d / kGroup, pb = piece_bytes(a.d);
  const uint8_t* p = a.k_pool + ((long long)page * a.Hkv + h) * (a.blk / kPiece) * pb;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
  if (g < groups) {
    for (int t = sub; t < a.blk; t += subs) {
      const uint8_t* piece = p + (t / kPiece) * pb;
      const int tok = t % kPiece;
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(piece + g * 128 + tok * 8));
      const float s = e4m3_to_f32(__ldcg(piece + 8 * a.d + tok * groups + g));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = f16x2_to_f32(e2m1x2_to_f16x2((i < 4 ? v.x : v.y) >> (i % 4 * 8) & 0xffu));
        x[2 * i] += f.x * s;
        x[2 * i + 1] += f.y * s;
      }
    }
  }
  for (int o = 16; o >= gp; o >>= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
  if (sub || g >= groups) return;
  const float unit = exp2i(head_exp(a.k_exp, h));
  float* to = a.reps + (((long long)b * a.Hkv + h) * a.nb_max + j) * a.d + g * kGroup;
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i] * unit, (float)a.blk);
  store16(to, x);
}

unsigned row_blocks(const Rows4Args& a) {
  const long long pairs = (long long)a.Hkv * (a.d / kGroup);
  const long long warps = (a.n + 15ll) / 16 * pairs;
  return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
}

}  // namespace

cudaError_t launch_write_kv4(const Rows4Args& a, int dtype, cudaStream_t st) {
  const dim3 grid(row_blocks(a)), block(kThreads);
  return dtype == SV_BF16 ? launch_pdl(write_kv4_kernel<__nv_bfloat16>, grid, block, 0, st, a)
                          : launch_pdl(write_kv4_kernel<float>, grid, block, 0, st, a);
}

cudaError_t launch_read_kv4(const Rows4Args& a, int dtype, cudaStream_t st) {
  const dim3 grid(row_blocks(a)), block(kThreads);
  return dtype == SV_BF16 ? launch_pdl(read_kv4_kernel<__nv_bfloat16>, grid, block, 0, st, a)
                          : launch_pdl(read_kv4_kernel<float>, grid, block, 0, st, a);
}

cudaError_t launch_reps_kv4(const Reps4Args& a, cudaStream_t st) {
  int gp = 1;
  while (gp < a.d / kGroup) gp <<= 1;
  const long long warps = (long long)a.B * a.Hkv * a.max_blocks;
  return launch_pdl(reps_kv4_kernel, dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32))),
                    dim3(kThreads), 0, st, a, gp);
}

}  // namespace sva
