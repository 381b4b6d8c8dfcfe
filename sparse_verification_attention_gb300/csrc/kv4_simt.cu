// Attention over a 4-bit cache on the CUDA cores, for every type and shape: keys
// and values are taken apart into 32-bit tiles in shared memory, all sums are fp32.
// The path of fp32 and of head dims above 128.
//
// A tile of 64 keys and 32 rows: a thread has 2 rows and 4 keys of the scores, 2 rows and
// 4 dims (in every 64) of the outputs. Bound by shared memory (12 wavefronts a warp for 4 dims of
// the scores) where contexts are long, by the latency of one round and its cold code where
// they are short: 5 sequences of 0 to 1500 tokens, 4 heads of 64, 18 us a call.
#include <algorithm>
#include <atomic>

#include "kv4.cuh"

namespace sva {
namespace {

using namespace kv4;

constexpr int kThreads = 256;
constexpr int kRows = kSimt4Rows;
constexpr int kKeys = 64, kPieces = kKeys / kPiece;  // (ppt_shift)
constexpr int kGroup = 16;

struct Control {
  Line line;
  long long piece[kPieces];
  int valid[kPieces];
  float m[kRows], l[kRows];
};

__host__ __device__ constexpr int tile_stride(int d) { return d + 4; }  // floats
size_t smem_bytes(int d) {
  return sizeof(Control) + sizeof(float) * (kRows * d + kKeys * tile_stride(d) + kRows * (kKeys + 1));
}

template <typename T>
__device__ __forceinline__ float as_float(T x) {
  if constexpr (sizeof(T) == 4) return x;
  else return __bfloat162float(x);
}

// D4: float4 columns of d per thread, ceil(d / 64).
template <typename T, int D4>
__global__ void __launch_bounds__(kThreads) attend4_simt_kernel(const __grid_constant__ Attend4Args a) {
  extern __shared__ float4 smem4[];
  float* q = reinterpret_cast<float*>(smem4);           // [kRows][d], times scale
  float* kv = q + kRows * a.d;                          // [kKeys][stride]
  float* p = kv + kKeys * tile_stride(a.d);             // [kRows][kKeys + 1]
  Control& sh = *reinterpret_cast<Control*>(p + kRows * (kKeys + 1));
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int stride = tile_stride(a.d), groups = a.d / kGroup, pb = piece_bytes(a.d);
  const int inv = quotient(65535, groups) + 1;  // x * inv >> 16 = x / groups for x < 64, groups <= 16
  unsigned flags = 0;
  pdl_wait();
  pdl_trigger();
  if (tid < 32) {
    const bool bad = make_line(a, &sh.line);
    if (bad) flags |= SV_FLAG_BAD_LENGTH;
  }
  __syncthreads();
  const int pairs = a.B * a.Hkv * a.row_tiles, cta = blockIdx.x;
  for (int p = cta * kThreads + tid; p < pairs; p += gridDim.x * kThreads) a.slots[p] = slots_of(a, sh.line, p);
  const int end = sh.line.begin(cta + 1);
  for (int x = sh.line.begin(cta); x < end;) {
    const Segment s = segment_at(a, sh.line, x, end, cta);
    x = s.next;
    if (s.tiles == 0) continue;
    const int row0 = s.rt * a.rows, rows = min(a.rows, a.T * a.G - row0);
    const float scale = a.scale_log2 * exp2i(head_exp(a.k_exp, s.h));
#pragma unroll 1
    for (int r = ty; r < kRows; r += 16) {
      const T* from = static_cast<const T*>(a.q) + (r < rows ? row_at(a, s.b, s.h, row0 + r) : 0) * a.d;
      for (int c = tx; c < a.d; c += 16) q[r * a.d + c] = r < rows ? as_float(from[c]) * scale : 0.f;
    }
    // rows ty and ty + 16: reference and sum (the same in the row's 16 threads), outputs
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float4 o[2][D4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < D4; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int tile = s.tile0; tile < s.tile0 + s.tiles; ++tile) {
      __syncthreads();
      if (tid < kPieces) sh.piece[tid] = piece_at(a, s, tile * kPieces + tid, &sh.valid[tid], &flags);
      __syncthreads();
      // K: a thread takes 8 bytes (a group of a token) at a time
      for (int i = tid; i < kKeys * groups; i += kThreads) {
        const int key = i & 15, rest = i >> 4, pc = rest * inv >> 16, g = rest - pc * groups;
        float f[16];
        const bool on = key < sh.valid[pc];
        const uint8_t* piece = a.k_pool + (on ? sh.piece[pc] : 0) * pb;
        const uint2 w = on ? __ldcg(reinterpret_cast<const uint2*>(piece + g * 128 + key * 8)) : make_uint2(0, 0);
        const float sc = on ? e4m3_to_f32(__ldcg(piece + 8 * a.d + key * groups + g)) : 0.f;
        float* to = kv + (pc * kPiece + key) * stride + g * kGroup;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 v = f16x2_to_f32(e2m1x2_to_f16x2((j < 4 ? w.x : w.y) >> (j % 4 * 8) & 0xffu));
          f[2 * j] = v.x * sc;
          f[2 * j + 1] = v.y * sc;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          reinterpret_cast<float4*>(to)[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
      }
      __syncthreads();
      float sc[2][4] = {};
      for (int c = 0; c < a.d; c += 4) {
        const float4 q0 = *reinterpret_cast<const float4*>(q + ty * a.d + c);
        const float4 q1 = *reinterpret_cast<const float4*>(q + (ty + 16) * a.d + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 k = *reinterpret_cast<const float4*>(kv + (tx + 16 * j) * stride + c);
          sc[0][j] += q0.x * k.x + q0.y * k.y + q0.z * k.z + q0.w * k.w;
          sc[1][j] += q1.x * k.x + q1.y * k.y + q1.z * k.z + q1.w * k.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // key tx + 16 j is token tx of piece j
          if (tx >= sh.valid[j]) sc[i][j] = -INFINITY;
          mx = fmaxf(mx, sc[i][j]);
        }
#pragma unroll
        for (int off = 8; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float next = fmaxf(m[i], mx), base = next == -INFINITY ? 0.f : next;
        const float keep = exp2f(m[i] - base);
        m[i] = next;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(sc[i][j] - base);
          p[(ty + 16 * i) * (kKeys + 1) + tx + 16 * j] = e;
          sum += e;
        }
#pragma unroll
        for (int off = 8; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l[i] = l[i] * keep + sum;
#pragma unroll
        for (int j = 0; j < D4; ++j) {
          o[i][j].x *= keep;
          o[i][j].y *= keep;
          o[i][j].z *= keep;
          o[i][j].w *= keep;
        }
      }
      __syncthreads();
      // V: a thread takes one code row of a piece (two dims of 16 tokens) at a time; tokens that
      // do not count are zero whatever their bytes hold. (A byte at a time, with its loads one
      // after the other, took 6000 cycles a tile of 64 dims.)
      for (int i = tid; i < kPieces * groups * 8; i += kThreads) {
        const int c = i & 7, rest = i >> 3, pc = rest * inv >> 16, g = rest - pc * groups, valid = sh.valid[pc];
        uint4 w = make_uint4(0, 0, 0, 0), sv = w;
        if (valid > 0) {
          const uint8_t* piece = a.v_pool + sh.piece[pc] * pb;
          w = __ldcg(reinterpret_cast<const uint4*>(piece + g * 128 + c * 16));
          sv = __ldcg(reinterpret_cast<const uint4*>(piece + 8 * a.d + g * 16));
        }
        float* to = kv + pc * kPiece * stride + g * kGroup + c;
#pragma unroll
        for (int t = 0; t < kPiece; t += 4, to += 4 * stride) {
          uint32_t x[4], y[2];
          e2m1x8_to_f16(t == 0 ? w.x : t == 4 ? w.y : t == 8 ? w.z : w.w, x);
          e4m3x4_to_f16(t == 0 ? sv.x : t == 4 ? sv.y : t == 8 ? sv.z : sv.w, y[0], y[1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = f16x2_to_f32(x[e]), ss = f16x2_to_f32(y[e / 2]);
            const float sc = e % 2 ? ss.y : ss.x;
            to[e * stride] = t + e < valid ? v.x * sc : 0.f;
            to[e * stride + 8] = t + e < valid ? v.y * sc : 0.f;
          }
        }
      }
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < kKeys; ++k) {
        const float p0 = p[ty * (kKeys + 1) + k], p1 = p[(ty + 16) * (kKeys + 1) + k];
#pragma unroll
        for (int j = 0; j < D4; ++j) {
          const int c = tx * 4 + 64 * j;
          if (c >= a.d) continue;
          const float4 v = *reinterpret_cast<const float4*>(kv + k * stride + c);
          o[0][j].x += p0 * v.x, o[0][j].y += p0 * v.y, o[0][j].z += p0 * v.z, o[0][j].w += p0 * v.w;
          o[1][j].x += p1 * v.x, o[1][j].y += p1 * v.y, o[1][j].z += p1 * v.z, o[1][j].w += p1 * v.w;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = ty + 16 * i;
      if (r >= rows) continue;
      const long long at = (long long)s.slot * a.rows + r;
      if (tx == 0) a.part_ml[at] = make_float2(m[i], l[i]);
#pragma unroll
      for (int j = 0; j < D4; ++j)
        if (tx * 4 + 64 * j < a.d) *reinterpret_cast<float4*>(a.part_o + at * a.d + tx * 4 + 64 * j) = o[i][j];
    }
  }
  if (flags) atomicOr(a.status, flags);
}

template <typename T, int D4>
cudaError_t launch(const Attend4Args& a, cudaStream_t st) {
  static std::atomic<int> per_sm[kMaxDevices];  // resident CTAs at the widest head
  const int dev = current_device();
  const size_t most = smem_bytes(std::min(64 * D4, kMaxD));
  int n = per_sm[dev].load();
  if (n == 0) {
    cudaError_t e = cudaFuncSetAttribute(attend4_simt_kernel<T, D4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)most);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attend4_simt_kernel<T, D4>, kThreads, most);
    if (e != cudaSuccess) return e;
    per_sm[dev].store(n = std::max(n, 1));
  }
  Attend4Args b = a;
  b.ctas = std::min(kMaxSimt4Ctas, sm_count() * n);
  const cudaError_t e = launch_pdl(attend4_simt_kernel<T, D4>, dim3(b.ctas), dim3(kThreads), smem_bytes(a.d), st, b);
  return e == cudaSuccess ? launch_join4(b, sizeof(T) == 4 ? SV_F32 : SV_BF16, st) : e;
}

template <typename T>
cudaError_t launch_as(const Attend4Args& a, cudaStream_t st) {
  if (a.d <= 64) return launch<T, 1>(a, st);
  if (a.d <= 128) return launch<T, 2>(a, st);
  return launch<T, 4>(a, st);
}

}  // namespace

cudaError_t launch_attend4_simt(Attend4Args a, int dtype, cudaStream_t st) {
  a.rows = std::min(kRows, a.T * a.G);
  a.row_tiles = (a.T * a.G + a.rows - 1) / a.rows;
  a.ppt = kPieces;
  a.ppt_shift = 2;
  a.streams = 1;
  a.pair_cost = 1;
  return dtype == SV_BF16 ? launch_as<__nv_bfloat16>(a, st) : launch_as<float>(a, st);
}

}  // namespace sva
