// Attention over a 4-bit cache on the CUDA cores, for every type and shape: the path of
// fp32 and of head dims above 128. All sums are fp32.
//
// Neither K nor V passes through shared memory. Scores: a lane has a key and every fourth
// group of dims, and dots them with all rows of Q, which it reads with its whole warp; the
// four parts of a score meet in shared memory. Outputs: a thread has two dims (a code row of V, 16
// tokens a load) of some rows, and reads weights that its warp has in common. Rows are
// tiles of 4 to 32, the smallest that holds them.
//
// Bound by issue slots (a fifth of the scores' instructions are loads of Q, an eighth of the
// outputs' loads of weights): fp32, 16384 tokens, 32 rows of 8 heads of 128, 92 us, 23 TFLOP/s;
// bf16 heads of 256, 2 x 131072 tokens, 8 tokens each, 517 us, one, 155. K a tile ahead in
// registers gained nothing. Where contexts are short by the latency of one round: 5 sequences
// of 0 to 1500 tokens, 8 rows of 4 heads of 64, 14 us.
// (With K and V taken apart into 32-bit tiles in shared memory for both products: 123, 1264,
// 1260 and 18 us.)
#include <algorithm>
#include <atomic>

#include "kv4.cuh"

namespace sva {
namespace {

using namespace kv4;

constexpr int kThreads = 256;
constexpr int kKeys = 64, kPieces = kKeys / kPiece;  // (ppt_shift)
constexpr int kGroup = 16;
constexpr int kSlices = 4;  // warps that share a key's dims
static_assert(kThreads == kSlices * kKeys, "a lane a key and slice");

struct Control {
  Line line;
  long long piece[2][kPieces];  // of this tile and the next
  int valid[2][kPieces];
  float keep[kSimt4Rows];       // what a row's sums shrink by
  float unit;                   // of a segment's scores: Q times more than 1 may overflow where no score does
};

// Rows of p: keys, their lanes' rows in different banks.
template <int RT>
struct P {
  static constexpr int kStride = RT == 4 ? 4 : RT + 4;
};
template <int RT>
size_t smem_bytes(int d) {
  return sizeof(Control) + sizeof(float) * (RT * d + kSlices * kKeys * P<RT>::kStride);
}

// RT: rows of a tile at most. GR: groups of threads that share the tile's rows in the product
// with V (d / 2 threads each).
template <int RT, int GR>
__global__ void __launch_bounds__(kThreads, 2) attend4_simt_kernel(const __grid_constant__ Attend4Args a, int f32) {
  constexpr int PS = P<RT>::kStride, RG = RT < GR ? 1 : RT / GR;
  extern __shared__ float4 smem4[];
  float* q = reinterpret_cast<float*>(smem4);  // [RT][d], times scale
  float* p = q + RT * a.d;                     // [kSlices][kKeys][PS]: parts of scores; weights in the first
  Control& sh = *reinterpret_cast<Control*>(p + kSlices * kKeys * PS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = a.d / kGroup, pb = piece_bytes(a.d);
  unsigned flags = 0;
  pdl_wait();
  pdl_trigger();
  if (tid < 32 && make_line(a, &sh.line)) flags |= SV_FLAG_BAD_LENGTH;
  __syncthreads();
  const int pairs = a.B * a.Hkv * a.row_tiles, cta = blockIdx.x;
  for (int i = cta * kThreads + tid; i < pairs; i += gridDim.x * kThreads) a.slots[i] = slots_of(a, sh.line, i);
  // scores: key and every fourth group of dims; softmax: row and keys part + 8 j; outputs: rows
  // r0 .. and dims 16 vg + vc and 8 behind
  const int key = warp / kSlices * 32 + lane, slice = warp % kSlices, row = tid >> 3, part = tid & 7;
  const int vgrp = quotient(tid, a.d / 2), vx = tid - vgrp * (a.d / 2), vc = vx & 7, vg = vx >> 3, r0 = vgrp * RG;
  const bool has_v = vgrp < GR && r0 < RT, has_row = row < RT;
  const int end = sh.line.begin(cta + 1);
  for (int x = sh.line.begin(cta); x < end;) {
    const Segment s = segment_at(a, sh.line, x, end, cta);
    x = s.next;
    if (s.tiles == 0) continue;
    const int row0 = s.rt * a.rows, rows = min(a.rows, a.T * a.G - row0);
    const int k_exp = head_exp(a.k_exp, s.h);
    const float scale = a.scale_log2 * exp2i(min(k_exp, 0));
    __syncthreads();  // the segment before has read q and p
    if (tid == 0) sh.unit = exp2i(max(k_exp, 0));
#pragma unroll 1
    for (int r = warp; r < RT; r += kThreads / 32) {
      const long long from = (r < rows ? row_at(a, s.b, s.h, row0 + r) : 0) * a.d;
      for (int c = lane; c < a.d; c += 32) {
        float y = 0.f;
        if (r < rows) y = f32 ? static_cast<const float*>(a.q)[from + c] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[from + c]);
        q[r * a.d + c] = y * scale;
      }
    }
    auto look_up = [&](int tile) {
      if (tid < kPieces) sh.piece[tile & 1][tid] = piece_at(a, s, tile * kPieces + tid, &sh.valid[tile & 1][tid], &flags);
    };
    look_up(s.tile0);
    __syncthreads();
    float m = -INFINITY, l = 0.f;  // the row's reference and sum, the same in its 8 threads
    float o[RG][2];
#pragma unroll
    for (int i = 0; i < RG; ++i) o[i][0] = o[i][1] = 0.f;
#pragma unroll 1
    for (int tile = s.tile0; tile < s.tile0 + s.tiles; ++tile) {
      const long long* piece = sh.piece[tile & 1];
      const int* valid = sh.valid[tile & 1];
      {
        float acc[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = 0.f;
        const bool on = (key & 15) < valid[key >> 4];
        const uint8_t* from = a.k_pool + (on ? piece[key >> 4] : 0) * pb + (key & 15) * 8;
        const uint8_t* sc = a.k_pool + (on ? piece[key >> 4] : 0) * pb + 8 * a.d + (key & 15) * groups;
#pragma unroll(RT <= 8 ? 2 : 1)
        for (int g = slice; g < groups; g += kSlices) {
          uint2 w = make_uint2(0, 0);
          uint32_t e = 0;
          if (on) {
            w = __ldcg(reinterpret_cast<const uint2*>(from + g * 128));
            e = __ldcg(sc + g);
          }
          const float f = e4m3_to_f32(e);
          const float* qq = q + g * kGroup;
          uint32_t h[8];
          e2m1x8_to_f16(w.x, h);
          e2m1x8_to_f16(w.y, h + 4);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 k01 = f16x2_to_f32(h[2 * c]), k23 = f16x2_to_f32(h[2 * c + 1]);
            const float k0 = k01.x * f, k1 = k01.y * f, k2 = k23.x * f, k3 = k23.y * f;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const float4 y = *reinterpret_cast<const float4*>(qq + r * a.d + 4 * c);
              acc[r] = fmaf(y.x, k0, fmaf(y.y, k1, fmaf(y.z, k2, fmaf(y.w, k3, acc[r]))));
            }
          }
        }
        float4* to = reinterpret_cast<float4*>(p + (slice * kKeys + key) * PS);
        const float unit = sh.unit;
#pragma unroll
        for (int i = 0; i < RT; i += 4) to[i / 4] = make_float4(acc[i] * unit, acc[i + 1] * unit, acc[i + 2] * unit, acc[i + 3] * unit);
      }
      // V's bytes are on their way while the weights are made
      uint4 w[kPieces], sv[kPieces];
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        w[c] = sv[c] = make_uint4(0, 0, 0, 0);
        if (has_v && valid[c] > 0) {
          const uint8_t* from = a.v_pool + piece[c] * pb;
          w[c] = __ldcg(reinterpret_cast<const uint4*>(from + vg * 128 + vc * 16));
          sv[c] = __ldcg(reinterpret_cast<const uint4*>(from + 8 * a.d + vg * 16));
        }
      }
      __syncthreads();
      if (tile + 1 < s.tile0 + s.tiles) look_up(tile + 1);
      if (has_row) {
        float y[kKeys / 8], mx = m;
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) {
          const int k = part + 8 * j;
          const float* x = p + k * PS + row;
          y[j] = (k & 15) < valid[k >> 4] ? (x[0] + x[kKeys * PS]) + (x[2 * kKeys * PS] + x[3 * kKeys * PS]) : -INFINITY;
          mx = fmaxf(mx, y[j]);
        }
#pragma unroll
        for (int off = 4; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off, 8));
        const float base = mx == -INFINITY ? 0.f : mx, keep = exp2f(m - base);
        m = mx;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) {
          y[j] = exp2f(y[j] - base);
          p[(part + 8 * j) * PS + row] = y[j];
          sum += y[j];
        }
#pragma unroll
        for (int off = 4; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off, 8);
        l = l * keep + sum;
        if (part == 0) sh.keep[row] = keep;
      }
      __syncthreads();
      if (has_v) {
#pragma unroll
        for (int i = 0; i < RG; ++i) {
          o[i][0] *= sh.keep[r0 + i];
          o[i][1] *= sh.keep[r0 + i];
        }
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const int n = valid[c];
          if (n <= 0) continue;
          const float* pp = p + c * kPiece * PS + r0;
#pragma unroll
          for (int t = 0; t < kPiece; t += 4) {
            uint32_t h[4], f[2];
            e2m1x8_to_f16(t == 0 ? w[c].x : t == 4 ? w[c].y : t == 8 ? w[c].z : w[c].w, h);
            e4m3x4_to_f16(t == 0 ? sv[c].x : t == 4 ? sv[c].y : t == 8 ? sv[c].z : sv[c].w, f[0], f[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 v = f16x2_to_f32(h[e]), ff = f16x2_to_f32(f[e / 2]);
              // (tokens that do not count are zero whatever their bytes hold)
              const float sc = t + e < n ? (e % 2 ? ff.y : ff.x) : 0.f, v0 = v.x * sc, v1 = v.y * sc;
              float y[RG];
              if constexpr (RG % 4 == 0) {
#pragma unroll
                for (int i = 0; i < RG; i += 4) {
                  const float4 z = *reinterpret_cast<const float4*>(pp + (t + e) * PS + i);
                  y[i] = z.x, y[i + 1] = z.y, y[i + 2] = z.z, y[i + 3] = z.w;
                }
              } else {
#pragma unroll
                for (int i = 0; i < RG; ++i) y[i] = pp[(t + e) * PS + i];
              }
#pragma unroll
              for (int i = 0; i < RG; ++i) {
                o[i][0] = fmaf(y[i], v0, o[i][0]);
                o[i][1] = fmaf(y[i], v1, o[i][1]);
              }
            }
          }
        }
      }
      __syncthreads();
    }
    const long long at = (long long)s.slot * a.rows;
    if (part == 0 && row < rows) a.part_ml[at + row] = make_float2(m, l);
    if (has_v) {
      float* to = a.part_o + (at + r0) * a.d + vg * kGroup + vc;
#pragma unroll
      for (int i = 0; i < RG; ++i)
        if (r0 + i < rows) {
          to[i * a.d] = o[i][0];
          to[i * a.d + 8] = o[i][1];
        }
    }
  }
  if (flags) atomicOr(a.status, flags);
}

template <int RT, int GR>
cudaError_t launch(const Attend4Args& a, int dtype, cudaStream_t st) {
  static std::atomic<int> per_sm[kMaxDevices];  // resident CTAs at the widest head
  const int dev = current_device();
  const size_t most = smem_bytes<RT>(2 * kThreads / GR);
  int n = per_sm[dev].load();
  if (n == 0) {
    cudaError_t e = cudaFuncSetAttribute(attend4_simt_kernel<RT, GR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)most);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attend4_simt_kernel<RT, GR>, kThreads, most);
    if (e != cudaSuccess) return e;
    per_sm[dev].store(n = std::max(n, 1));
  }
  Attend4Args b = a;
  b.ctas = std::min(kMaxSimt4Ctas, sm_count() * n);
  const cudaError_t e = launch_pdl(attend4_simt_kernel<RT, GR>, dim3(b.ctas), dim3(kThreads), smem_bytes<RT>(a.d), st, b,
                                   (int)(dtype == SV_F32));
  return e == cudaSuccess ? launch_join4(b, dtype, st) : e;
}

template <int RT>
cudaError_t launch_rows(const Attend4Args& a, int dtype, cudaStream_t st) {
  if (a.d <= 64) return launch<RT, 8>(a, dtype, st);
  if (a.d <= 128) return launch<RT, 4>(a, dtype, st);
  return launch<RT, 2>(a, dtype, st);
}

}  // namespace

cudaError_t launch_attend4_simt(Attend4Args a, int dtype, cudaStream_t st) {
  const int stacked = a.T * a.G;
  a.row_tiles = (stacked + kSimt4Rows - 1) / kSimt4Rows;
  a.rows = (stacked + a.row_tiles - 1) / a.row_tiles;
  a.ppt = kPieces;
  a.ppt_shift = 2;
  a.streams = 1;
  // (1, 2 and 4 tiles: 16 sequences of 1 to 32768 tokens, 8 heads of 128, one token, 243, 245 and
  // 248 us; 64 of 50 to 3000, 4 heads of 64, 8 rows, 55, 56 and 62)
  a.pair_cost = 1;
  if (a.rows <= 4) return launch_rows<4>(a, dtype, st);
  if (a.rows <= 8) return launch_rows<8>(a, dtype, st);
  if (a.rows <= 16) return launch_rows<16>(a, dtype, st);
  return launch_rows<32>(a, dtype, st);
}

}  // namespace sva
