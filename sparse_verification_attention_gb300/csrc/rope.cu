// Norms of query and key heads and the rotation to their positions in one pass
// over the rows, keys (and values beside them) on the way into the paged cache
// where the call names one.
#include <algorithm>

#include "kv4.h"
#include "ptx.h"

namespace sva {
namespace {

constexpr int kThreads = 256;
constexpr int kFlight = 4;  // rows that a thread has in flight

// V elements (8 or 4) of bf16 or fp32, as 32-bit floats and back. (Loads past L1:
// under a programmatic launch the rows may be written while this grid is already
// resident, and a row that is rotated in place is.)
template <typename T, int V>
struct Chunk {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 2) {
      const uint2 x = __ldcg(reinterpret_cast<const uint2*>(p));
      w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 x = __ldcg(reinterpret_cast<const uint4*>(p) + i / 4);
        w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(w[i]);
      else f[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void put(const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
      else w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  }
};

// A segment of `width` lanes takes a head's row, each lane two chunks of V
// elements: the two halves that rotate with each other, or neighbouring chunks when
// neighbours do (and behind the rotated dims). So a pair's elements meet in one
// lane, its angle's V cosines and sines stay in the lane's registers for all heads
// of the token, and a head's sum of squares needs log2(width) exchanges. `parts`
// warps share a token's heads.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int width) {
  const int lane = threadIdx.x & 31, l = lane & (width - 1), seg = lane / width, segs = 32 / width;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long token = w / a.parts;
  const int part = (int)(w - token * a.parts);
  pdl_wait();
  pdl_trigger();
  if (token >= a.n) return;
  const int pos = a.positions ? a.positions[token] : 0;
  if (pos < 0 || (a.rot && pos >= a.max_pos)) {
    if (pos != -1 && lane == 0 && part == 0 && a.status) atomicOr(a.status, SV_FLAG_BAD_LENGTH);
    return;
  }
  long long page = -1, off = 0;
  if (a.k_pool) {
    const int slot = a.slots[token];
    if (slot >= 0) {
      page = slot / a.blk;
      off = slot - page * a.blk;
    }
    if (slot < -1 || page >= a.num_pages) {
      if (lane == 0 && part == 0 && a.status) atomicOr(a.status, SV_FLAG_BAD_PAGE);
      page = -1;
    }
  }
  // the lane's chunks
  const int chunks = a.d / V, half = INTER ? 0 : a.rot / (2 * V);
  const int c0 = INTER || l >= half ? 2 * l : l;
  const int c1 = INTER || l >= half ? 2 * l + 1 : l + half;
  const bool has0 = c0 < chunks, has1 = c1 < chunks;
  float cos[V], sin[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int i = l * V + e;
    const bool turns = i < a.rot / 2;
    cos[e] = turns ? __ldcg(a.table + (long long)pos * a.rot + i) : 1.f;
    sin[e] = turns ? __ldcg(a.table + (long long)pos * a.rot + a.rot / 2 + i) : 0.f;
  }
  const int hq = a.q ? a.Hq : 0, hk = hq + a.Hkv, heads = a.v ? hk + a.Hkv : hk;
  const T *q = static_cast<const T*>(a.q) + token * a.q_stride, *k = static_cast<const T*>(a.k) + token * a.k_stride,
          *v = static_cast<const T*>(a.v) + token * a.v_stride;
  const int step = segs * a.parts;
  for (int h0 = part * segs + seg; h0 - seg < heads; h0 += step * kFlight) {
    Chunk<T, V> x[kFlight][2];
    T* to[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int h = h0 + f * step;
      to[f] = nullptr;
      if (h >= heads) continue;
      const T* from;
      if (h < hq) {
        from = q + (long long)h * a.d;
        to[f] = static_cast<T*>(a.q_out) + token * a.qo_stride + (long long)h * a.d;
      } else {
        const bool is_v = h >= hk;
        const int kh = h - (is_v ? hk : hq);
        from = (is_v ? v : k) + (long long)kh * a.d;
        if (!a.k_pool) to[f] = static_cast<T*>(a.k_out) + token * a.ko_stride + (long long)kh * a.d;
        else if (page >= 0)
          to[f] = static_cast<T*>(is_v ? a.v_pool : a.k_pool) + ((page * a.Hkv + kh) * a.blk + off) * a.d;
      }
      if (!to[f]) continue;
      if (has0) x[f][0].load(from + c0 * V);
      if (has1) x[f][1].load(from + c1 * V);
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int h = h0 + f * step;
      const bool turn = h < hk;
      const void* weight = h < hq ? a.q_weight : a.k_weight;
      float y0[V], y1[V];
#pragma unroll
      for (int e = 0; e < V; ++e) y0[e] = y1[e] = 0.f;
      if (to[f] && has0) x[f][0].get(y0);
      if (to[f] && has1) x[f][1].get(y1);
      if (a.q_weight || a.k_weight) {  // (all lanes take part in the exchange)
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) sum += y0[e] * y0[e] + y1[e] * y1[e];
        for (int o = width / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (weight && turn && to[f]) {
          const float r = rsqrtf(sum / (float)a.d + a.eps);
          Chunk<T, V> g;
          float m[V];
          if (has0) {
            g.load(static_cast<const T*>(weight) + c0 * V);
            g.get(m);
#pragma unroll
            for (int e = 0; e < V; ++e) y0[e] = y0[e] * r * m[e];
          }
          if (has1) {
            g.load(static_cast<const T*>(weight) + c1 * V);
            g.get(m);
#pragma unroll
            for (int e = 0; e < V; ++e) y1[e] = y1[e] * r * m[e];
          }
        }
      }
      if (!to[f]) continue;
      if (turn) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (l * V + e >= a.rot / 2) continue;
          float &p = INTER ? (2 * e < V ? y0[2 * e % V] : y1[2 * e % V]) : y0[e];
          float &r = INTER ? (2 * e < V ? y0[(2 * e + 1) % V] : y1[(2 * e + 1) % V]) : y1[e];
          const float p0 = p, r0 = r;
          p = p0 * cos[e] - r0 * sin[e];
          r = r0 * cos[e] + p0 * sin[e];
        }
        x[f][0].put(y0);
        x[f][1].put(y1);
      }
      if (has0) x[f][0].store(to[f] + c0 * V);
      if (has1) x[f][1].store(to[f] + c1 * V);
    }
  }
}

template <typename T, int V, bool INTER>
cudaError_t launch(RopeArgs a, cudaStream_t st) {
  const int lanes = (a.d / V + 1) / 2;
  int width = 1;
  while (width < lanes) width <<= 1;
  const int heads = (a.q ? a.Hq : 0) + a.Hkv + (a.v ? a.Hkv : 0);
  const int rounds = std::max(1, (heads * width + 31) / 32);  // of a warp alone with a token
  // One warp a token for many tokens; for few, as many as the heads give work, so that
  // a decoding step's loads are all in flight at once.
  a.parts = 1;
  while (a.parts < rounds && (long long)a.n * a.parts < 152 * 32) a.parts *= 2;
  const long long warps = (long long)a.n * a.parts;
  return launch_pdl(rope_kernel<T, V, INTER>, dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32))),
                    dim3(kThreads), 0, st, a, width);
}

template <typename T>
cudaError_t launch_as(const RopeArgs& a, cudaStream_t st) {
  // 8 elements a chunk where both halves are whole chunks, else 4
  if (a.interleaved) return launch<T, 8, true>(a, st);
  return a.rot % 16 == 0 ? launch<T, 8, false>(a, st) : launch<T, 4, false>(a, st);
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int dtype, cudaStream_t st) {
  return dtype == SV_BF16 ? launch_as<__nv_bfloat16>(a, st) : launch_as<float>(a, st);
}

}  // namespace sva
