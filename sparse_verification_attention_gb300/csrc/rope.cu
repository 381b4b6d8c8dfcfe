// Norms of query and key heads and the rotation to their positions in one pass
// over the rows, keys (and values beside them) on the way into the paged cache
// where the call names one.
#include <algorithm>

#include "kv4.h"
#include "ptx.h"
#include "tc_issue.cuh"

namespace sva {
namespace {

constexpr int kThreads = 32;  // a warp: its place is taken again as soon as its token is done

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// V elements (4) of bf16 or fp32, as 32-bit floats and back. (Loads past L1:
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
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(w[i]);
      else f[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void put(const float* f) {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
      else w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  }
};

// A segment of `width` lanes takes a head's row, each lane two chunks of V
// elements: the two halves that rotate with each other, or neighbouring chunks when
// neighbours do (and behind the rotated dims). So a pair's elements meet in one
// lane, and a head's sum of squares needs log2(width) exchanges. `parts` warps share a
// token's heads, side by side: queries, keys, values (copied).
//
// Norm and rotation of a pair (a, b) with weights m, n are four products
//   r (a (m c) - b (n s)),  r (b (n c) + a (m s)),
// of which the four in brackets are the same for all heads of a side and token: a lane
// makes them once and keeps them in registers, r is the row's 1 / sqrt(mean + eps).
//
// Bound by HBM: every row is read and written once. 20,011 rows of 36 normed heads of 128 in
// bf16: 63.9 us, 5.9 TB/s, 0.87 of the copy rate; 15,439 rows of 32 + 8 + 8 heads into the
// cache: 61.9 us, 0.92. (28 CTAs of a warp an SM; 24 66.1 and 64.3, 32, in fewer registers, 65.9 and
// 64.8; CTAs of eight warps 74.5 and 68.4. Two or three rows in flight a lane: 84 and 80 us.)
// fp32 spills in the 72 registers that this leaves: 10,007 rows of 36 normed heads 63 us (floor 55),
// half of each head rotated 84, neighbours paired without a norm 77; 20 CTAs, which spill nothing,
// 61, 62 and 63.
// FULL: every lane has two chunks and all of them turn.
template <typename T, int V, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, 28) rope_kernel(const __grid_constant__ RopeArgs a, int width) {
  constexpr int kFlight = 4;  // rows that a lane has in flight
  const int lane = threadIdx.x & 31, l = lane & (width - 1), seg = lane / width, segs = 32 / width;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int token = (int)(w >> a.parts_shift), part = (int)w & ((1 << a.parts_shift) - 1);
  pdl_wait();
  pdl_trigger();
  if (token >= a.n) return;
  const int pos = a.positions ? a.positions[token] : 0;
  const int slot = a.k_pool ? a.slots[token] : 0;
  const bool one_side = gridDim.y > 1, reports = lane == 0 && part == 0 && blockIdx.y == 0 && a.status;
  if (pos < 0 || (a.rot && pos >= a.max_pos)) {
    if (pos != -1 && reports) atomicOr(a.status, SV_FLAG_BAD_LENGTH);
    return;
  }
  const int page = slot < 0 ? -1 : slot / a.blk;
  const bool stored = page >= 0 && page < a.num_pages;
  if (a.k_pool && !stored && slot != -1 && reports) atomicOr(a.status, SV_FLAG_BAD_PAGE);
  // the lane's chunks, and its pairs' cosines and sines
  const int chunks = a.d / V, half = INTER ? 0 : a.rot / (2 * V);
  const int c0 = INTER || l >= half ? 2 * l : l;
  const int c1 = INTER || l >= half ? 2 * l + 1 : l + half;
  const bool has0 = FULL || c0 < chunks, has1 = FULL || c1 < chunks;
  const int turning = FULL ? V : a.rot / 2 - l * V;  // pairs of the lane that turn (at most V)
  float cos[V], sin[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    cos[e] = 1.f;
    sin[e] = 0.f;
  }
  if (turning > 0) {  // (four pairs at a time: rot is a multiple of 8)
    const float* t = a.table + (long long)pos * a.rot + l * V;
#pragma unroll
    for (int e = 0; e < V; e += 4)
      if (e < turning) {
        const float4 c = __ldcg(reinterpret_cast<const float4*>(t + e));
        const float4 s = __ldcg(reinterpret_cast<const float4*>(t + a.rot / 2 + e));
        cos[e] = c.x, cos[e + 1] = c.y, cos[e + 2] = c.z, cos[e + 3] = c.w;
        sin[e] = s.x, sin[e + 1] = s.y, sin[e + 2] = s.z, sin[e + 3] = s.w;
      }
  }
  // element i of the pair e: which of the lane's 2 V elements
  auto first = [](int e) { return INTER ? 2 * e : e; };
  auto second = [](int e) { return INTER ? 2 * e + 1 : e + V; };
#pragma unroll 1
  for (int side = one_side ? blockIdx.y : 0, last = one_side ? side : 2; side <= last; ++side) {
    const T* from;
    T* to;
    long long to_step = a.d;
    int heads = a.Hkv;
    const void* weight = nullptr;
    if (side == 0) {
      if (!a.q) continue;
      from = static_cast<const T*>(a.q) + token * a.q_stride;
      to = static_cast<T*>(a.q_out) + token * a.qo_stride;
      heads = a.Hq;
      weight = a.q_weight;
    } else {
      if (side == 2 && !a.v) break;
      from = side == 1 ? static_cast<const T*>(a.k) + token * a.k_stride : static_cast<const T*>(a.v) + token * a.v_stride;
      if (side == 1) weight = a.k_weight;
      if (a.k_pool) {
        if (!stored) break;
        to_step = (long long)a.blk * a.d;
        to = static_cast<T*>(side == 1 ? a.k_pool : a.v_pool) +
             (page * (long long)a.Hkv * a.blk + (slot - page * a.blk)) * a.d;
      } else {
        to = static_cast<T*>(a.k_out) + token * a.ko_stride;
      }
    }
    // (two pairs' factors each)
    uint64_t mc[V / 2], ns[V / 2], nc[V / 2], ms[V / 2];
    const int step = segs << a.parts_shift;
    const long long from_step = (long long)step * a.d, out_step = step * to_step;
    const int apart = (c1 - c0) * V;  // of the lane's two chunks
    from += (long long)(part * segs + seg) * a.d + c0 * V;
    to += (part * segs + seg) * to_step + c0 * V;
#pragma unroll 1
    for (int h0 = part * segs; h0 < heads; h0 += step * kFlight) {
      Chunk<T, V> x[kFlight][2];
#pragma unroll
      for (int f = 0; f < kFlight; ++f, from += from_step)
        if (h0 + f * step + seg < heads) {
          if (has0) x[f][0].load(from);
          if (has1) x[f][1].load(from + apart);
        }
      if (side < 2 && h0 == part * segs) {  // (behind the first loads, which wait for neither angles nor weights)
        float m[2 * V];
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) m[e] = 1.f;
        if (weight) {
          Chunk<T, V> g;
          if (has0) {
            g.load(static_cast<const T*>(weight) + c0 * V);
            g.get(m);
          }
          if (has1) {
            g.load(static_cast<const T*>(weight) + c1 * V);
            g.get(m + V);
          }
        }
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float m0 = m[first(e)], m1 = m[first(e + 1)], n0 = m[second(e)], n1 = m[second(e + 1)];
          mc[e / 2] = pack2(m0 * cos[e], m1 * cos[e + 1]);
          ms[e / 2] = pack2(m0 * sin[e], m1 * sin[e + 1]);
          nc[e / 2] = pack2(n0 * cos[e], n1 * cos[e + 1]);
          ns[e / 2] = pack2(-n0 * sin[e], -n1 * sin[e + 1]);
        }
      }
      // 1 / sqrt of the rows' mean squares: the rows' exchanges side by side (one row after
      // the other, with its rotation in between, took 78 us where this took 73: 20,011 rows of 36 heads)
      float inv[kFlight];
      if (weight) {
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
          float y[2 * V], sum = 0.f;
          x[f][0].get(y);
          x[f][1].get(y + V);
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) sum += FULL || (e < V ? has0 : has1) ? y[e] * y[e] : 0.f;
          inv[f] = sum;
        }
        for (int o = width / 2; o; o >>= 1)
#pragma unroll
          for (int f = 0; f < kFlight; ++f) inv[f] += __shfl_xor_sync(0xffffffffu, inv[f], o);
#pragma unroll
        for (int f = 0; f < kFlight; ++f) inv[f] = rsqrtf(inv[f] * a.inv_d + a.eps);
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f, to += out_step) {
        if (h0 + f * step >= heads) break;  // (the same for all lanes)
        if (side < 2) {
          float y[2 * V];
          x[f][0].get(y);
          x[f][1].get(y + V);
          uint64_t u[V / 2], v[V / 2];
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            u[e / 2] = pack2(y[first(e)], y[first(e + 1)]);
            v[e / 2] = pack2(y[second(e)], y[second(e + 1)]);
          }
          const uint64_t r = weight ? pack2(inv[f], inv[f]) : pack2(1.f, 1.f);
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            // (a dim that does not turn takes nothing of another, which may be infinite;
            // pairs turn or do not in fours)
            uint64_t p = mul2(u[e / 2], mc[e / 2]), q = mul2(v[e / 2], nc[e / 2]);
            if (FULL || turning > 0) {
              p = fma2(v[e / 2], ns[e / 2], p);
              q = fma2(u[e / 2], ms[e / 2], q);
            }
            const float2 pp = unpack2(mul2(p, r)), qq = unpack2(mul2(q, r));
            y[first(e)] = pp.x;
            y[first(e + 1)] = pp.y;
            y[second(e)] = qq.x;
            y[second(e + 1)] = qq.y;
          }
          x[f][0].put(y);
          x[f][1].put(y + V);
        }
        if (h0 + f * step + seg < heads) {
          if (has0) x[f][0].store(to);
          if (has1) x[f][1].store(to + apart);
        }
      }
    }
  }
}

template <typename T, int V, bool INTER>
cudaError_t launch(RopeArgs a, cudaStream_t st) {
  const int lanes = (a.d / V + 1) / 2;
  int width = 1;
  while (width < lanes) width <<= 1;
  const int heads = std::max(a.q ? a.Hq : 0, a.Hkv);
  // One warp a token for many tokens; for few, as many as a side's heads give work, so
  // that a decoding step's loads are all in flight at once.
  a.parts_shift = 0;
  while ((32 << a.parts_shift) < heads * width && ((long long)a.n << a.parts_shift) < 152 * 32)
    ++a.parts_shift;
  a.inv_d = 1.f / (float)a.d;
  const long long warps = (long long)a.n << a.parts_shift;
  const bool full = a.rot == a.d && a.d == 2 * V * width;
  const unsigned blocks = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
  // Few warps take a side each: one side's rows after the other's wait for memory three
  // times (23 tokens of 16 heads: 2.6 us a call, 5.0 with the sides in turn; 32 of 40, without
  // values: 2.1 and 2.5).
  const dim3 grid(blocks, warps < 16 * 152 ? 3 : 1);
  return launch_pdl(full ? rope_kernel<T, V, INTER, true> : rope_kernel<T, V, INTER, false>, grid, dim3(kThreads), 0, st, a,
                    width);
}

template <typename T>
cudaError_t launch_as(const RopeArgs& a, cudaStream_t st) {
  return a.interleaved ? launch<T, 4, true>(a, st) : launch<T, 4, false>(a, st);
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int dtype, cudaStream_t st) {
  return dtype == SV_BF16 ? launch_as<__nv_bfloat16>(a, st) : launch_as<float>(a, st);
}

}  // namespace sva
