// The drafts, and the join of a row's segments: what sv_attend_kv4 does behind the
// attention over the cache. A row's own drafts stay in the call's type; there are at
// most 64 of them, so fp32 on the CUDA cores costs little and needs no tile.
// Bound by latency: a row's loads (q, drafts, slots, parts) come one after the other, so that
// rows in flight are what counts (4096 rows of 16 drafts and 7 parts: 11.6 us in 64 registers,
// 17 in 87).
#include "kv4.cuh"

namespace sva {
namespace {

using namespace kv4;

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // drafts, or parts of a row, whose loads are under way together

// Four consecutive elements as floats, and back.
__device__ __forceinline__ float4 load4(const float* p) { return __ldcg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = __ldcg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}
__device__ __forceinline__ float dot4(float4 a, float4 b) { return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w; }
__device__ __forceinline__ void axpy4(float4& o, float w, float4 x) {
  o.x += w * x.x;
  o.y += w * x.y;
  o.z += w * x.z;
  o.w += w * x.w;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// One warp per output row; a lane has dims 4 lane .. + 3 (and 128 + that for NJ = 2, d > 128).
template <typename T, int NJ>
__global__ void __launch_bounds__(kThreads, NJ == 1 ? 4 : 2) join4_kernel(const __grid_constant__ Attend4Args a) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.T * a.Hq) return;
  const int tok = quotient((int)row, a.Hq), head = (int)row - tok * a.Hq, b = quotient(tok, a.T), t = tok - b * a.T;
  const int h = a.g_shift >= 0 ? head >> a.g_shift : quotient(head, a.G), r = t * a.G + head - h * a.G;
  const int rt = a.row_tiles == 1 ? 0 : quotient(r, a.rows);
  bool has[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) has[j] = 128 * j + lane * 4 < a.d;
  float4 q[NJ], o[NJ];
#pragma unroll
  for (int i = 0; i < NJ; ++i) {
    q[i] = o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (has[i]) q[i] = load4(static_cast<const T*>(a.q) + row * a.d + 128 * i + lane * 4);
  }
  // the drafts that t sees: scores of the i-th in lane i % 32
  const unsigned long long see = a.anc[t];
  const int n = __popcll(see);
  const T* dk = static_cast<const T*>(a.draft_k) + ((long long)b * a.T * a.Hkv + h) * a.d;
  const T* dv = static_cast<const T*>(a.draft_v) + ((long long)b * a.T * a.Hkv + h) * a.d;
  const long long step = (long long)a.Hkv * a.d;
  float s0 = -INFINITY, s1 = -INFINITY;
  int u[kBatch];
#pragma unroll 1
  for (unsigned long long w = see, i = 0; w; i += kBatch) {
    float x[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {  // (a batch's loads are under way together)
      u[e] = w ? __ffsll(w) - 1 : -1;
      w &= w - 1;
      x[e] = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (u[e] >= 0 && has[j]) x[e] += dot4(q[j], load4(dk + u[e] * step + 128 * j + lane * 4));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int e = 0; e < kBatch; ++e) x[e] += __shfl_xor_sync(0xffffffffu, x[e], o);
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (u[e] >= 0 && lane == (((int)i + e) & 31)) ((int)i < 32 ? s0 : s1) = x[e] * a.scale_log2;
  }
  // What comes above is older than the attention kernel, which began to let this one in
  // only behind its own wait for its predecessors; what follows is the attention's.
  pdl_wait();
  pdl_trigger();
  // the row's parts
  const int2 slots = __ldcg(a.slots + (b * a.Hkv + h) * a.row_tiles + rt);
  const int parts = slots.y * a.streams;
  const long long at0 = (long long)slots.x * a.streams * a.rows + r - rt * a.rows;
  // the largest reference, of the segments and of the drafts
  float m = fmaxf(s0, s1);
  for (int c = lane; c < parts; c += 32) m = fmaxf(m, a.part_ml[at0 + (long long)c * a.rows].x);
  m = warp_max(m);
  const float p0 = lane < n ? exp2f(s0 - m) : 0.f, p1 = lane + 32 < n ? exp2f(s1 - m) : 0.f;
  float l = warp_sum(p0 + p1);
  const float unit = exp2i(head_exp(a.v_exp, h));
#pragma unroll 1
  for (int c0 = 0; c0 < parts; c0 += kBatch) {
    float2 ml[kBatch];
    float4 x[kBatch][NJ];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const long long at = at0 + (long long)(c0 + e) * a.rows;
      if (c0 + e >= parts) continue;
      ml[e] = __ldcg(a.part_ml + at);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (has[j]) x[e][j] = load4(a.part_o + at * a.d + 128 * j + lane * 4);
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (c0 + e >= parts || (ml[e].x == -INFINITY && ml[e].y == 0.f)) continue;  // no key of the part counted
      const float w = exp2f(ml[e].x - m);
      l += w * ml[e].y;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (has[j]) axpy4(o[j], w * unit, x[e][j]);
    }
  }
#pragma unroll 1
  for (unsigned long long w = see, i = 0; w; i += kBatch) {
    float4 x[kBatch][NJ];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      u[e] = w ? __ffsll(w) - 1 : -1;
      w &= w - 1;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (u[e] >= 0 && has[j]) x[e][j] = load4(dv + u[e] * step + 128 * j + lane * 4);
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const float p = __shfl_sync(0xffffffffu, (int)i < 32 ? p0 : p1, ((int)i + e) & 31);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (u[e] >= 0 && has[j]) axpy4(o[j], p, x[e][j]);
    }
  }
  const float inv = __frcp_rn(l);
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    if (has[j]) {
      const float4 y = make_float4(o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv);
      store4(static_cast<T*>(a.out) + row * a.d + 128 * j + lane * 4, y);
    }
}

template <typename T>
cudaError_t launch_as(const Attend4Args& a, cudaStream_t st) {
  const long long rows = (long long)a.B * a.T * a.Hq;
  const dim3 grid((unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32)));
  return a.d <= 128 ? launch_pdl(join4_kernel<T, 1>, grid, dim3(kThreads), 0, st, a)
                    : launch_pdl(join4_kernel<T, 2>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_join4(const Attend4Args& a, int dtype, cudaStream_t st) {
  return dtype == SV_BF16 ? launch_as<__nv_bfloat16>(a, st) : launch_as<float>(a, st);
}

}  // namespace sva
