// Attention of packed or stacked query rows over the paged cache on the CUDA
// cores: fp32 tensors, and head dims or alignments that the tensor-core
// kernel does not take. Every product and sum is fp32.
//
// One pass over the keys with the running maximum m and sum l of a softmax
// (log2 domain): for a tile of keys, s = q k^T, m' = max(m, max s),
// o = o 2^(m - m') + 2^(s - m') v, l = l 2^(m - m') + sum 2^(s - m').
//
// A CTA holds a tile of 64 rows (64 / gs tokens of one KV head's gs query
// heads, so that K and V are read once for all of them) and walks 64 keys at
// a time; a thread computes 4 x 4 of S and 4 x 4 per 64 columns of O. fp32 K and V
// tiles are copied asynchronously, one tile ahead where two stages fit (d <= 128).
//
// Bound by issue: packed fp32 prompts of up to 1500 tokens (8/2 heads of 64) run at
// 24 TFLOP/s of the about 74 that the cores' FMAs could do, 103 us; the products are
// 45% of the instructions, issue slots 58% full. Products on fp32 pairs take 98 us there
// but 24 instead of 21 us in calls of a few rows (longer code); 8 rows a thread, so a
// third fewer shared loads but half the warps, 110 us.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "internal.h"
#include "paged.cuh"
#include "ptx.h"

namespace sva {
namespace {

using namespace paged;

constexpr int kRows = kSimtRows;
constexpr int kKeys = 64;     // keys of a tile
constexpr int kThreads = 256;
constexpr int kPPitch = kKeys + 4;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return __ldcg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = __ldcg(reinterpret_cast<const uint2*>(p));
  const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
  const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// 16 bytes global -> shared without registers, zeros where src is null.
__device__ __forceinline__ void copy16(float* dst, const void* src, const void* any) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src ? src : any),
               "r"(src ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared memory: Q, and stages of K (whose place P takes) and V. NC: 64-column
// groups of d.
template <int NC>
struct SimtCfg {
  static constexpr int kPitch = 64 * NC + 4;
  static constexpr int kStages = NC <= 2 ? 2 : 1;
  static constexpr int kStage = 2 * kKeys * kPitch;
  static constexpr int kSmem = (kRows * kPitch + kStages * kStage) * 4;
  static constexpr int kCtas = NC == 1 ? 2 : 1;  // per SM, where their stages fit
  static_assert(kRows * kPPitch <= kKeys * kPitch, "P takes the place of K");
};

template <typename T, int NC>
__global__ void __launch_bounds__(kThreads, SimtCfg<NC>::kCtas) paged_simt_kernel(const __grid_constant__ PagedArgs a) {
  extern __shared__ __align__(16) float smem[];
  __shared__ Plan plan;
  __shared__ Item s_item;
  using C = SimtCfg<NC>;
  constexpr int kPitch = C::kPitch, kStages = C::kStages, kStage = C::kStage;
  float* sq = smem;                 // [kRows][kPitch]
  float* ring = sq + kRows * kPitch;  // stages of K and V, [kKeys][kPitch] each
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const T* q = static_cast<const T*>(a.q);

  pdl_wait();
  pdl_trigger();
  make_plan(a, &plan, reinterpret_cast<int*>(smem));

  save_plan(a, &plan);
  Cursor cursor{};  // thread 0's
  if (tid == 0) cursor = start_cursor(a, &plan);
  while (true) {
    if (tid == 0) s_item = next_item(a, &plan, &cursor);
    __syncthreads();
    const Item it = s_item;
    if (!it.valid) break;
    const int rows = it.ntok * it.heads;
    const bool live = (tid >> 5) * 8 < rows;  // the warp's eight rows hold any
    // Q rows r = token * heads + head; rows past the tile's are zero
    for (int e = tid; e < kRows * 16 * NC; e += kThreads) {
      const int r = e / (16 * NC), c = e % (16 * NC) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows && c < a.d)
        x = load4<T>(q + (size_t)(it.tok0 + r / it.heads) * a.q_stride +
                     (size_t)(it.head0 + r % it.heads) * a.d + c);
      *reinterpret_cast<float4*>(sq + r * kPitch + c) = x;
    }
    int vis[4];                 // keys that row i of this thread sees
    unsigned long long anc[4];  // drafts that it sees
    float m[4], l[4], o[4][4 * NC];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i, t = r / it.heads;
      vis[i] = r < rows ? (it.causal ? it.vis0 + t : it.ctx) : 0;
      anc[i] = r < rows && it.draft ? a.anc[it.draft0 + t] : 0ull;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c) o[i][c] = 0.f;
    }
    // K and V rows of key tile kt into its stage, four threads per key; keys past the
    // context, and pages outside the pool, are zero. The page was looked up a
    // tile ahead (-1: none).
    auto lookup = [&](int kt) {
      const int key = (it.k0 + kt) * kKeys + (tid >> 2);
      if (kt >= it.nk || (it.draft && kt == it.nk - 1) || key >= it.ctx) return -1;
      const int page = __ldcg(a.block_table + it.tab + key / a.blk);
      if (page >= 0 && page < a.num_pages) return page;
      if ((tid & 3) == 0) atomicOr(a.status, SV_FLAG_BAD_PAGE);
      return -1;
    };
    auto load = [&](int kt, int page) {
      const int r = tid >> 2;
      const T *kr = nullptr, *vr = nullptr;
      if (it.draft && kt == it.nk - 1) {
        if (r < a.T) {
          const size_t off = (((size_t)it.seq * a.T + r) * a.Hkv + it.kvh) * a.d;
          kr = static_cast<const T*>(a.draft_k) + off;
          vr = static_cast<const T*>(a.draft_v) + off;
        }
      } else if (page >= 0) {
        const int key = (it.k0 + kt) * kKeys + r;
        const size_t off = (((size_t)page * a.Hkv + it.kvh) * a.blk + key % a.blk) * a.d;
        kr = static_cast<const T*>(a.k_pool) + off;
        vr = static_cast<const T*>(a.v_pool) + off;
      }
      float* dk = ring + kt % kStages * kStage + r * kPitch;
      float* dv = dk + kKeys * kPitch;
#pragma unroll
      for (int c0 = 0; c0 < 64 * NC; c0 += 16) {
        const int c = c0 + 4 * (tid & 3);
        const bool in = kr && c < a.d;
        if constexpr (sizeof(T) == 4) {
          copy16(dk + c, in ? kr + c : nullptr, a.k_pool);
          copy16(dv + c, in ? vr + c : nullptr, a.k_pool);
        } else {
          const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<float4*>(dk + c) = in ? load4<T>(kr + c) : zero;
          *reinterpret_cast<float4*>(dv + c) = in ? load4<T>(vr + c) : zero;
        }
      }
    };
    int page = lookup(0);
    if (it.nk > 0) load(0, page);
    copies_issued();
    page = lookup(1);
    for (int kt = 0; kt < it.nk; ++kt) {
      const int key0 = (it.k0 + kt) * kKeys;
      const bool drafts = it.draft && kt == it.nk - 1;
      float* sk = ring + kt % kStages * kStage;  // then P [kRows][kPPitch]
      float* sp = sk;
      const float* sv = sk + kKeys * kPitch;
      if (kStages > 1) {
        if (kt + 1 < it.nk) load(kt + 1, page);
        copies_issued();
        page = lookup(kt + 2);
      }
      copies_wait<kStages - 1>();  // this tile's
      __syncthreads();
      float s[4][4];  // rows ty * 4 + i, keys tx + 16 * j
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
      if (live)
#pragma unroll 2
      for (int c = 0; c < 64 * NC; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(sq + (ty * 4 + i) * kPitch + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * kPitch + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
      }
      __syncthreads();  // every read of K is done: P takes its place
      // a tile where some row of the item misses some key: masked entries get
      // P = -1 and their V is not touched (it may hold anything)
      const bool masked = drafts || key0 + kKeys > (it.causal ? it.vis0 : it.ctx);
#pragma unroll
      for (int i = 0; i < 4 && live; ++i) {
        bool keep[4];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = tx + 16 * j;
          keep[j] = !masked || (drafts ? (anc[i] >> k & 1ull) != 0 : key0 + k < vis[i]);
          s[i][j] = keep[j] ? s[i][j] * a.scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m[i], mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(m[i] - base);  // 0 before the first key
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(s[i][j] - base);
          sum += p;
          sp[(ty * 4 + i) * kPPitch + tx + 16 * j] = keep[j] ? p : -1.f;
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l[i] = l[i] * alpha + sum;
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < 4 * NC; ++c) o[i][c] *= alpha;
      }
      __syncwarp();  // a row's P is written and read by the same half-warp
      // O += P V; where the tile is masked, a masked key's V is not touched
      auto product = [&](auto tag) {
        constexpr bool select = decltype(tag)::value;
        for (int k = 0; k < kKeys; k += 4) {
          float4 p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (ty * 4 + i) * kPPitch + k);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
            for (int cg = 0; cg < NC; ++cg) {
              const float4 v = *reinterpret_cast<const float4*>(sv + (k + kk) * kPitch + 64 * cg + 4 * tx);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                if (!select || w >= 0.f || w != w) {
                  o[i][4 * cg] = fmaf(w, v.x, o[i][4 * cg]);
                  o[i][4 * cg + 1] = fmaf(w, v.y, o[i][4 * cg + 1]);
                  o[i][4 * cg + 2] = fmaf(w, v.z, o[i][4 * cg + 2]);
                  o[i][4 * cg + 3] = fmaf(w, v.w, o[i][4 * cg + 3]);
                }
              }
            }
          }
        }
      };
      if (live) {
        if (masked) product(std::true_type{});
        else product(std::false_type{});
      }
      __syncthreads();  // the stage is free again
      if (kStages == 1) {
        if (kt + 1 < it.nk) load(kt + 1, page);
        copies_issued();
        page = lookup(kt + 2);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i, t = r / it.heads, g = r % it.heads;
      if (r >= rows) continue;
      if (it.part < 0) {
        const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i];
        T* dst = static_cast<T*>(a.out) + ((size_t)(it.tok0 + t) * a.Hq + it.head0 + g) * a.d;
#pragma unroll
        for (int cg = 0; cg < NC; ++cg) {
          const int c = 64 * cg + 4 * tx;
          if (c < a.d)
            store4<T>(dst + c, o[i][4 * cg] * inv, o[i][4 * cg + 1] * inv, o[i][4 * cg + 2] * inv,
                      o[i][4 * cg + 3] * inv);
        }
      } else {
        const size_t row = (size_t)it.part + t * a.gs + g;
#pragma unroll
        for (int cg = 0; cg < NC; ++cg) {
          const int c = 64 * cg + 4 * tx;
          if (c < a.d)
            store4<float>(a.part_o + row * a.d + c, o[i][4 * cg], o[i][4 * cg + 1], o[i][4 * cg + 2],
                          o[i][4 * cg + 3]);
        }
        if (tx == 0) a.part_ml[row] = make_float2(m[i], l[i]);
      }
    }
    __syncthreads();  // s_item and the tiles are free again
  }
  if (tid == 0) leave(a);
}

template <typename T, int NC>
cudaError_t launch_cfg(PagedArgs a, int dtype, cudaStream_t st) {
  const int dev = current_device();
  static std::atomic<int> per_sm[kMaxDevices];
  int n = per_sm[dev].load();
  if (n <= 0) {
    cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<T, NC>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, SimtCfg<NC>::kSmem);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, paged_simt_kernel<T, NC>, kThreads,
                                                        SimtCfg<NC>::kSmem);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    per_sm[dev].store(n);
  }
  a.ctas = std::min(sm_count() * n, kMaxPlanCtas);
  const cudaError_t e = launch_pdl(paged_simt_kernel<T, NC>, dim3(a.ctas), dim3(kThreads),
                                   SimtCfg<NC>::kSmem, st, a);
  return e == cudaSuccess ? launch_paged_merge(a, dtype, st) : e;
}

template <typename T>
cudaError_t launch_type(const PagedArgs& a, int dtype, cudaStream_t st) {
  if (a.d <= 64) return launch_cfg<T, 1>(a, dtype, st);
  if (a.d <= 128) return launch_cfg<T, 2>(a, dtype, st);
  if (a.d <= 192) return launch_cfg<T, 3>(a, dtype, st);
  return launch_cfg<T, 4>(a, dtype, st);
}

}  // namespace

cudaError_t launch_paged_simt(PagedArgs a, int dtype, cudaStream_t st) {
  paged_heads(&a, kRows);
  a.min_run = 1;
  a.tile = kRows / a.gs;
  a.one_set = 1 << 30;
  a.item_cost = 1;
  a.key_shift = 6;
  return dtype == SV_BF16 ? launch_type<__nv_bfloat16>(a, dtype, st) : launch_type<float>(a, dtype, st);
}

}  // namespace sva
