// The join of a shared-prefix verification: every row's partial rows (its
// shared tile's runs of keys, then its own) summed with log-sum-exp weights.
#include "internal.h"
#include "paged.cuh"
#include "ptx.h"

namespace sva {
namespace {

using namespace paged;

constexpr int kThreads = 256;

// One warp per output row. A launch of its own and not the last arrival's
// work inside the attention kernel: the last shared item to finish completes
// the rows of the whole batch at once, and one CTA merging them took longer
// than the attention (48 single-token steps over a 16384-token prefix 228 us,
// 16-draft trees of 8 over 65536 tokens 322 us). The plan depends on the
// arguments only, so it is rebuilt while the attention drains.
template <typename T>
__global__ void __launch_bounds__(kThreads) prefix_merge_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ Plan plan;
  __shared__ __align__(16) int scratch[kPlanScratch];
  make_plan(a, &plan, scratch);
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= a.n_rows * a.Hq) return;
  const int tok = row / a.Hq, head = row % a.Hq, kvh = head / a.G, in = head % a.G;
  const int hv = kvh * a.hs + in / a.gs, g = in % a.gs, b = tok / a.T, t = tok % a.T;
  // rows of a segment lie by head group, row tile, run, token, head
  const int n0 = a.n_shared ? a.n_rows : 0, rr0 = min(a.tile, n0) * a.gs, rr1 = min(a.tile, a.T) * a.gs;
  const int s0 = a.n_shared ? plan.split[0] : 0, s1 = plan.split[b + 1];
  const int tiles0 = ceil_div(n0, a.tile), tiles1 = ceil_div(a.T, a.tile);
  const Group gr[2] = {
      {plan.rows[0] + (long long)(hv * tiles0 + tok / a.tile) * s0 * rr0 + tok % a.tile * a.gs + g, rr0, s0},
      {plan.rows[b + 1] + (long long)(hv * tiles1 + t / a.tile) * s1 * rr1 + t % a.tile * a.gs + g, rr1, s1}};
  merge_row<T>(a, gr, static_cast<T*>(a.out) + (size_t)row * a.d);
}

}  // namespace

cudaError_t launch_prefix_merge(const PagedArgs& a, int dtype, cudaStream_t st) {
  const int per = kThreads / 32;
  const dim3 grid((unsigned)(((long long)a.n_rows * a.Hq + per - 1) / per));
  return dtype == SV_BF16 ? launch_pdl(prefix_merge_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a)
                          : launch_pdl(prefix_merge_kernel<float>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace sva
