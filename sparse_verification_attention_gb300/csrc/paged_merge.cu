// The join of rows whose keys were cut into runs: their partial rows summed
// with log-sum-exp weights. A launch of its own and not the last arrival's work
// inside the attention: one CTA merging a tile's rows held up its next item
// (a 16-sequence decoding step waited about 5 us an item), and in the prefix form
// the last shared item completes the rows of the whole batch at once (that
// merge took longer than the attention).
#include <algorithm>

#include "internal.h"
#include "paged.cuh"
#include "ptx.h"

namespace sva {
namespace {

using namespace paged;

constexpr int kThreads = 256;

// The plan depends on the lengths only, so it is rebuilt while the attention
// drains. One warp per output row.
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_merge_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ Plan plan;
  __shared__ __align__(16) int scratch[kPlanScratch];
  constexpr int kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5;
  make_plan(a, &plan, scratch);
  pdl_wait();
  pdl_trigger();
  T* out = static_cast<T*>(a.out);
  if (a.prefix) {
    const int i = blockIdx.x * kWarps + warp;
    if (i >= a.n_rows * a.Hq) return;
    const int tok = i / a.Hq, head = i % a.Hq, b = tok / a.T;
    const int in = head % a.G, hv = head / a.G * a.hs + in / a.gs;
    // the partial rows of token t of the segment at position pos, of n tokens
    auto group = [&](int pos, int n, int t) {
      const int rows = min(a.tile, n) * a.gs, runs = plan.split[pos];
      return Group{plan.rows[pos] + (long long)(hv * ceil_div(n, a.tile) + t / a.tile) * runs * rows +
                       t % a.tile * a.gs + in % a.gs,
                   rows, runs};
    };
    const Group g[2] = {a.n_shared ? group(0, a.n_rows, tok) : Group{0, 0, 0},
                        group(b + 1, a.T, tok % a.T)};
    merge_row<T>(a, g, out + (size_t)i * a.d);
    return;
  }
  if (!plan.stream) return;
  // Block x looks at the boundary between the shares of CTAs x and x + 1. A unit
  // that it cuts, and no boundary before it, is this block's to join: its beginning
  // lies in slot 2 x + 1, the rest in slots 2 x + 2, 2 x + 4, ...
  const int nseg = n_segs(a), total = plan.first[nseg], x = blockIdx.x;
  const int cut = share_start(total, a.ctas, x + 1);
  if (cut >= total) return;
  const int lo = find_seg(&plan, nseg, cut), id = plan.order[lo];
  const Seg s = seg_of(a, id);
  const int cost = unit_cost(a, s), tiles = ceil_div(s.n, a.tile);
  const int unit = (cut - plan.first[lo]) / cost, begin = plan.first[lo] + unit * cost;
  if (begin == cut || share_of(total, a.ctas, begin) != x) return;
  const int more = share_of(total, a.ctas, begin + cost - 1) - x, slot = slot_rows(a);
  const int hv = unit / tiles, t = tiles - 1 - unit % tiles;
  const Item it = make_item(a, s, id, t, hv, 0, 0);
  for (int r = blockIdx.y * kWarps + warp; r < it.ntok * it.heads; r += gridDim.y * kWarps) {
    const int tok = r / it.heads, in = r % it.heads;
    const long long row = tok * a.gs + in;
    const Group g[2] = {{(2ll * x + 1) * slot + row, 0, 1}, {(2ll * x + 2) * slot + row, 2 * slot, more}};
    merge_row<T>(a, g, out + ((size_t)(it.tok0 + tok) * a.Hq + it.head0 + in) * a.d);
  }
}

}  // namespace

cudaError_t launch_paged_merge(const PagedArgs& a, int dtype, cudaStream_t st) {
  // prefix: a warp per row; prompt: a block per share boundary and 32 rows
  const int per = kThreads / 32;
  const dim3 grid = a.prefix ? dim3((unsigned)(((long long)a.n_rows * a.Hq + per - 1) / per))
                             : dim3(a.ctas - 1, (std::min(a.tile, a.n_rows) * a.gs + 4 * per - 1) / (4 * per));
  if (grid.x == 0) return cudaSuccess;
  return dtype == SV_BF16 ? launch_pdl(paged_merge_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a)
                          : launch_pdl(paged_merge_kernel<float>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace sva
