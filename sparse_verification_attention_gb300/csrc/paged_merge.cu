// The join of rows whose keys were cut into runs: their partial rows summed
// with log-sum-exp weights. A launch of its own and not the last arrival's work
// inside the attention: one CTA merging a tile's rows held up its next item
// (a 16-sequence decoding step waited about 5 us an item), and in the prefix form
// the last shared item completes the rows of the whole batch at once (that
// merge took longer than the attention: 48 single-token steps over a shared
// prefix 228 us with it, 182 us without).
//
// Bound by latency: three dependent loads (what to join, the maxima and sums, the
// rows) behind the attention's end, 4 to 10 us of a launch measured alone.
#include <algorithm>

#include "internal.h"
#include "paged.cuh"
#include "ptx.h"

namespace sva {
namespace {

using namespace paged;

constexpr int kThreads = 256;

// One warp per output row.
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_merge_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, x = blockIdx.x;
  T* out = static_cast<T*>(a.out);
  if (a.prefix) {
    const int i = x * kWarps + warp;
    const int tok = i / a.Hq, head = i - tok * a.Hq, b = tok / a.T, in = head % a.G;
    const int hv = head / a.G * a.hs + in / a.gs;
    pdl_wait();
    pdl_trigger();
    if (i >= a.n_rows * a.Hq) return;
    const int2 sh = a.n_shared ? __ldcg(a.segs) : make_int2(0, 0), own = __ldcg(a.segs + b + 1);
    // the partial rows of token t of a segment of n tokens
    auto group = [&](int2 s, int n, int t) {
      const int rows = min(a.tile, n) * a.gs;
      return Group{s.x + (long long)(hv * ceil_div(n, a.tile) + t / a.tile) * s.y * rows +
                       t % a.tile * a.gs + in % a.gs,
                   rows, s.y};
    };
    const Group g[2] = {group(sh, a.n_rows, tok), group(own, a.T, tok - b * a.T)};
    merge_row<T>(a, g, out + (size_t)i * a.d);
    return;
  }
  pdl_wait();
  pdl_trigger();
  // Block x joins the unit that CTA x ended with, if it is cut: its beginning lies
  // in slot 2 x + 1, the rest in slots 2 x + 2, 2 x + 4, ...
  const PagedJoin j = a.joins[x];
  if (j.more == 0) return;
  const int slot = slot_rows(a);
  for (int r = blockIdx.y * kWarps + warp; r < j.ntok * j.heads; r += gridDim.y * kWarps) {
    const int tok = r / j.heads, in = r - tok * j.heads;
    const long long row = tok * a.gs + in;
    const Group g[2] = {{(2ll * x + 1) * slot + row, 0, 1}, {(2ll * x + 2) * slot + row, 2 * slot, j.more}};
    merge_row<T>(a, g, out + ((size_t)(j.tok0 + tok) * a.Hq + j.head0 + in) * a.d);
  }
}

}  // namespace

cudaError_t launch_paged_merge(const PagedArgs& a, int dtype, cudaStream_t st) {
  // prefix: a warp per row; prompt: a block per CTA and 32 rows
  const int per = kThreads / 32;
  const dim3 grid = a.prefix ? dim3((unsigned)(((long long)a.n_rows * a.Hq + per - 1) / per))
                             : dim3(a.ctas, (std::min(a.tile, a.n_rows) * a.gs + 4 * per - 1) / (4 * per));
  return dtype == SV_BF16 ? launch_pdl(paged_merge_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a)
                          : launch_pdl(paged_merge_kernel<float>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace sva
