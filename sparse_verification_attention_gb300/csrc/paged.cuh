// Work split, item decoding and the log-sum-exp merge that the paged
// attention kernels share (device code).
//
// A segment's rows are cut into tiles of `tile` tokens, its keys into tiles
// of `keys` tokens (the prefix form's drafts are one more key tile). An item
// is one row tile of one head group over a run of key tiles. Lengths may live
// in device memory only, so every CTA derives the same plan from them: a
// segment whose row tiles see more than C key tiles is cut into s =
// ceil(kt / C) runs, with C such that the grid gets about two items per CTA.
// That bounds the partial rows by a number the host knows: the items of cut
// segments are at most twice sum(tiles * kt) / C <= 4 * CTAs.
#pragma once

#include "paged.h"
#include "ptx.h"

namespace sva {
namespace paged {

struct Seg {
  int tok0, n;  // first row and number of rows
  int ctx;      // keys
  int draft;    // 1: the sequence's drafts follow the keys
  int tab;      // first block-table entry
  int bad;      // a length was clamped
};

__device__ __forceinline__ Seg seg_of(const PagedArgs& a, int i) {
  Seg s;
  s.draft = s.bad = 0;
  if (!a.prefix) {
    const int r0 = a.cu_q[i], r1 = a.cu_q[i + 1], c = a.seq_ctx[i];
    s.tok0 = min(max(r0, 0), a.n_rows);
    s.n = min(max(r1, s.tok0), a.n_rows) - s.tok0;
    s.ctx = min(max(c, 0), a.nb_max * a.blk);
    s.tab = i * a.nb_max;
    s.bad = s.tok0 != r0 || s.tok0 + s.n != r1 || s.ctx != c || s.n > s.ctx;
  } else if (i == 0) {
    s.tok0 = 0;
    s.n = a.n_shared ? a.B * a.T : 0;
    s.ctx = a.n_shared * a.blk;
    s.tab = 0;
  } else {
    s.tok0 = (i - 1) * a.T;
    s.n = a.T;
    s.ctx = (a.var ? a.seq_len[i - 1] : a.ctx) - a.n_shared * a.blk;
    s.draft = 1;
    s.tab = (i - 1) * a.nb_max + a.n_shared;
  }
  return s;
}

__device__ __forceinline__ int n_segs(const PagedArgs& a) { return a.prefix ? a.B + 1 : a.B; }

// The plan in shared memory.
struct Plan {
  int items[kMaxSegs + 1];  // first item of every segment; [nseg] = all items
  int rows[kMaxSegs];       // first partial row of every segment
  int split[kMaxSegs];      // runs of key tiles (>= 1)
};

__device__ __forceinline__ int ceil_div(int x, int y) { return (x + y - 1) / y; }

// Fill `p` (all threads of the CTA call it; a barrier follows inside). tile:
// tokens per row tile, keys: tokens per key tile, min_run: the fewest key
// tiles that a run is worth.
__device__ inline void make_plan(const PagedArgs& a, Plan* p, int tile, int keys, int min_run) {
  const int nseg = n_segs(a), lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < nseg; i += blockDim.x) {
    const Seg s = seg_of(a, i);
    if (s.bad && blockIdx.x == 0) atomicOr(a.status, SV_FLAG_BAD_LENGTH);
    p->rows[i] = s.n;
    p->split[i] = s.n ? ceil_div(s.ctx, keys) + s.draft : 0;  // key tiles
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int per = ceil_div(nseg, 32), b0 = min(nseg, lane * per), b1 = min(nseg, b0 + per);
    unsigned long long units = 0;
    for (int i = b0; i < b1; ++i)
      units += (unsigned long long)ceil_div(p->rows[i], tile) * a.hv * p->split[i];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) units += __shfl_xor_sync(0xffffffffu, units, off);
    const unsigned long long ctas = min((int)gridDim.x, kMaxPlanCtas);
    const unsigned long long want = (units + 2 * ctas - 1) / (2 * ctas);
    const int run = (int)min(max(want, (unsigned long long)min_run), 1ull << 30);
    // items and partial rows of every segment, scanned
    int items = 0, rows = 0;
    for (int i = b0; i < b1; ++i) {
      const int kt = p->split[i], n = p->rows[i];
      int s = kt > run ? ceil_div(kt, run) : 1;
      if (s > 1) s = ceil_div(kt, ceil_div(kt, s));  // no empty run
      const int it = ceil_div(n, tile) * a.hv * s;
      p->split[i] = s;
      items += it;
      rows += s > 1 || a.prefix ? it * min(tile, n) * a.gs : 0;
      p->rows[i] = s > 1 || a.prefix ? it * min(tile, n) * a.gs : 0;
      p->items[i] = it;
    }
    int ix = items, rx = rows;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, ix, off), z = __shfl_up_sync(0xffffffffu, rx, off);
      if (lane >= off) {
        ix += y;
        rx += z;
      }
    }
    int at = ix - items, row = rx - rows;
    for (int i = b0; i < b1; ++i) {
      const int it = p->items[i], r = p->rows[i];
      p->items[i] = at;
      p->rows[i] = row;
      at += it;
      row += r;
    }
    if (lane == 31) p->items[nseg] = at;
  }
  __syncthreads();
}

struct Item {
  int valid;
  int tok0, ntok;     // rows of the tile
  int head0, heads;   // first query head and number of heads of the group
  int kvh;            // KV head
  int vis0;           // keys that the tile's first token sees (causal form; may be <= 0)
  int causal;         // token i of the tile sees vis0 + i keys, else all of them
  int ctx;            // keys of the segment
  int k0, nk;         // first key tile and number of key tiles of the run
  int draft;          // 1: the run's last key tile is the sequence's drafts
  int draft0;         // draft index of the tile's first token
  int seq;            // sequence (drafts)
  int tab;            // first block-table entry of the segment's keys
  int part;           // first partial row, -1: the run is the whole row (written to out)
  // the unit that the item's partial rows belong to (prompt form): first
  // partial row of its first run, runs, rows between runs
  int unit, runs, run_rows;
};

__device__ inline Item decode_item(const PagedArgs& a, const Plan* p, int idx, int tile, int keys) {
  Item it;
  const int nseg = n_segs(a);
  it.valid = idx < p->items[nseg];
  if (!it.valid) return it;
  int lo = 0, hi = nseg;  // the last segment whose items start at or before idx
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (p->items[m] <= idx) lo = m;
    else hi = m;
  }
  const Seg s = seg_of(a, lo);
  const int runs = p->split[lo], tiles = ceil_div(s.n, tile), local = idx - p->items[lo];
  // neighbours in the list share a head's run of keys (they meet in L2), the
  // rows that see most first
  const int t = tiles - 1 - local % tiles, rest = local / tiles;
  const int run = rest % runs, hv = rest / runs;
  it.tok0 = s.tok0 + t * tile;
  it.ntok = min(tile, s.n - t * tile);
  it.kvh = hv / a.hs;
  it.head0 = it.kvh * a.G + hv % a.hs * a.gs;
  it.heads = min(a.gs, a.G - hv % a.hs * a.gs);
  it.causal = !a.prefix;
  it.ctx = s.ctx;
  it.vis0 = a.prefix ? s.ctx : s.ctx - s.n + t * tile + 1;
  const int last = a.prefix ? s.ctx : max(0, it.vis0 + it.ntok - 1);
  const int kt = ceil_div(last, keys) + s.draft;
  const int len = ceil_div(ceil_div(s.ctx, keys) + s.draft, runs);
  it.k0 = run * len;
  it.nk = max(0, min(kt, it.k0 + len) - it.k0);
  it.draft = s.draft && it.nk > 0 && it.k0 + it.nk == kt;
  it.draft0 = t * tile;
  it.seq = a.prefix ? lo - 1 : lo;
  it.tab = s.tab;
  it.runs = runs;
  it.run_rows = min(tile, s.n) * a.gs;
  it.unit = p->rows[lo] + (hv * tiles + t) * runs * it.run_rows;
  it.part = runs > 1 || a.prefix ? it.unit + run * it.run_rows : -1;
  return it;
}

// One group of partial rows of an output row: `runs` rows, `step` apart.
struct Group {
  long long row;
  int step, runs;
};

template <typename T>
__device__ __forceinline__ void store4(T* dst, float x, float y, float z, float w);
template <>
__device__ __forceinline__ void store4<float>(float* dst, float x, float y, float z, float w) {
  *reinterpret_cast<float4*>(dst) = make_float4(x, y, z, w);
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* dst, float x, float y, float z,
                                                      float w) {
  uint2 u;
  u.x = pack_bf16(x, y);
  u.y = pack_bf16(z, w);
  *reinterpret_cast<uint2*>(dst) = u;
}

// out row = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j over the partial
// rows of up to two groups; a row that saw no key is zero. One warp per row;
// the partial rows are taken in order, so the sum does not depend on which
// CTA merges.
template <typename T>
__device__ inline void merge_row(const PagedArgs& a, const Group (&g)[2], T* dst) {
  const int lane = threadIdx.x & 31, total = g[0].runs + g[1].runs;
  auto row_at = [&](int j) {
    return j < g[0].runs ? g[0].row + (long long)j * g[0].step
                         : g[1].row + (long long)(j - g[0].runs) * g[1].step;
  };
  float M = -INFINITY;
  for (int j = lane; j < total; j += 32) M = fmaxf(M, __ldcg(a.part_ml + row_at(j)).x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  float L = 0.f;
  for (int j0 = 0; j0 < total; j0 += 32) {
    float w = 0.f, wl = 0.f;
    if (j0 + lane < total) {
      const float2 ml = __ldcg(a.part_ml + row_at(j0 + lane));
      w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      wl = w * ml.y;
      // a run without a visible key has weight 0 (a NaN maximum stays one)
    }
    const int nj = min(32, total - j0);
#pragma unroll 4
    for (int j = 0; j < nj; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      L += __shfl_sync(0xffffffffu, wl, j);
      const float* src = a.part_o + row_at(j0 + j) * a.d;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 4 * lane + 128 * c;
        if (col < a.d) {
          const float4 o = __ldcg(reinterpret_cast<const float4*>(src + col));
          acc[c].x += wj * o.x;
          acc[c].y += wj * o.y;
          acc[c].z += wj * o.z;
          acc[c].w += wj * o.w;
        }
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int col = 4 * lane + 128 * c;
    if (col < a.d) store4<T>(dst + col, acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv);
  }
}

// What a finished item leaves to merge: in the prompt form its own unit, in
// the prefix form the drafts of (sequence, head group) pairs. `units` (shared
// memory) receives the units that this arrival completed. Called by `nthr`
// threads (tid in [0, nthr)) after every partial row of the item is written
// and ordered before (barrier and device-scope fence); the caller
// synchronises before reading the list. *n must be 0 on entry.
__device__ inline void arrive_item(const PagedArgs& a, const Plan* p, const Item& it, int tile,
                                   int tid, int nthr, int* units, int* n) {
  const int hv = it.kvh * a.hs + (it.head0 - it.kvh * a.G) / a.gs;
  if (!a.prefix) {
    if (tid == 0) {
      const unsigned old = arrive_acq_rel(a.unit_ctr + it.unit);
      if (old + 1 == (unsigned)it.runs) units[(*n)++] = 0;
      else if (old >= (unsigned)it.runs) atomicOr(a.status, SV_FLAG_STALE_WORKSPACE);
    }
    return;
  }
  const int b0 = it.tok0 / a.T, b1 = (it.tok0 + it.ntok - 1) / a.T;
  for (int b = b0 + tid; b <= b1; b += nthr) {
    // arrivals that complete the pair: the runs of every shared row tile its
    // drafts lie in, and its own
    int need = ceil_div(a.T, tile) * p->split[b + 1];
    if (a.n_shared) need += ((b * a.T + a.T - 1) / tile - b * a.T / tile + 1) * p->split[0];
    const unsigned old = arrive_acq_rel(a.unit_ctr + b * a.hv + hv);
    if (old + 1 == (unsigned)need) units[atomicAdd(n, 1)] = b;
    else if (old >= (unsigned)need) atomicOr(a.status, SV_FLAG_STALE_WORKSPACE);
  }
}

// Merge one completed unit (see arrive_item) with `nwarp` warps and return
// its count to zero.
template <typename T>
__device__ inline void merge_unit(const PagedArgs& a, const Plan* p, const Item& it, int unit,
                                  int tile, int warp, int nwarp) {
  T* out = static_cast<T*>(a.out);
  if (!a.prefix) {
    for (int r = warp; r < it.ntok * it.heads; r += nwarp) {
      const int t = r / it.heads, g = r % it.heads;
      const Group gr[2] = {{it.unit + t * a.gs + g, it.run_rows, it.runs}, {0, 0, 0}};
      merge_row<T>(a, gr, out + ((size_t)(it.tok0 + t) * a.Hq + it.head0 + g) * a.d);
    }
    if (warp == 0 && (threadIdx.x & 31) == 0) a.unit_ctr[it.unit] = 0;
    return;
  }
  const int b = unit, hv = it.kvh * a.hs + (it.head0 - it.kvh * a.G) / a.gs;
  const int n0 = a.n_shared ? a.B * a.T : 0, tiles0 = ceil_div(n0, tile), rr0 = min(tile, n0) * a.gs;
  const int tiles1 = ceil_div(a.T, tile), rr1 = min(tile, a.T) * a.gs;
  const int s0 = a.n_shared ? p->split[0] : 0, s1 = p->split[b + 1];
  for (int r = warp; r < a.T * it.heads; r += nwarp) {
    const int t = r / it.heads, g = r % it.heads, tok = b * a.T + t;
    const Group gr[2] = {
        {p->rows[0] + (long long)(hv * tiles0 + tok / tile) * s0 * rr0 + tok % tile * a.gs + g, rr0, s0},
        {p->rows[b + 1] + (long long)(hv * tiles1 + t / tile) * s1 * rr1 + t % tile * a.gs + g, rr1, s1}};
    merge_row<T>(a, gr, out + ((size_t)tok * a.Hq + it.head0 + g) * a.d);
  }
  if (warp == 0 && (threadIdx.x & 31) == 0) a.unit_ctr[b * a.hv + hv] = 0;
}

// The scheduler hands out item gridDim.x + old count; the last CTA to leave
// returns both words to zero.
__device__ __forceinline__ int next_item(const PagedArgs& a) {
  return (int)gridDim.x + (int)atomicAdd(a.sched, 1u);
}
__device__ __forceinline__ void leave(const PagedArgs& a) {
  if (arrive_acq_rel(a.sched + 1) + 1 == gridDim.x) {
    a.sched[0] = 0;
    a.sched[1] = 0;
  }
}

}  // namespace paged
}  // namespace sva
