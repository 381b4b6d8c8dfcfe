// Work split, item decoding and the log-sum-exp merge that the paged
// attention kernels share (device code).
//
// A segment's rows are cut into tiles of `tile` tokens, its keys into tiles
// of `keys` tokens (the prefix form's drafts are one more key tile). An item
// is one row tile of one head group over a run of key tiles. Lengths may live
// in device memory only, so every CTA derives the same plan from them: a
// segment whose row tiles see more than C key tiles is cut into s =
// ceil(kt / C) runs, with C such that the grid gets about kItemsPerCta items per
// CTA. That bounds the partial rows by a number the host knows: the items of
// cut segments are at most twice sum(tiles * kt) / C <= 2 * kItemsPerCta * CTAs.
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

// The plan in shared memory: segments in the order in which their items are
// handed out.
struct Plan {
  int items[kMaxSegs + 1];  // first item of every segment; [nseg] = all items
  int rows[kMaxSegs];       // first partial row of every segment
  int split[kMaxSegs];      // runs of key tiles (>= 1)
  int order[kMaxSegs];      // the segment
};
constexpr int kPlanScratch = 2 * (kMaxSegs + 3);  // ints that make_plan needs besides

constexpr long long kL2Keys = 32ll << 20;  // a quarter of L2

__device__ __forceinline__ int ceil_div(int x, int y) { return (x + y - 1) / y; }

// Fill `p` (all threads of the CTA call it; barriers inside). scratch:
// kPlanScratch ints of shared memory on a 16-byte boundary.
//
// Prompt segments go out in descending order of key tiles, so that what starts
// last is short (a dynamic schedule is as good as its last items are small).
// The prefix form keeps its order: the shared segment comes first.
__device__ inline void make_plan(const PagedArgs& a, Plan* p, int* scratch) {
  const int nseg = n_segs(a), lane = threadIdx.x & 31, padded = (nseg + 3) & ~3;
  int* kts = scratch;                    // key tiles of segment i
  int* ns = scratch + ((kMaxSegs + 3) & ~3);  // rows of segment i
  for (int i = threadIdx.x; i < padded; i += blockDim.x) {
    kts[i] = -1;
    if (i >= nseg) continue;
    const Seg s = seg_of(a, i);
    if (s.bad && blockIdx.x == 0) atomicOr(a.status, SV_FLAG_BAD_LENGTH);
    ns[i] = s.n;
    kts[i] = s.n ? ceil_div(s.ctx, a.keys) + s.draft : 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nseg; i += blockDim.x) {
    int rank = i;
    if (!a.prefix && nseg > 1) {
      const int kt = kts[i];
      rank = 0;
      for (int j = 0; j < padded; j += 4) {
        const int4 k = *reinterpret_cast<const int4*>(kts + j);
        rank += (k.x > kt || (k.x == kt && j < i)) + (k.y > kt || (k.y == kt && j + 1 < i)) +
                (k.z > kt || (k.z == kt && j + 2 < i)) + (k.w > kt || (k.w == kt && j + 3 < i));
      }
    }
    p->order[rank] = i;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int per = ceil_div(nseg, 32), b0 = min(nseg, lane * per), b1 = min(nseg, b0 + per);
    unsigned long long units = 0;
    for (int i = b0; i < b1; ++i)
      units += (unsigned long long)ceil_div(ns[i], a.tile) * a.hv * kts[i];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) units += __shfl_xor_sync(0xffffffffu, units, off);
    const unsigned long long parts = (unsigned long long)a.per_cta * a.ctas;
    const unsigned long long want = (units + parts - 1) / parts;
    const int run = (int)min(max(want, (unsigned long long)a.min_run), 1ull << 30);
    // items and partial rows of every segment, scanned
    int items = 0, rows = 0;
    for (int i = b0; i < b1; ++i) {
      const int kt = kts[p->order[i]], n = ns[p->order[i]];
      int s = kt > run ? ceil_div(kt, run) : 1;
      if (s > 1) s = ceil_div(kt, ceil_div(kt, s));  // no empty run
      const int it = ceil_div(n, a.tile) * a.hv * s;
      const int r = s > 1 || a.prefix ? it * min(a.tile, n) * a.gs : 0;
      p->split[i] = s;
      p->items[i] = it;
      p->rows[i] = r;
      items += it;
      rows += r;
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
  // the partial rows of all runs of this row tile and head group: the first
  // one, the number of runs, rows between runs
  int unit, runs, run_rows;
};

__device__ inline Item decode_item(const PagedArgs& a, const Plan* p, int idx) {
  const int tile = a.tile, keys = a.keys;
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
  const int id = p->order[lo];
  const Seg s = seg_of(a, id);
  const int runs = p->split[lo], tiles = ceil_div(s.n, tile);
  // Neighbours in the list share keys (they meet in L2): groups of heads whose
  // keys and values fit kL2Keys, in a group run by run, in a run the rows
  // that see most first.
  const long long kv = (long long)s.ctx * a.d * 2 * a.elt + 1;
  const int fit = (int)min(max(kL2Keys / kv, 1ll), (long long)a.hv);
  const int gh = ceil_div(a.hv, ceil_div(a.hv, fit)), per = gh * tiles * runs;
  const int local = idx - p->items[lo], h0 = local / per * gh, in = local % per;
  const int gw = min(gh, a.hv - h0), hv = h0 + in % gw;
  const int t = tiles - 1 - in / gw % tiles, run = in / gw / tiles;
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
  it.seq = a.prefix ? id - 1 : id;
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
#pragma unroll 8
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

// A prompt item's partial rows are written and ordered (barrier and
// device-scope fence): true when they were the last of their unit, which the
// caller then merges. One thread calls it.
__device__ __forceinline__ bool arrive_unit(const PagedArgs& a, const Item& it) {
  const unsigned old = arrive_acq_rel(a.unit_ctr + it.unit);
  if (old >= (unsigned)it.runs) atomicOr(a.status, SV_FLAG_STALE_WORKSPACE);
  return old + 1 == (unsigned)it.runs;
}

// Merge a prompt item's unit with `nwarp` warps and return its count to zero.
template <typename T>
__device__ inline void merge_unit(const PagedArgs& a, const Item& it, int warp, int nwarp) {
  T* out = static_cast<T*>(a.out);
  for (int r = warp; r < it.ntok * it.heads; r += nwarp) {
    const int t = r / it.heads, g = r % it.heads;
    const Group gr[2] = {{it.unit + t * a.gs + g, it.run_rows, it.runs}, {0, 0, 0}};
    merge_row<T>(a, gr, out + ((size_t)(it.tok0 + t) * a.Hq + it.head0 + g) * a.d);
  }
  if (warp == 0 && (threadIdx.x & 31) == 0) a.unit_ctr[it.unit] = 0;
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
