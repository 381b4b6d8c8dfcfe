// Work split, item decoding and the log-sum-exp merge that the paged
// attention kernels share (device code).
//
// A segment's rows are cut into tiles of `tile` tokens, its keys into tiles
// of `keys` tokens (the prefix form's drafts are one more key tile). A unit is
// one row tile of one head group, an item a unit or a run of its key tiles.
// Lengths may live in device memory only, so every CTA derives the same plan
// from them (make_plan).
#pragma once

#include "paged.h"
#include "ptx.h"

namespace sva {
namespace paged {

// Order this thread's plain accesses to shared memory before bulk copies and
// MMAs that a barrier orders behind it.
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

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

// The plan in shared memory: segments in the order in which their units are
// handed out.
struct Plan {
  int first[kMaxSegs + 1];  // what lies before a segment: items, or (stream) cost
  int order[kMaxSegs];      // the segment
  int rows[kMaxSegs];       // prefix form: first partial row
  int split[kMaxSegs];      // prefix form: runs of key tiles (>= 1)
  int stream;               // prompt form: equal shares of the flattened units
};
constexpr int kPlanScratch = 2 * (kMaxSegs + 3);  // ints that make_plan needs besides

constexpr long long kL2Keys = 32ll << 20;  // a quarter of L2

__device__ __forceinline__ int ceil_div(int x, int y) { return (x + y - 1) / y; }
__device__ __forceinline__ int key_tiles(const PagedArgs& a, int keys) {
  return (int)(((unsigned)keys + (1u << a.key_shift) - 1) >> a.key_shift);
}
// What a key tile of an item of n tokens costs: two sets of rows take twice
// the tensor cores' time.
__device__ __forceinline__ int weight_of(const PagedArgs& a, int n) { return n > a.one_set ? 2 : 1; }

// Prompt form: what the units of one head group of a segment cost, in keys of
// one set of rows. Row tile t sees the keys before the segment's rows and
// (t + 1) * tile of its own; starting and ending an item takes as long as
// item_cost key tiles besides.
struct Cost {
  int w, base, tile, tiles;

  // before unit t, and of unit t
  __device__ __forceinline__ int before(int t) const { return w * (t * base + tile * (t * (t + 1) / 2)); }
  __device__ __forceinline__ int of(int t) const { return w * (base + tile * (t + 1)); }
  __device__ __forceinline__ float total() const {
    return (float)w * tiles * (base + 0.5f * tile * (tiles + 1));
  }
  // the unit that position x of the group lies in
  __device__ __forceinline__ int unit_at(int x) const {
    const float b = base + 0.5f * tile, y = (float)x / (w * tile);
    const float p = b / tile;
    int t = min(max((int)(sqrtf(p * p + 2.f * y) - p), 0), tiles - 1);
    while (t > 0 && before(t) > x) --t;
    while (t + 1 < tiles && before(t + 1) <= x) ++t;
    return t;
  }
};

__device__ __forceinline__ Cost cost_of(const PagedArgs& a, int n, int ctx) {
  return {weight_of(a, n), max(0, ctx - n) + (a.item_cost << a.key_shift), a.tile, ceil_div(n, a.tile)};
}

// Fill `p` (all threads of the CTA call it; barriers inside). scratch:
// kPlanScratch ints of shared memory on a 16-byte boundary.
//
// Segments go out in descending order of their units' cost, so that what starts
// last is short (the prefix form's shared segment first).
//
// Prefix form: items go out dynamically. The shared segment's keys are cut into
// the number of runs that is expected to end first (8 trees of 16 drafts over
// 65536 shared tokens: 144 items for 152 CTAs 139 us, 160 items 185 us, 304 items
// 156 us), the sequences' own so that they are about kOwnItemsPerCta items per CTA.
// The partial rows are then at most those of the uncut segments and
// kOwnItemsPerCta + kSharedItemsPerCta items per CTA more.
//
// Prompt form, one of two ways, whichever is expected to end earlier:
//   whole units, handed out dynamically. Ends at about the average load
//     plus part of the longest unit (at least at the longest);
//   stream: the units laid end to end, CTA c taking the c-th equal share, at
//     most two cut units each. Ends at the average load and the join of the cut
//     units, but CTAs on the same keys are far apart in them.
// Few rows over long contexts stream (16 ragged decoding sequences: 154 us cut
// into runs and scheduled, CTAs ending between 60 and 100% of it, 119 us as
// equal shares), long prompts do not. What whole units lose at their end (half of the
// longest unit, a tenth when every CTA has four or more), the 5% by which streaming has to
// win and kStreamCost are estimates from such runs; they have not been swept around
// the point where the two ways meet.
__device__ inline void make_plan(const PagedArgs& a, Plan* p, int* scratch) {
  const int nseg = n_segs(a), lane = threadIdx.x & 31, padded = (nseg + 3) & ~3;
  int* kts = scratch;                         // cost of segment i's last unit
  int* ns = scratch + ((kMaxSegs + 3) & ~3);  // rows of segment i
  int* ctxs = p->rows;                        // prompt form: keys of segment i
  for (int i = threadIdx.x; i < padded; i += blockDim.x) {
    kts[i] = -1;
    if (i >= nseg) continue;
    const Seg s = seg_of(a, i);
    if (s.bad && blockIdx.x == 0) atomicOr(a.status, SV_FLAG_BAD_LENGTH);
    ns[i] = s.n;
    if (a.prefix) {
      kts[i] = s.n ? key_tiles(a, s.ctx) + s.draft : 0;
    } else {
      const Cost c = cost_of(a, s.n, s.ctx);
      kts[i] = s.n ? (int)fminf((float)c.w * ((float)c.base + (float)c.tile * c.tiles), 1e9f) : 0;
      ctxs[i] = s.ctx;
    }
  }
  __syncthreads();
  if (nseg > 1) {
    for (int i = threadIdx.x; i < nseg; i += blockDim.x) {
      const int kt = kts[i];
      int rank = 0;
      for (int j = 0; j < padded; j += 4) {
        const int4 k = *reinterpret_cast<const int4*>(kts + j);
        rank += (k.x > kt || (k.x == kt && j < i)) + (k.y > kt || (k.y == kt && j + 1 < i)) +
                (k.z > kt || (k.z == kt && j + 2 < i)) + (k.w > kt || (k.w == kt && j + 3 < i));
      }
      // the shared segment counts as the costliest
      if (a.prefix) rank = i == 0 ? 0 : rank + (kts[0] < kt);
      p->order[rank] = i;
    }
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    const int per = nseg > 32 ? (nseg + 31) >> 5 : 1, b0 = min(nseg, lane * per), b1 = min(nseg, b0 + per);
    int at = 0, row = 0;  // this lane's totals, then what lies before them
    if (a.prefix) {
      unsigned long long units = 0;
      float own = 0.f;  // cost of the sequences' own units, in key tiles of one set
      for (int i = b0; i < b1; ++i) {
        const int n = ceil_div(ns[i], a.tile) * a.hv;
        units += (unsigned long long)n * kts[i];
        if (i) own += (float)n * (kts[i] * weight_of(a, ns[i]) + a.item_cost);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        units += __shfl_xor_sync(0xffffffffu, units, off);
        own += __shfl_xor_sync(0xffffffffu, own, off);
      }
      const unsigned parts = kOwnItemsPerCta * a.ctas;
      const unsigned long long want =
          units >> 31 ? (units + parts - 1) / parts : ((unsigned)units + parts - 1) / parts;
      const int run = (int)min(max(want, (unsigned long long)a.min_run), 1ull << 30);
      // Lane l tries l + 1 runs and l + 33: rounds of shared items on every CTA, the
      // last one shared with the own ones, and what joining takes.
      const int kt0 = kts[0], n0 = ceil_div(ns[0], a.tile) * a.hv;
      const float join = (float)a.n_rows * a.Hq * (1.f / 16384.f);
      float best = INFINITY;
      int shared = 1;
      for (int s = lane + 1; s <= 64; s += 32) {
        if (s > 1 && (n0 * (s - 1) > kSharedItemsPerCta * a.ctas || s * a.min_run > kt0)) continue;
        const int len = ceil_div(kt0, s), items = n0 * (len ? ceil_div(kt0, len) : 0);
        const float cost = (float)(len * weight_of(a, ns[0]) + a.item_cost);
        const int rounds = items / a.ctas, rest = items - rounds * a.ctas;
        const float end = rounds * cost + fmaxf(rest ? cost : 0.f, (rest * cost + own) / a.ctas) + join * s;
        if (end < best) {
          best = end;
          shared = s;
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const float e = __shfl_xor_sync(0xffffffffu, best, off);
        const int s = __shfl_xor_sync(0xffffffffu, shared, off);
        if (e < best || (e == best && s < shared)) {
          best = e;
          shared = s;
        }
      }
      for (int i = b0; i < b1; ++i) {
        const int id = p->order[i], kt = kts[id], n = ns[id];
        int s = id == 0 ? shared : kt > run ? ceil_div(kt, run) : 1;
        if (s > 1) s = ceil_div(kt, ceil_div(kt, s));  // no empty run
        const int it = ceil_div(n, a.tile) * a.hv * s;
        p->split[i] = s;
        p->first[i] = it;
        p->rows[i] = it * min(a.tile, n) * a.gs;
        at += it;
        row += p->rows[i];
      }
    } else {
      float cost = 0.f, units = 0.f, most = 0.f;
      for (int i = b0; i < b1; ++i) {
        if (nseg == 1) p->order[0] = 0;
        const int id = p->order[i];
        if (ns[id] == 0) continue;
        const Cost c = cost_of(a, ns[id], ctxs[id]);
        units += (float)c.tiles * a.hv;
        cost += c.total() * a.hv;
        most = fmaxf(most, (float)(kts[id] - c.w * (a.item_cost << a.key_shift)));  // (both ways have the ends)
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        cost += __shfl_xor_sync(0xffffffffu, cost, off);
        units += __shfl_xor_sync(0xffffffffu, units, off);
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
      }
      const float ctas = (float)a.ctas, load = cost / ctas;
      const float whole = units <= ctas ? most : fmaxf(most, load + (units < 4.f * ctas ? 0.5f : 0.1f) * most);
      const bool stream = cost < 1e9f && 1.05f * load + (kStreamCost << a.key_shift) < whole;
      if (lane == 0) p->stream = stream;
      for (int i = b0; i < b1; ++i) {
        const int id = p->order[i];
        const Cost c = cost_of(a, ns[id], ctxs[id]);
        p->first[i] = a.hv * (stream ? c.before(c.tiles) : c.tiles);
        at += p->first[i];
      }
    }
    int ax = at, rx = row;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, ax, off), y = __shfl_up_sync(0xffffffffu, rx, off);
      if (lane >= off) {
        ax += x;
        rx += y;
      }
    }
    at = ax - at;
    row = rx - row;
    for (int i = b0; i < b1; ++i) {
      const int x = p->first[i];
      p->first[i] = at;
      at += x;
      if (a.prefix) {
        const int r = p->rows[i];
        p->rows[i] = row;
        row += r;
      }
    }
    if (lane == 31) p->first[nseg] = at;
  }
  // the scratch is done with: the bulk copies that the caller may send there come behind it
  fence_proxy_async_shared();
  __syncthreads();
}

// The last segment (in plan order) that starts at or before x.
__device__ __forceinline__ int find_seg(const Plan* p, int nseg, int x) {
  int lo = 0, hi = nseg;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (p->first[m] <= x) lo = m;
    else hi = m;
  }
  return lo;
}

// Stream: where CTA c's share of a total starts, and the CTA that position x
// lies in.
__device__ __forceinline__ int share_start(int total, int ctas, int c) {
  const int q = total / ctas, r = total % ctas;
  return c * q + min(c, r);
}
__device__ __forceinline__ int share_of(int total, int ctas, int x) {
  const int q = total / ctas, r = total % ctas, head = r * (q + 1);
  return x < head ? x / (q + 1) : r + (x - head) / q;
}
// Stream: partial rows of a cut unit lie in slots of slot_rows rows, two per
// CTA: 2 c for the end (or middle) of a unit that CTA c starts with, 2 c + 1 for
// the beginning of the unit that it ends with.
__device__ __forceinline__ int slot_rows(const PagedArgs& a) { return min(a.tile, a.n_rows) * a.gs; }

// What the merge launch needs of the prefix form's plan, by segment.
__device__ inline void save_plan(const PagedArgs& a, const Plan* p) {
  if (!a.prefix || blockIdx.x) return;
  for (int i = threadIdx.x; i < n_segs(a); i += blockDim.x)
    a.segs[p->order[i]] = make_int2(p->rows[i], p->split[i]);
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
};

// The item of row tile t and head group hv of segment `id` over key tiles
// [k0, k1).
__device__ __forceinline__ Item make_item(const PagedArgs& a, const Seg& s, int id, int t, int hv, int k0,
                                          int k1) {
  Item it;
  it.valid = 1;
  it.tok0 = s.tok0 + t * a.tile;
  it.ntok = min(a.tile, s.n - t * a.tile);
  it.kvh = a.hs > 1 ? hv / a.hs : hv;
  const int sub = (hv - it.kvh * a.hs) * a.gs;
  it.head0 = it.kvh * a.G + sub;
  it.heads = min(a.gs, a.G - sub);
  it.causal = !a.prefix;
  it.ctx = s.ctx;
  it.vis0 = a.prefix ? s.ctx : s.ctx - s.n + t * a.tile + 1;
  const int last = a.prefix ? s.ctx : max(0, it.vis0 + it.ntok - 1);
  const int kt = key_tiles(a, last) + s.draft;
  it.k0 = k0;
  it.nk = max(0, min(kt, k1) - k0);
  it.draft = s.draft && it.nk > 0 && k0 + it.nk == kt;
  it.draft0 = t * a.tile;
  it.seq = a.prefix ? id - 1 : id;
  it.tab = s.tab;
  it.part = -1;
  return it;
}

// A CTA's place in the plan.
struct Cursor {
  int at, end;  // item number, or (stream) position in the flattened cost
};

// One thread calls it, and next_item.
__device__ __forceinline__ Cursor start_cursor(const PagedArgs& a, const Plan* p) {
  if (!a.prefix) a.joins[blockIdx.x].more = 0;
  if (a.prefix || !p->stream) return {(int)blockIdx.x, 0};
  const int total = p->first[n_segs(a)];
  return {share_start(total, a.ctas, blockIdx.x), share_start(total, a.ctas, blockIdx.x + 1)};
}

// The item at the cursor (valid = 0 behind the last one), and the cursor
// moved on.
__device__ inline Item next_item(const PagedArgs& a, const Plan* p, Cursor* c) {
  const int nseg = n_segs(a);
  if (!a.prefix && p->stream) {
    if (c->at >= c->end) {
      Item it;
      it.valid = 0;
      return it;
    }
    const int lo = find_seg(p, nseg, c->at), id = p->order[lo];
    const Seg s = seg_of(a, id);
    const Cost k = cost_of(a, s.n, s.ctx);
    const int group = k.before(k.tiles), local = c->at - p->first[lo], hv = local / group;
    const int t = k.unit_at(local - hv * group), cost = k.of(t);
    const int off = local - hv * group - k.before(t), upto = min(cost, off + c->end - c->at);
    // the key tile that position x of a unit lies in
    auto tile_at = [&](int x) {
      return key_tiles(a, max(0, (x + k.w - 1) / k.w - (a.item_cost << a.key_shift)));
    };
    Item it = make_item(a, s, id, t, hv, tile_at(off), upto == cost ? 1 << 28 : tile_at(upto));
    if (off > 0 || upto < cost) it.part = (2 * blockIdx.x + (off > 0 ? 0 : 1)) * slot_rows(a);
    if (off == 0 && upto < cost)  // begun here, ended by others: the merge's to join
      a.joins[blockIdx.x] = {share_of(p->first[nseg], a.ctas, c->at + cost - 1) - (int)blockIdx.x,
                             it.tok0, it.ntok, it.head0, it.heads};
    c->at += upto - off;
    return it;
  }
  if (c->at >= p->first[nseg]) {
    Item it;
    it.valid = 0;
    return it;
  }
  const int lo = find_seg(p, nseg, c->at), id = p->order[lo];
  const Seg s = seg_of(a, id);
  const int runs = a.prefix ? p->split[lo] : 1, tiles = ceil_div(s.n, a.tile);
  // Neighbours in the list share keys (they meet in L2): groups of heads whose
  // keys and values fit kL2Keys, in a group run by run, in a run the rows
  // that see most first.
  const unsigned kv = (unsigned)(((long long)s.ctx * a.d * a.elt) >> 9) + 1;  // KB of keys and values
  const int fit = min((int)((unsigned)(kL2Keys >> 10) / kv) + 1, a.hv);
  const int gh = fit < a.hv ? ceil_div(a.hv, ceil_div(a.hv, fit)) : a.hv, per = gh * tiles * runs;
  const int local = c->at - p->first[lo], h0 = local / per * gh, in = local % per;
  const int gw = min(gh, a.hv - h0), u = in / gw, hv = h0 + in - u * gw;
  const int run = u / tiles, t = tiles - 1 - (u - run * tiles);
  const int len = a.prefix ? ceil_div(key_tiles(a, s.ctx) + s.draft, runs) : 1 << 28;
  Item it = make_item(a, s, id, t, hv, run * len, (run + 1) * len);
  // partial rows of a segment lie by head group, row tile, run, token, head
  if (a.prefix) it.part = p->rows[lo] + ((hv * tiles + t) * runs + run) * min(a.tile, s.n) * a.gs;
  c->at = (int)gridDim.x + (int)atomicAdd(a.sched, 1u);
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
  float2 ml = make_float2(-INFINITY, 0.f);  // of partial row j0 + lane
  if (lane < total) ml = __ldcg(a.part_ml + row_at(lane));
  float M = ml.x;
  for (int j = lane + 32; j < total; j += 32) M = fmaxf(M, __ldcg(a.part_ml + row_at(j)).x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  float L = 0.f;
  for (int j0 = 0; j0 < total; j0 += 32) {
    float w = 0.f, wl = 0.f;
    if (j0 + lane < total) {
      if (j0) ml = __ldcg(a.part_ml + row_at(j0 + lane));
      // a run without a visible key has weight 0 (a NaN sum stays one)
      w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      wl = w * ml.y;
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

// A CTA has drawn its last item; the last CTA to leave returns the scheduler's
// words to zero.
__device__ __forceinline__ void leave(const PagedArgs& a) {
  if (arrive_acq_rel(a.sched + 1) + 1 == gridDim.x) {
    a.sched[0] = 0;
    a.sched[1] = 0;
  }
}

}  // namespace paged
}  // namespace sva
