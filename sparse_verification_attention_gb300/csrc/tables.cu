// Pages for requests whose lengths change, and K/V rows into those pages: the
// two steps of a serving loop between "these requests run now" and the first
// attention over the cache.
#include <atomic>

#include "internal.h"
#include "paged.h"
#include "ptx.h"

namespace sva {
namespace {

constexpr int kTabThreads = 1024;
constexpr int kTabPer = kMaxRequests / kTabThreads;  // requests per thread
constexpr int kTabTokens = 4;                        // tokens per thread and round

// A store to shared memory of any CTA of the cluster, and the two halves of
// cluster_sync_all.
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// x / blk of a non-negative x: pages are powers of two nearly always.
__device__ __forceinline__ int block_of(const TablesArgs& a, int x) {
  return a.blk_shift >= 0 ? x >> a.blk_shift : x / a.blk;
}

struct Lens {
  int o, n;    // old and new length, clamped to the table's width
  int held;    // blocks held before
  int need;    // blocks needed after
  int keep;    // first block let go (blocks [keep, held) are, if any)
};

__device__ __forceinline__ Lens lens_of(const TablesArgs& a, int b) {
  const int most = a.nb_max * a.blk;
  Lens l;
  l.o = min(max(a.old_len[b], 0), most);
  l.n = min(max(a.new_len[b], 0), most);
  l.held = block_of(a, l.o + a.blk - 1);
  l.need = block_of(a, l.n + a.blk - 1);
  l.keep = max(l.need, a.pinned ? a.pinned[b] : 0);
  return l;
}

// The last index b in [0, B) with start[b] <= i (start is non-decreasing and
// start[0] = 0): the request that item i of a scanned list belongs to.
__device__ __forceinline__ int owner(const int* start, int B, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (start[m] <= i) lo = m;
    else hi = m;
  }
  return lo;
}

// Block of item i of the releases, in [0, num_pages), -1 for an entry outside the
// pool, kNoPage for a block that never got one.
constexpr int kNoPage = -2;
__device__ __forceinline__ int released_page(const TablesArgs& a, const int* s_rel, int i) {
  const int b = owner(s_rel, a.B, i);
  const int page = a.block_table[(size_t)b * a.nb_max + lens_of(a, b).keep + i - s_rel[b]];
  return page == -1 ? kNoPage : page < 0 || page >= a.num_pages ? -1 : page;
}

// Push the releases again, the blocks without a page left out (all threads of one
// CTA): from the last one on, a round of kTabThreads at a time. Returns their number.
__device__ inline int push_held(const TablesArgs& a, const int* s_rel, int R, int count) {
  __shared__ int s_held[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
  for (int end = R; end > 0; end -= kTabThreads) {
    const int i = end - 1 - (int)threadIdx.x;
    const int page = i >= 0 ? released_page(a, s_rel, i) : kNoPage;
    const unsigned held = __ballot_sync(0xffffffffu, page != kNoPage);
    if (lane == 0) s_held[warp] = __popc(held);
    __syncthreads();
    int rank = before + __popc(held & ((1u << lane) - 1u));
    for (int w = 0; w < 32; ++w) {
      if (w < warp) rank += s_held[w];
      before += s_held[w];
    }
    if (page != kNoPage && (long long)count + rank < a.num_pages) a.free_pages[count + rank] = page;
    __syncthreads();
  }
  return before;
}

// One thread-block cluster does the whole call. Every CTA scans the lengths
// of all requests into shared memory (three exclusive sums: blocks let go,
// blocks taken, new tokens); the CTAs then share the lists' items. The
// free-page stack is addressed by rank, not popped: item i of the ascending
// (request, block) list of releases goes to stack[count + R - 1 - i], item i
// of the allocations comes from stack[count + R - 1 - i], so the result does
// not depend on the order of execution and a release undoes the allocation it
// mirrors. One cluster barrier separates the two. (Blocks for which an earlier call
// found no page have none to give back and break that numbering: where a thread
// meets one, all CTAs are told ahead of the barrier, and one CTA pushes the
// releases again, counted.)
//
// Latency bound (a step of a decoding batch moves a few KB): one launch, no
// atomics, two dependent rounds of loads before the barrier, two after. In a
// replayed graph a step of 8 requests takes 4.9 us and the admission of 144 prompts
// (74,000 tokens) 9.9 us; making the call takes the host about 10 us.
__global__ void __launch_bounds__(kTabThreads) build_tables_kernel(const __grid_constant__ TablesArgs a) {
  extern __shared__ int s_start[];
  int* s_rel = s_start;                  // [B + 1]
  int* s_alc = s_rel + a.B + 1;          // [B + 1]
  int* s_tok = s_alc + a.B + 1;          // [B + 1]
  int* s_old = s_tok + a.B + 1;          // [B]: old lengths
  __shared__ long long s_warp[3][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ncta = gridDim.x, rank = blockIdx.x;
  const int step = ncta * kTabThreads, first = rank * kTabThreads + tid;
  unsigned flags = 0;
  __shared__ int s_missing, s_pushed;  // written by any CTA of the cluster
  if (tid == 0) s_missing = 0;
  __syncwarp();
  if (ncta > 1) cluster_arrive();
  auto tell = [&](int* word, int value) {
    for (int r = 0; r < ncta; ++r)
      if (ncta > 1) st_cluster_u32(cluster_map(smem_u32(word), r), value);
      else *word = value;
  };

  pdl_wait();
  pdl_trigger();

  // thread t owns the requests [t * per, (t + 1) * per)
  const int per = (a.B + kTabThreads - 1) / kTabThreads;
  long long sum[3] = {0, 0, 0};
  int rel[kTabPer], alc[kTabPer], tok[kTabPer];
#pragma unroll
  for (int e = 0; e < kTabPer; ++e) {
    const int b = tid * per + e;
    rel[e] = alc[e] = tok[e] = 0;
    if (e < per && b < a.B) {
      const Lens l = lens_of(a, b);
      if (l.o != a.old_len[b] || l.n != a.new_len[b]) flags |= SV_FLAG_BAD_LENGTH;
      rel[e] = max(0, l.held - l.keep);
      alc[e] = max(0, l.need - l.held);
      tok[e] = max(0, l.n - l.o);
      s_old[b] = l.o;
    }
    sum[0] += rel[e];
    sum[1] += alc[e];
    sum[2] += tok[e];
  }
  long long mine[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long x = sum[k];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    mine[k] = x - sum[k];
    if (lane == 31) s_warp[k][warp] = x;
  }
  __syncthreads();
  if (warp < 3) {
    long long x = s_warp[warp][lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    s_warp[warp][lane] = x;  // inclusive over warps
  }
  __syncthreads();
  auto sat = [](long long x) { return (int)min(x, 0x7fffffffll); };
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long x = mine[k] + (warp ? s_warp[k][warp - 1] : 0);
    int* dst = k == 0 ? s_rel : k == 1 ? s_alc : s_tok;
    const int* cnt = k == 0 ? rel : k == 1 ? alc : tok;
#pragma unroll
    for (int e = 0; e < kTabPer; ++e) {
      const int b = tid * per + e;
      if (e < per && b < a.B) dst[b] = sat(x);
      x += cnt[e];
    }
  }
  const int R = sat(s_warp[0][31]), A = sat(s_warp[1][31]), N = sat(s_warp[2][31]);
  if (tid == 0) {
    s_rel[a.B] = R;
    s_alc[a.B] = A;
    s_tok[a.B] = N;
  }
  __syncthreads();

  const int count = min(max(*a.free_count, 0), a.num_pages);
  if (count != *a.free_count || N > a.n_max) flags |= SV_FLAG_BAD_LENGTH;

  // releases, onto the stack in descending (request, block) order
  bool missing = false;
  for (int i = first; i < R; i += step) {
    const int page = released_page(a, s_rel, i);
    if (page == -1) flags |= SV_FLAG_BAD_PAGE;
    missing |= page == kNoPage;
    const long long at = (long long)count + R - 1 - i;
    if (at < a.num_pages) a.free_pages[at] = page;
  }
  __syncwarp();
  if (ncta > 1) cluster_wait();  // every s_missing has been set to zero
  if (missing) tell(&s_missing, 1);
  __syncwarp();
  if (ncta > 1) cluster_sync_all();
  else __syncthreads();
  int pushed = R;
  if (s_missing) {
    if (rank == 0) {
      pushed = push_held(a, s_rel, R, count);
      if (tid == 0) tell(&s_pushed, pushed);
      __syncwarp();
    }
    if (ncta > 1) cluster_sync_all();
    else __syncthreads();
    pushed = s_pushed;
  }
  const int top = min((long long)count + pushed, (long long)a.num_pages);
  if ((long long)count + pushed > a.num_pages) flags |= SV_FLAG_BAD_LENGTH;

  // allocations, from the top of the stack in ascending (request, block) order
  auto taken = [&](int i) {
    const int at = top - 1 - i;
    if (at < 0) return -2;  // the pool has no page left
    const int page = __ldcg(a.free_pages + at);
    return page < 0 || page >= a.num_pages ? -1 : page;
  };
  for (int i = first; i < A; i += step) {
    const int b = owner(s_alc, a.B, i);
    const int page = taken(i);
    if (page < 0) flags |= page == -2 ? SV_FLAG_NO_PAGE : SV_FLAG_BAD_PAGE;
    a.block_table[(size_t)b * a.nb_max + lens_of(a, b).held + i - s_alc[b]] = max(page, -1);
  }
  // slots and positions of the new tokens; -1 behind the last one. Four tokens
  // per thread and round: their searches and page loads overlap.
  for (int i0 = first; i0 < a.n_max; i0 += kTabTokens * step) {
    int pos[kTabTokens], page[kTabTokens];
#pragma unroll
    for (int e = 0; e < kTabTokens; ++e) {
      const int i = i0 + e * step;
      pos[e] = page[e] = -1;
      if (i >= N || i >= a.n_max) continue;
      const int b = owner(s_tok, a.B, i);
      pos[e] = s_old[b] + i - s_tok[b];
      const int j = block_of(a, pos[e]), held = block_of(a, s_old[b] + a.blk - 1);
      if (j < held) {  // the last block held before, partly filled
        page[e] = a.block_table[(size_t)b * a.nb_max + j];
        if (page[e] < 0 || page[e] >= a.num_pages) {
          flags |= SV_FLAG_BAD_PAGE;
          page[e] = -1;
        }
      } else {
        page[e] = taken(s_alc[b] + j - held);  // flagged above
      }
    }
#pragma unroll
    for (int e = 0; e < kTabTokens; ++e) {
      const int i = i0 + e * step;
      if (i >= a.n_max) continue;
      a.slot_map[i] = page[e] >= 0 ? page[e] * a.blk + pos[e] - block_of(a, pos[e]) * a.blk : -1;
      if (a.positions) a.positions[i] = pos[e];
    }
  }
  if (rank == 0) {
    for (int b = tid; b <= a.B; b += kTabThreads) a.cu_new[b] = s_tok[b];
    if (tid == 0) *a.free_count_out = max(0, top - A);
  }
  if (flags && a.status) atomicOr(a.status, flags);
}

// ---------------------------------------------------------------- K/V rows
constexpr int kWriteThreads = 256;
constexpr int kWriteRows = 4;  // tokens per thread

// Chunk c (16 bytes) of a token's [Hkv, d] row goes to head c / per_head of
// its page. A CTA takes kWriteRows * (kWriteThreads / width) tokens; a thread
// keeps one chunk column and issues all its loads before its stores. (Loads past
// L1: under a programmatic launch the rows may be written while this grid is
// already resident, so they are not read-only for its lifetime.)
// Bound by HBM: every byte is read once and written once. 126.5 MB of prompt rows
// take 21.9 us, 5.77 TB/s.
__global__ void __launch_bounds__(kWriteThreads) write_kv_kernel(const __grid_constant__ WriteArgs a) {
  const int per_head = a.row_bytes / 16, chunks = a.Hkv * per_head;
  const int width = min(chunks, kWriteThreads), side = kWriteThreads / width;
  const int c0 = threadIdx.x % width, t0 = threadIdx.x / width;
  pdl_wait();
  pdl_trigger();
  if (t0 >= side) return;
  const long long base = (long long)blockIdx.x * side * kWriteRows + t0;
  long long dst[kWriteRows];
#pragma unroll
  for (int e = 0; e < kWriteRows; ++e) {
    const long long t = base + (long long)e * side;
    const int slot = t < a.n ? a.slots[t] : -1;
    dst[e] = -1;
    if (slot >= 0) {
      const int page = slot / a.blk;
      if (page < a.num_pages)
        dst[e] = ((long long)page * a.Hkv * a.blk + slot % a.blk) * a.row_bytes;
    }
    if (slot < -1 || (slot >= 0 && dst[e] < 0))
      if (a.status && c0 == 0) atomicOr(a.status, SV_FLAG_BAD_PAGE);
  }
  for (int c = c0; c < chunks; c += width) {
    const long long off = (long long)(c / per_head) * a.blk * a.row_bytes + (c % per_head) * 16;
    uint4 k[kWriteRows], v[kWriteRows];
#pragma unroll
    for (int e = 0; e < kWriteRows; ++e) {
      if (dst[e] >= 0) {
        const long long t = base + (long long)e * side;
        k[e] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) + t * a.k_stride) + c);
        v[e] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const char*>(a.v) + t * a.v_stride) + c);
      }
    }
#pragma unroll
    for (int e = 0; e < kWriteRows; ++e) {
      if (dst[e] >= 0) {
        *reinterpret_cast<uint4*>(static_cast<char*>(a.k_pool) + dst[e] + off) = k[e];
        *reinterpret_cast<uint4*>(static_cast<char*>(a.v_pool) + dst[e] + off) = v[e];
      }
    }
  }
}

}  // namespace

cudaError_t launch_build_tables(const TablesArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)4 * (a.B + 1) * sizeof(int);
  const int dev = current_device();
  static std::atomic<int> ready[kMaxDevices];
  if (!ready[dev].load()) {
    const cudaError_t e =
        cudaFuncSetAttribute(build_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * (kMaxRequests + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    const cudaError_t e16 = cudaFuncSetAttribute(
        build_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e16 != cudaSuccess) return e16;
    ready[dev].store(1);
  }
  // A CTA writes a slot and a position in 1.2 ns: 74,000 tokens took 88 us with one
  // CTA, 47 with two, 26 with four and 15.5 with eight
  const int ncta = a.n_max <= 4 * kTabThreads ? 1 : a.n_max <= 32 * kTabThreads ? 8 : 16;
  if (ncta == 1) return launch_pdl(build_tables_kernel, dim3(1), dim3(kTabThreads), smem, st, a);
  return launch_pdl_cluster(build_tables_kernel, dim3(ncta), dim3(kTabThreads), smem, ncta, st, a);
}

cudaError_t launch_write_kv(const WriteArgs& a, cudaStream_t st) {
  if (a.n == 0) return cudaSuccess;
  const int chunks = a.Hkv * (a.row_bytes / 16);
  const int side = kWriteThreads / (chunks < kWriteThreads ? chunks : kWriteThreads);
  const int per_cta = side * kWriteRows;
  return launch_pdl(write_kv_kernel, dim3((unsigned)((a.n + (long long)per_cta - 1) / per_cta)),
                    dim3(kWriteThreads), 0, st, a);
}

}  // namespace sva
