// Device code that the 4-bit cache kernels share: the two 4- and 8-bit formats,
// and the attention's work split.
#pragma once

#include <cuda_fp16.h>

#include "kv4.h"
#include "ptx.h"

namespace sva {
namespace kv4 {

// ---------------------------------------------------------------- formats
// E2M1 codes of the four bytes of a word (low bits first) as pairs of halves, exact. The
// word is taken apart by a move, which leaves one instruction a byte: with shifts and
// masks it was three, all for the same half-rate pipe.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t* r) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// E4M3 scales of the four bytes of a word as two pairs of halves, exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& r01, uint32_t& r23) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(r01), "=r"(r23)
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
// r[0 .. 8) times half H of s (the multiplication picks the half itself).
template <int H>
__device__ __forceinline__ void scale_f16x2(uint32_t* r, uint32_t s) {
  const __half2 ss = *reinterpret_cast<const __half2*>(&s), f = H ? __high2half2(ss) : __low2half2(ss);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&r[e]), f);
    r[e] = *reinterpret_cast<const uint32_t*>(&x);
  }
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) { return f16x2_to_f32(e4m3x2_to_f16x2(byte & 0xffu)).x; }
// lo and hi, rounded to E2M1 (ties to even, 6 at most), in one byte.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}
// x >= 0 rounded to E4M3 (ties to even, 448 at most; NaN to NaN).
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}

constexpr int kMaxExp = 32;  // a head's exponent lies in [-32, 32]
__device__ __forceinline__ int head_exp(const int32_t* e, int h) {
  return e ? min(max(e[h], -kMaxExp), kMaxExp) : 0;
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((127 + e) << 23); }

// ---------------------------------------------------------------- work split
// One division for all of a kernel: an int division is some thirty instructions, and
// what runs once costs the fetch of its code (about 12 cycles an instruction).
static __device__ __noinline__ int quotient(int x, int y) { return x / y; }

// (Pages and groups of query heads are powers of two nearly always.)
__device__ __forceinline__ int blocks_in(const Attend4Args& a, int ctx) {
  return a.ppb_shift >= 0 ? ctx >> (a.ppb_shift + 4) : quotient(ctx, a.blk);
}
__device__ __forceinline__ int pieces_of(const Attend4Args& a, int ctx) {
  const int full = blocks_in(a, ctx), rest = ctx - full * a.blk;
  return (a.sel ? a.n_sel : full) * a.ppb + (rest + kPiece - 1) / kPiece;
}

// The line that the CTAs share: the pairs' key tiles, and ahead of each pair's as many units
// as beginning it takes (a.pair_cost; pairs without keys have none). In shared memory:
struct Line {
  int first[kMaxB4 + 1];  // units of one pair, summed over the sequences before
  int ctx[kMaxB4];
  int ctas, each, more;   // CTAs with a share; its units, and how many CTAs have one unit more

  __device__ __forceinline__ int begin(int cta) const { return cta < ctas ? cta * each + min(cta, more) : ctas * each + more; }
  // the CTA that has unit x
  __device__ __forceinline__ int cta_of(int x) const {
    const int big = more * (each + 1);
    return x < big ? quotient(x, each + 1) : more + quotient(x - big, each);
  }
};

// Fill it (one warp). Returns whether a length was clamped, in any lane that saw one.
__device__ __forceinline__ bool make_line(const Attend4Args& a, Line* line) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  bool bad = false;
  if (lane == 0) line->first[0] = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    int x = 0;
    if (b < a.B) {
      const int c = a.seq_ctx[b], n = min(max(c, 0), a.nb_max * a.blk);
      bad |= c != n;
      line->ctx[b] = n;
      x = (pieces_of(a, n) + a.ppt - 1) >> a.ppt_shift;
      if (x) x += a.pair_cost;
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (b < a.B) line->first[b + 1] = carry + x;
    carry += __shfl_sync(0xffffffffu, x, 31);
  }
  const int total = carry * a.Hkv * a.row_tiles;  // (below 2^31: the call's limits)
  const int ctas = min(a.ctas, total), each = ctas ? quotient(total, ctas) : 0;
  if (lane == 0) {
    line->ctas = ctas;
    line->each = each;
    line->more = total - each * ctas;
  }
  return bad;
}

struct Segment {
  int b, h, rt;      // the pair
  int tile0, tiles;  // its key tiles (none if the share ends ahead of them)
  int ctx, full, pieces;  // tokens, full blocks, pieces of the (sequence, head)
  int slot;
  int next;          // where the next segment begins
};
// The segment that begins at position x of the line (x < end, the end of the CTA's share).
__device__ __forceinline__ Segment segment_at(const Attend4Args& a, const Line& line, int x, int end, int cta) {
  Segment s;
  const int per = a.Hkv * a.row_tiles;
  int lo = 0, hi = a.B;  // the last sequence that begins at x or before (those without keys do not count)
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (line.first[m] * per <= x) lo = m;
    else hi = m;
  }
  s.b = lo;
  const int n = line.first[lo + 1] - line.first[lo], in = x - line.first[lo] * per, pair = quotient(in, n);
  const int unit = in - pair * n;
  s.tile0 = max(unit - a.pair_cost, 0);
  s.h = a.row_tiles == 1 ? pair : quotient(pair, a.row_tiles);
  s.rt = pair - s.h * a.row_tiles;
  s.next = min(x - unit + n, end);
  s.tiles = max(s.next - (x - unit) - a.pair_cost - s.tile0, 0);
  s.ctx = line.ctx[lo];
  s.full = blocks_in(a, s.ctx);
  s.pieces = (a.sel ? a.n_sel : s.full) * a.ppb + (s.ctx - s.full * a.blk + kPiece - 1) / kPiece;
  s.slot = lo * per + pair + cta;
  return s;
}
// Key tiles of the line that lie before position x (by one warp).
__device__ __forceinline__ int tiles_before(const Attend4Args& a, const Line& line, int x) {
  const int per = a.Hkv * a.row_tiles;
  int tiles = 0;
#pragma unroll 1
  for (int b = threadIdx.x & 31; b < a.B; b += 32) {
    const int n = line.first[b + 1] - line.first[b], in = x - line.first[b] * per;
    if (in <= 0) break;
    if (n == 0) continue;
    if (in >= n * per) {
      tiles += (n - a.pair_cost) * per;
      continue;
    }
    const int pair = quotient(in, n);
    tiles += pair * (n - a.pair_cost) + max(in - pair * n - a.pair_cost, 0);
  }
  return __reduce_add_sync(0xffffffffu, tiles);
}
// What the join needs of pair p (of all sequences): its first slot and the number of slots.
__device__ __forceinline__ int2 slots_of(const Attend4Args& a, const Line& line, int p) {
  const int per = a.Hkv * a.row_tiles, b = quotient(p, per), n = line.first[b + 1] - line.first[b];
  if (n == 0) return make_int2(0, 0);
  const int x = line.first[b] * per + (p - b * per) * n;
  const int c0 = line.cta_of(x + a.pair_cost), c1 = line.cta_of(x + n - 1);
  return make_int2(p + c0, c1 - c0 + 1);
}

// Where piece i of a segment's (sequence, head) lies in the pools (in pieces, -1:
// nowhere), and how many of its tokens count.
__device__ __forceinline__ long long piece_at(const Attend4Args& a, const Segment& s, int i, int* valid,
                                              unsigned* flags) {
  *valid = 0;
  if (i >= s.pieces) return -1;
  const int slots = a.sel ? a.n_sel : s.full, at = a.ppb_shift >= 0 ? i >> a.ppb_shift : quotient(i, a.ppb);
  int block = at, sub = i - at * a.ppb;
  if (at >= slots) {  // the partial last block
    block = s.full;
    sub = i - slots * a.ppb;
    *valid = min(kPiece, s.ctx - s.full * a.blk - sub * kPiece);
  } else {
    if (a.sel) {
      block = a.sel[((long long)s.b * a.Hkv + s.h) * a.sel_stride + at];
      if (block < 0 || block >= s.full) {
        if (block != -1) *flags |= SV_FLAG_BAD_BLOCK_INDEX;
        return -1;
      }
    }
    *valid = kPiece;
  }
  const int page = a.block_table[(long long)s.b * a.nb_max + block];
  if (page < 0 || page >= a.num_pages) {
    *flags |= SV_FLAG_BAD_PAGE;
    *valid = 0;
    return -1;
  }
  return ((long long)page * a.Hkv + s.h) * a.ppb + sub;
}

// Row r of a (sequence, head): draft t, query head h * G + g, r = t * G + g.
__device__ __forceinline__ long long row_at(const Attend4Args& a, int b, int h, int r) {
  const int t = a.g_shift >= 0 ? r >> a.g_shift : quotient(r, a.G);
  return ((long long)b * a.T + t) * a.Hq + h * a.G + (r - t * a.G);
}

}  // namespace kv4
}  // namespace sva
