// kv4.cuh -- the paged 4-bit KV cache on the device: its addresses, its
// number formats, and how the attention kernels share out its keys.
//
// A row of d channels (one position of one KV head) is held as d/2 bytes of
// e2m1 codes, two per byte with the even channel in the low half, and d/16
// e4m3 scales, one per 16 consecutive channels:
//   value = code * scale * (k_scale | v_scale).
// A code has 2 and a scale 4 significant bits, so code * scale has at most 6
// and lies in [2^-10, 2688]: it is exact in fp16.
#pragma once
#include <float.h>

#include "internal.cuh"
#include "ptx.cuh"

namespace herald {

// The page of logical page lp of sequence n, or -1 where the table has no
// page in range (such positions are never read or written).
HERALD_DEV int kv4_page(const Kv4Dev& c, int n, int lp) {
  const int p = c.table[size_t(n) * c.max_pages + lp];
  return p >= 0 && p < c.n_pages ? p : -1;
}
// Row index of position pos in page `phys` (64 bits: a long cache has more
// bytes than 32 bits count).
HERALD_DEV size_t kv4_row(const Kv4Dev& c, int phys, int Hkv, int g, int pos) {
  return ((size_t(phys) * Hkv + g) << c.page_log2) + (pos & ((1 << c.page_log2) - 1));
}

// The four bytes of a word of codes -> four fp16 pairs, a byte's low half first.
HERALD_DEV void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "mov.b32 {t0, t1, t2, t3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, t1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, t2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, t3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two scales (bits 0-15) -> fp16 pair (exact: 4 significant bits).
HERALD_DEV uint32_t e4m3x2_to_half2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(b)));
  return r;
}
HERALD_DEV float e4m3_to_float(uint32_t b) {
  const uint32_t h = e4m3x2_to_half2(b & 0xFFu);
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}
HERALD_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A query row as fp16: values are multiplied by *up, the power of two that
// brings the row's largest magnitude mx to [2^14, 2^15), and *f turns a product
// with the codes * scales of a key into a log2-unit score; the softmax scale times
// k_scale times log2(e) is sc 2^sc_e with sc in [1, 2) (its own exponent: either
// factor may be near the ends of fp32 where the scores are not).  (mx below 2^-112
// counts as that, infinities as 2^127; *f stays positive and finite: a masked score
// of -inf times 0, or a zero score times inf, would be NaN.)
HERALD_DEV void kv4_query_scale(float mx, float sc, int sc_e, float* up, float* f) {
  const int e = min(max(int(__float_as_uint(mx) >> 23) - 127, -112), 127);
  *up = __uint_as_float(uint32_t(14 - e + 127) << 23);
  *f = sc * __uint_as_float(uint32_t(min(max(sc_e + e - 14, -126), 127) + 127) << 23);
}

// Weights of the block's own keys.  Their values are bf16 and an mma's operands have
// one type, so P is bf16 too, as the sum of two numbers (the second what the first
// left: 16 bits in all, beside fp16's 11 over the cache), each multiplied with V: with
// one, 8 bits, a short context's output was off by up to 2^-8 of its weighted |values|
// before its own rounding.
HERALD_DEV uint32_t take_bf16(float& a, float& b) {  // a, b: left with the remainders
  const uint32_t w = pack_bf16(a, b);
  a -= bf16lo(w), b -= bf16hi(w);
  return w;
}

// Scores s f whose fp32 steps are no longer small beside the distance of a base m
// from its row's largest score (log2 units).  2^(s f - m) takes the product exactly
// (one fma), but m stands on the fp32 grid: rounded to nearest it may lie steps above
// every score (all weights 0) or far enough below for P to pass fp16's range.
// Past this size the base is rounded down and 2^(s f - m) ends at P's largest value:
// keys within a step or so of the largest score, which fp32 holds to no more than
// that, weigh alike.  (Without it scores past 2^26 gave NaN.)
constexpr float kKv4Far = 0x1p20f;

// ---- attention arguments shared by its kernels
struct Kv4AttnArgs {
  const uint16_t *q, *bk, *bv;
  const int32_t* ctx;
  uint16_t* out;
  float* opart;  // [slots][D/4][R16][4]
  float2* ml;    // [slots][R16]
  float scale;   // of the block's keys' scores
  float sc;      // of the cache's keys' (kv4_query_scale)
  int sc_e;
  int N, Hq, Hkv, B, L_max, R16, ctas;
  int pad;       // what a piece costs beside its tiles, in tiles (kv4_units)
  Kv4Dev c;
};
constexpr int kKv4Tile = 128;  // keys per tile of the attention kernels
// The tensor-core kernel (kv4_attn_tc.cu) for `rows` <= 256 query rows per KV
// head.
cudaError_t launch_kv4_attn_tc(int d, int rows, const Kv4AttnArgs& a, uint32_t* err,
                               cudaStream_t st);

// Shared memory by 32-bit address (the aligned base of the dynamic part is a
// generic pointer to the compiler).
HERALD_DEV uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
HERALD_DEV uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
HERALD_DEV uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
HERALD_DEV uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
HERALD_DEV uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
HERALD_DEV void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Bounded wait; false when it ran out: the roles then stop copying and issuing and
// the kernel returns.  (A role that has seen a wait run out waits no more; the others'
// run out beside it.)  Counted, not timed, and small: the roles of a kernel share the
// issue slots and the instruction cache.  With a timer around the tries and a look at
// the others' failures in each, 4 x 64K blocks took 127 us instead of 120.
struct Kv4Wait {
  uint32_t* failed;  // shared: the waits that ran out
  uint32_t limit = kKv4Tries;
  // The answer for a whole warp, which leaves converged: lanes may see a
  // barrier complete in different polls, and the tensor-memory instructions
  // that follow (.sync.aligned) want the warp in one piece.
  HERALD_DEV bool operator()(uint64_t* bar, uint32_t parity, uint32_t which) const {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
      uint32_t tries = 0;
#pragma unroll 1
      do ok = mbar_try_wait_for(bar, parity, 4000u);
      while (!ok && ++tries < limit);
    }
    if (__all_sync(0xffffffffu, ok)) return true;
    atomicOr(failed, which);
    return false;
  }
};

// ---- how attention CTAs share the keys
// The keys of every (sequence, KV head) segment, in tiles of 128 cache positions,
// are laid end to end, segments in order, and the block's own keys with them:
// blk_units tiles of their own per segment, or (blk_units = kKv4BlkJoined) as
// part of the segment's first tile, which then exists without cache keys too.
// Every segment with keys also has `pad` units in front of its tiles that stand
// for the cost of starting on it (queries, the first copies, the piece's end).
// CTA c takes units [c*share, (c+1)*share).  Equal shares keep ragged batches
// balanced; a CTA's range may cover the end of one segment, whole segments, and
// the start of another (its pieces).  Piece (c, segment s) has partial slot c +
// s: from one piece to the next c or s grows.  All counts fit 31 bits
// (N*Hkv*L_max < 2^31).  The results are handed to every lane from one, which
// tells the compiler that what follows from them is the same for the whole warp.
constexpr int kKv4BlkJoined = -1;
struct Kv4Split {
  int total;  // units of all segments
  int share;  // units per CTA
};
HERALD_DEV int warp_same(int x) { return __shfl_sync(0xffffffffu, x, 0); }
HERALD_DEV int kv4_units(int ctx, int L_max, int blk_units, int pad) {
  int t = (min(max(ctx, 0), L_max) + kKv4Tile - 1) / kKv4Tile;
  t = blk_units == kKv4BlkJoined ? max(t, 1) : t + blk_units;
  return t > 0 ? t + pad : 0;
}
// Sum over the first N sequences of their units (per KV head); called by a
// whole warp.
HERALD_DEV int kv4_total_units(const int32_t* ctx, int N, int L_max, int blk_units, int pad) {
  int sum = 0;
  for (int n = int(threadIdx.x & 31); n < N; n += 32)
    sum += kv4_units(ctx[n], L_max, blk_units, pad);
  return warp_same(__reduce_add_sync(0xffffffffu, sum));
}
HERALD_DEV Kv4Split kv4_split(int per_head, int Hkv, int ctas) {
  Kv4Split s;
  s.total = per_head * Hkv;
  s.share = max((s.total + ctas - 1) / ctas, 1);
  return s;
}
// A CTA's share: units [at, end); with at < end, n is the sequence that holds
// unit `at` and first the first unit of that sequence's first segment.  Called
// by a whole warp.
struct Kv4Share {
  int at, end, n, first;
};
HERALD_DEV Kv4Share kv4_share(const Kv4AttnArgs& a, int blk_units, int cta) {
  const int32_t* ctx = a.ctx;
  const int N = a.N, L_max = a.L_max, Hkv = a.Hkv, pad = a.pad;
  const int lane = threadIdx.x & 31;
  // (the lengths of the first 32 sequences are loaded once)
  const int own0 = lane < N ? kv4_units(ctx[lane], L_max, blk_units, pad) : 0;
  int sum = own0;
  for (int n = lane + 32; n < N; n += 32) sum += kv4_units(ctx[n], L_max, blk_units, pad);
  const Kv4Split split = kv4_split(int(__reduce_add_sync(0xffffffffu, sum)), Hkv, a.ctas);
  Kv4Share r;
  r.at = warp_same(cta * split.share);
  r.end = warp_same(min(r.at + split.share, split.total));
  r.n = r.first = 0;
  if (r.at >= r.end) return r;
  int base = 0;
  for (int n0 = 0; n0 < N; n0 += 32) {
    const int n = n0 + lane;
    const int own = Hkv * (n0 == 0 ? own0 : n < N ? kv4_units(ctx[n], L_max, blk_units, pad) : 0);
    int inc = own;  // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + inc > r.at);
    if (hit) {
      const int l = __ffs(hit) - 1;
      r.n = warp_same(n0 + l);
      r.first = base + __shfl_sync(0xffffffffu, inc - own, l);
      return r;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return r;
}

}  // namespace herald
