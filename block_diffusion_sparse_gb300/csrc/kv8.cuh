// kv8.cuh -- the paged 8-bit KV cache on the device: its addresses, its number
// format, and the arguments of its attention kernels.
//
// A row of d channels (one position of one KV head) is d bytes of e4m3 codes; the
// rows of `block` consecutive positions of a head share one scale, a power of two
// whose biased exponent is a byte:  value = code * 2^(byte - 127).
// A code has 4 significant bits and the scale none, so a value is exact in bf16.
#pragma once
#include <float.h>

#include "kv4.cuh"

namespace herald {

constexpr int kKv8MinExp = -32, kKv8MaxExp = 32;  // exponents of the scales

// The page of logical page lp of sequence n, or -1 where the table has no page in
// range (such positions are never read or written).
HERALD_DEV int kv8_page(const Kv8Dev& c, int n, int lp) {
  const int p = c.table[size_t(n) * c.max_pages + lp];
  return p >= 0 && p < c.n_pages ? p : -1;
}
// Row index of position pos in page `phys` (64 bits: a long cache has more bytes
// than 32 bits count), and the index of its scale.
HERALD_DEV size_t kv8_row(const Kv8Dev& c, int phys, int Hkv, int g, int pos) {
  return size_t(uint32_t(phys)) * uint32_t(Hkv << c.page_log2) +
         uint32_t((g << c.page_log2) + (pos & ((1 << c.page_log2) - 1)));
}
HERALD_DEV size_t kv8_scale(const Kv8Dev& c, int phys, int Hkv, int g, int pos) {
  const int log2 = c.page_log2 - c.block_log2;  // (pages hold whole blocks)
  return size_t(uint32_t(phys)) * uint32_t(Hkv << log2) +
         uint32_t((g << log2) + ((pos & ((1 << c.page_log2) - 1)) >> c.block_log2));
}
// Exponent of a scale byte; bytes that no call writes count as the nearer end.
HERALD_DEV int kv8_exp(uint32_t byte) {
  return min(max(int(byte) - 127, kKv8MinExp), kKv8MaxExp);
}
HERALD_DEV float exp2_int(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }  // -126..127

// The four e4m3 codes of a word -> two fp16 pairs (exact).
HERALD_DEV void e4m3x4_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// fp32 pair -> e4m3 codes (lo in bits 0-7), to nearest even, past 448 to 448, NaN stays.
HERALD_DEV uint32_t float2_to_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// A query row as e4m3 numbers: values are multiplied by *up, the power of two that
// brings the row's largest magnitude mx to [2^7, 2^8), and *f turns a product with a
// key's codes into a log2-unit score (`scale` has log2(e) in it).  (mx below 2^-112
// counts as that; with an infinity *up is a NaN, as inf - inf makes the row.)
// *f times a key's scale, 2^-32 to 2^32, must not be 0 or infinite: a masked -inf times 0
// and a zero score times inf would be NaN.  Below 2^-94 *f counts as that (scores are then
// under 2^-38: 2^8 * 448 * 128 channels); the other end is the product's, not *f's
// (kv8_score_factor): with *f held to 2^90 for it, the cache's scores past that shrank
// beside those of the block's own keys.  2^127 is a row's largest value times the scale of 2^133.
HERALD_DEV void kv8_query_scale(float mx, float scale, float* up, float* f) {
  const int e = min(max(int(__float_as_uint(mx) >> 23) - 127, -112), 127);
  *up = mx < INFINITY ? exp2_int(7 - e) : __uint_as_float(0x7FC00000u);
  *f = fminf(fmaxf(scale * exp2_int(e - 7), 0x1p-94f), 0x1p127f);
}
// *f times a key's scale sk, finite.  (Past 2^127 any product of codes but the smallest
// scores past fp32.)
HERALD_DEV float kv8_score_factor(float f, float sk) { return fminf(f * sk, 0x1p127f); }
// One lane of a converged warp, the same every time: what it alone issues keeps its
// operands in uniform registers (with `lane == 0` each mma moved them there anew).
HERALD_DEV bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// fp16 pair -> e4m3 codes, as float2_to_e4m3 (a query goes through fp16, whose step below
// 2^-14 is far under e4m3's)
HERALD_DEV uint32_t half2_to_e4m3(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
HERALD_DEV uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest magnitudes so far and of a word of two bf16, as bits (a NaN does not count).
HERALD_DEV uint32_t max_bf16x2_abs(uint32_t m, uint32_t w) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w & 0x7FFF7FFFu));
  return d;
}

// Eight words at once, a whole sector, to an address of 32 bytes' alignment.
HERALD_DEV void store8(void* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// ---- attention arguments shared by its kernels
struct Kv8AttnArgs {
  const uint16_t *q, *bk, *bv;
  const int32_t* ctx;
  uint16_t* out;
  float* opart;  // [slots][R16][D]
  float2* ml;    // [slots][R16]
  float scale;   // softmax scale times log2(e): scores are in log2 units
  int N, Hq, Hkv, B, L_max, R16, ctas;
  int row_tiles; // of 128 rows (1 with few rows): a KV head has that many segments
  int pad;       // what a piece costs beside its tiles, in tiles (kv4_units)
  Kv8Dev c;
};
// The kernel for `rows` <= kKv8FewRows query rows per KV head (kv8_rows.cu).  It and the one
// for more rows, in us over 64 sequences of up to 8K tokens / one of 128K / one of 32K (8 KV
// heads, d = 128): 16 rows 103 / 48.8 / 16.3 here and 129 / 57.7 / 22.3 there, a form of it for 32
// rows 269 / 102 / 53 and the other kernel 134 / 58.5 / 22.3.  Its softmax keeps a row of a key in
// two registers and more: with 16 rows all 168 that 384 threads can have are in use and 72 bytes
// are spilled (64 with d = 64), with 8 rows 121 to 123 and none.
constexpr int kKv8FewRows = 16;
cudaError_t launch_kv8_rows(int d, int rows, const Kv8AttnArgs& a, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, uint32_t* err, cudaStream_t st);
// The kernel for more (kv8_attn_tc.cu).
cudaError_t launch_kv8_attn_tc(int d, const Kv8AttnArgs& a, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, uint32_t* err, cudaStream_t st);

// A CTA's share of the tiles of 128 keys, as kv4_share's (kv4.cuh) with the segments of
// heads * row tiles per sequence and no units for block keys: units [at, end); with at <
// end, n is the sequence that holds unit `at`, first the first unit of its first
// segment and ctx its length (a load that every role would wait for again).
struct Kv8Share {
  int at, end, n, first, ctx;
};
HERALD_DEV Kv8Share kv8_share(const Kv8AttnArgs& a, int cta) {
  const int lane = threadIdx.x & 31, heads = a.Hkv * a.row_tiles;
  auto length = [&](int n) { return n < a.N ? min(max(a.ctx[n], 0), a.L_max) : 0; };
  const int ctx0 = length(lane);  // (the lengths of the first 32 sequences are loaded once)
  int sum = kv4_units(ctx0, a.L_max, 0, a.pad);
  for (int n = lane + 32; n < a.N; n += 32) sum += kv4_units(length(n), a.L_max, 0, a.pad);
  const Kv4Split split = kv4_split(int(__reduce_add_sync(0xffffffffu, sum)), heads, a.ctas);
  Kv8Share r;
  r.at = warp_same(cta * split.share);
  r.end = warp_same(min(r.at + split.share, split.total));
  r.n = r.first = r.ctx = 0;
  if (r.at >= r.end) return r;
  int base = 0;
  for (int n0 = 0; n0 < a.N; n0 += 32) {
    const int ctx = n0 == 0 ? ctx0 : length(n0 + lane);
    const int own = heads * kv4_units(ctx, a.L_max, 0, a.pad);
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
      r.ctx = __shfl_sync(0xffffffffu, ctx, l);
      return r;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return r;
}

// The pieces of a CTA's share, in order: body(n, gt, seg, ctx, u0, u1) with gt = g *
// row_tiles + row tile, seg = n * Hkv * row_tiles + gt, tiles u0 <= u < u1 of 128 cache
// positions; it returns false to leave.
template <typename Body>
HERALD_DEV void kv8_pieces(const Kv8AttnArgs& a, const Kv8Share& sh, Body&& body) {
  const int heads = a.Hkv * a.row_tiles;
  int at = sh.at, first = sh.first, n = sh.n, ctx = sh.ctx;
  int next = a.ctx[min(n + 1, a.N - 1)];  // (of the sequence after, before it is asked for)
  while (at < sh.end) {
    const int units = kv4_units(ctx, a.L_max, 0, a.pad);
    if (units == 0 || at >= first + heads * units) {  // the next sequence
      first += heads * units;
      ++n;
      ctx = warp_same(min(max(next, 0), a.L_max));
      next = a.ctx[min(n + 1, a.N - 1)];
      continue;
    }
    const int gt = (at - first) / units;
    const int seg0 = first + gt * units;
    const int u0 = max(at - seg0 - a.pad, 0), u1 = min(units, sh.end - seg0) - a.pad;
    if (u1 > 0 && !body(n, gt, n * heads + gt, ctx, u0, u1)) return;
    at = seg0 + a.pad + u1;
  }
}

}  // namespace herald
