// kv4_attn.cu -- attention of a block's queries over the whole paged 4-bit
// cache and the block's own bf16 keys, for few query rows per KV head (one
// token, a short draft): bound by the cache's bytes, so the codes go from
// global memory through registers straight into matrix-instruction operands.
//
// A warp takes units of 16 keys.  With rows = the group's query rows,
//   S^T [16 keys x 8 rows] = K [16 x d] Q^T [d x 8]        (mma m16n8k16)
//   O^T [d x 8 rows]      += V^T [d x 16 keys] P^T [16 x 8] (mma m16n8k16)
// The keys are the M side of both products, so eight query rows fill an
// instruction (with the queries as M, half of every instruction would be
// padding).  The contraction index of an mma may be permuted as long as
// both operands agree, and so may the M rows of O^T, so each lane's share of
// a key row is a run of consecutive codes in memory:
//   K: lane (g = lane/4, t = lane%4) holds channels [t d/4, (t+1) d/4) of
//      keys g and g+8, as the A fragments of d/16 steps;
//   V: lane (g, t) holds channels [g d/8, (g+1) d/8) of keys 2t, 2t+1, 2t+8,
//      2t+9.  A V^T fragment pairs two keys in a register, so the nibbles of
//      two keys' words are interleaved (two AND-ORs per eight codes) and one
//      conversion yields the pair.
// code * scale is exact in fp16 (kv4.cuh).  Queries become fp16 scaled per
// row by a power of two that brings the row's largest value to [2^14, 2^15):
// exact for every value within 2^-32 of the largest (below, off by less than
// 2^-40 of the largest), the power undone in the fp32 scores.  P is fp16 (11
// bits against bf16's 8); scores, row sums and O are fp32.  P^T needs the
// scores transposed: one movmatrix per 8x8 tile.
//
// A row's exponent base is set 11 (log2) below its largest score so far and
// stays while no score exceeds it by 15: P lies in fp16's [0, 2^15], weights
// down to 2^-25 of the largest keep 11 bits, and most units need one vote and
// no exchange between lanes.
#include <float.h>

#include "kv4.cuh"

namespace herald {

constexpr int kKv4Warps = 8;
constexpr int kKv4Threads = kKv4Warps * 32;
constexpr int kKv4Unit = 16;        // keys per unit
constexpr int kKv4MinShare = kKv4Warps;  // units per CTA: at least one per warp
constexpr int kKv4MmaRows = 16;     // most rows per KV head of this kernel
constexpr float kKv4Below = 11.f, kKv4Above = 15.f;  // exponent base, log2 units


HERALD_DEV void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
HERALD_DEV void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
HERALD_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// fp16 pair {lo, hi}; bf16 pair: pack_bf16
HERALD_DEV uint32_t bcast16(uint32_t x, int half) {
  return half ? __byte_perm(x, 0, 0x3232) : __byte_perm(x, 0, 0x1010);
}

// One unit of cache keys as it comes from memory.
template <int D>
struct Kv4Raw {
  uint32_t k[2][D / 32];  // keys g, g+8: D/4 codes (D/32 words) each
  uint32_t v[4][D / 64];  // keys 2t, 2t+1, 2t+8, 2t+9: D/8 codes each
  uint32_t ks[2];         // their scales (D/64 bytes)
  uint32_t vs[4];
};

// Loads the unit at cache row `row` (kv4_row of its first key).  One address
// per array, the keys at constant offsets from it.
template <int D>
HERALD_DEV void kv4_load(Kv4Raw<D>& r, const Kv4Dev& c, size_t row, int lane) {
  constexpr int C = D / 2, S = D / 16;  // bytes of a row's codes and scales
  const int lg = lane >> 2, lt = lane & 3;
  const uint8_t* kc = c.kc + (row + lg) * C + lt * (C / 4);
  const uint8_t* ks = c.ks + (row + lg) * S + lt * (S / 4);
  const uint8_t* vc = c.vc + (row + 2 * lt) * C + lg * (C / 8);
  const uint8_t* vs = c.vs + (row + 2 * lt) * S + lg * S / 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (D == 128) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(kc + i * 8 * C));
      r.k[i][0] = w.x, r.k[i][1] = w.y, r.k[i][2] = w.z, r.k[i][3] = w.w;
      r.ks[i] = __ldg(reinterpret_cast<const uint16_t*>(ks + i * 8 * S));
    } else {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(kc + i * 8 * C));
      r.k[i][0] = w.x, r.k[i][1] = w.y;
      r.ks[i] = __ldg(ks + i * 8 * S);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int o = (i & 1) + 8 * (i >> 1);
    if constexpr (D == 128) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(vc + o * C));
      r.v[i][0] = w.x, r.v[i][1] = w.y;
    } else {
      r.v[i][0] = __ldg(reinterpret_cast<const uint32_t*>(vc + o * C));
    }
    r.vs[i] = __ldg(vs + o * S);
  }
}

// at most 8*NT query rows per KV head
template <int D, int NT>
__global__ void __launch_bounds__(kKv4Threads, NT == 1 ? 2 : 1)
    kv4_attn_kernel(const Kv4AttnArgs a) {
  constexpr int KS = D / 16;  // k steps of S, and M tiles of O^T
  constexpr int RT = 8 * NT;  // rows of a tile
  extern __shared__ float red[];  // [warps][RT][D + 4]
  __shared__ float red_m[kKv4Warps][RT], red_l[kKv4Warps][RT];
  griddep_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lg = lane >> 2, lt = lane & 3;
  const int G = a.Hq / a.Hkv, R = a.B * G;
  const int blk_units = a.bk ? (a.B + kKv4Unit - 1) / kKv4Unit : 0;
  const Kv4Split split =
      kv4_split(kv4_total_units(a.ctx, a.N, a.L_max, kKv4Unit, blk_units), a.Hkv, a.ctas,
                kKv4MinShare);
  int at = int(blockIdx.x) * split.share;
  const int end = min(at + split.share, split.total);
  if (at >= end) return;
  int n;
  int first;  // first unit of sequence n's first segment
  kv4_find(a.ctx, a.N, a.L_max, kKv4Unit, blk_units, a.Hkv, at, &n, &first);

  while (at < end) {
    const int ctx_raw = a.ctx[n];
    debug_flag(threadIdx.x == 0 && (ctx_raw < 0 || ctx_raw > a.L_max), DEV_BAD_COUNT);
    const int ctx = min(max(ctx_raw, 0), a.L_max);
    const int cache_units = (ctx + kKv4Unit - 1) / kKv4Unit, units = cache_units + blk_units;
    if (units == 0 || at >= first + a.Hkv * units) {  // the next sequence
      first += a.Hkv * units;
      ++n;
      continue;
    }
    const int g = (at - first) / units;
    const int seg0 = first + g * units;
    const int u0 = at - seg0, u1 = min(units, end - seg0);
    const int seg = n * a.Hkv + g;
    const int cu1 = min(u1, cache_units);
    auto page_of = [&](int u) {
      if (u >= cu1) return -1;
      const int p = kv4_page(a.c, n, (u * kKv4Unit) >> a.c.page_log2);
      debug_flag(p < 0, DEV_BAD_INDEX);  // positions below the length without a page
      return p;
    };

    // queries: B fragments (lane: row lg of each 8-row tile), fp16 scaled by
    // a power of two per row; rs[nt][2] undo it for the rows this lane's
    // scores belong to (2 lt, 2 lt + 1)
    uint32_t qf[NT][KS][2];
    float rs[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + lg;
      const bool on = r < R;
      const uint16_t* qp =
          a.q + ((size_t(n) * a.B + (on ? r / G : 0)) * a.Hq + g * G + (on ? r % G : 0)) * D +
          lt * (D / 4);
      float mx = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint2 w = make_uint2(0, 0);
        if (on) w = *reinterpret_cast<const uint2*>(qp + s * 4);
        qf[nt][s][0] = w.x;
        qf[nt][s][1] = w.y;
        mx = fmaxf(fmaxf(mx, fmaxf(fabsf(bf16lo(w.x)), fabsf(bf16hi(w.x)))),
                   fmaxf(fabsf(bf16lo(w.y)), fabsf(bf16hi(w.y))));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      float up, f;
      kv4_query_scale(mx, a.scale * a.c.k_scale, &up, &f);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qf[nt][s][i] = pack_half2(bf16lo(qf[nt][s][i]) * up, bf16hi(qf[nt][s][i]) * up);
      rs[nt][0] = __shfl_sync(0xffffffffu, f, 8 * lt);      // lane of row 2 lt
      rs[nt][1] = __shfl_sync(0xffffffffu, f, 8 * lt + 4);  // lane of row 2 lt + 1
    }

    float o[NT][KS][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) m[nt][i] = -FLT_MAX, l[nt][i] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][k][i] = 0.f;
    }
    // raw scores -> probabilities 2^(s f - m); moves the base where a score
    // stands more than kKv4Above over it
    auto probabilities = [&](float (&s)[NT][4], const float (&f)[NT][2]) {
      float x[NT][4];
      bool move = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[nt][i] = fmaf(s[nt][i], f[nt][i & 1], -m[nt][i & 1]);
        move |= fmaxf(fmaxf(x[nt][0], x[nt][1]), fmaxf(x[nt][2], x[nt][3])) > kKv4Above;
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float b = fmaxf(s[nt][i] * f[nt][i], s[nt][i + 2] * f[nt][i]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, d));
            b = fmaxf(m[nt][i], b - kKv4Below);
            const float w = fast_exp2(m[nt][i] - b);
            m[nt][i] = b;
            l[nt][i] *= w;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[nt][k][i] *= w;
              o[nt][k][i + 2] *= w;
            }
            x[nt][i] = fmaf(s[nt][i], f[nt][i], -b);
            x[nt][i + 2] = fmaf(s[nt][i + 2], f[nt][i], -b);
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[nt][i] = fast_exp2(x[nt][i]);
          l[nt][i & 1] += s[nt][i];
        }
    };

    // ------------------------------------------------------ cache units
    auto unit = [&](const Kv4Raw<D>& cur, int u, bool paged) {
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
      const uint32_t s0 = e4m3x2_to_half2(cur.ks[0]), s1 = e4m3x2_to_half2(cur.ks[1]);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {  // a word of codes per key: two k steps
        uint32_t h0[4], h1[4];
        e2m1x8_to_half2(cur.k[0][w], h0);
        e2m1x8_to_half2(cur.k[1][w], h1);
        const uint32_t f0 = bcast16(s0, w >> 1), f1 = bcast16(s1, w >> 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h0[i] = hmul2(h0[i], f0);
          h1[i] = hmul2(h1[i], f1);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(s[nt], h0[0], h1[0], h0[1], h1[1], qf[nt][2 * w][0], qf[nt][2 * w][1]);
          mma_f16(s[nt], h0[2], h1[2], h0[3], h1[3], qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
        }
      }
      uint32_t vs[4] = {cur.vs[0], cur.vs[1], cur.vs[2], cur.vs[3]};
      const int valid = paged ? ctx - u * kKv4Unit : 0;
      if (valid < kKv4Unit) {  // keys past the length, or without a page
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (lg + 8 * (i >> 1) >= valid) s[nt][i] = -INFINITY;
        // such a row may hold any bytes: 0 * NaN must not arise
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * lt + (i & 1) + 8 * (i >> 1) >= valid) vs[i] = 0;
      }
      probabilities(s, rs);
      uint32_t p0[NT], p1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        p0[nt] = transpose8x8(pack_half2(s[nt][0], s[nt][1]));
        p1[nt] = transpose8x8(pack_half2(s[nt][2], s[nt][3]));
      }
      const uint32_t f0 = e4m3x2_to_half2(vs[0] | vs[1] << 8),
                     f1 = e4m3x2_to_half2(vs[2] | vs[3] << 8);
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        uint32_t e0[4], d0[4], e1[4], d1[4];  // even, odd channels of the two key pairs
        e2m1x8_to_half2((cur.v[0][w] & 0x0F0F0F0Fu) | ((cur.v[1][w] << 4) & 0xF0F0F0F0u), e0);
        e2m1x8_to_half2(((cur.v[0][w] >> 4) & 0x0F0F0F0Fu) | (cur.v[1][w] & 0xF0F0F0F0u), d0);
        e2m1x8_to_half2((cur.v[2][w] & 0x0F0F0F0Fu) | ((cur.v[3][w] << 4) & 0xF0F0F0F0u), e1);
        e2m1x8_to_half2(((cur.v[2][w] >> 4) & 0x0F0F0F0Fu) | (cur.v[3][w] & 0xF0F0F0F0u), d1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e0[i] = hmul2(e0[i], f0);
          d0[i] = hmul2(d0[i], f0);
          e1[i] = hmul2(e1[i], f1);
          d1[i] = hmul2(d1[i], f1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(o[nt][w * 4 + i], e0[i], d0[i], e1[i], d1[i], p0[nt], p1[nt]);
        }
      }
    };
    // two units in flight: one is computed while the other one's bytes travel,
    // and the page of the one after is looked up a unit ahead of its load
    Kv4Raw<D> r0, r1;
    int u = u0 + warp;
    int pa = page_of(u), pb = page_of(u + kKv4Warps);
    auto load = [&](Kv4Raw<D>& r, int phys, int at_unit) {
      // (without a page: row 0, whose bytes the masks keep out)
      kv4_load<D>(r, a.c, phys < 0 ? 0 : kv4_row(a.c, phys, a.Hkv, g, at_unit * kKv4Unit), lane);
    };
    if (u < cu1) load(r0, pa, u);
    for (; u < cu1; u += 2 * kKv4Warps) {
      const int v = u + kKv4Warps;
      const bool ha = pa >= 0, hb = pb >= 0;
      pa = page_of(v + kKv4Warps);
      if (v < cu1) load(r1, pb, v);
      pb = page_of(v + 2 * kKv4Warps);
      unit(r0, u, ha);
      if (v >= cu1) {
        u = v;
        break;
      }
      if (v + kKv4Warps < cu1) load(r0, pa, v + kKv4Warps);
      unit(r1, v, hb);
    }

    // ------------------------------------- the block's own keys, in bf16
    // (P in units of v_scale so that O has one unit for all keys)
    for (; u < u1; u += kKv4Warps) {
      const int j0 = (u - cache_units) * kKv4Unit;
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
      const uint16_t* kp[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = j0 + lg + 8 * i;
        kp[i] = j < a.B ? a.bk + ((size_t(n) * a.B + j) * a.Hkv + g) * D + lt * (D / 4) : nullptr;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint2 w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[i] = kp[i] ? *reinterpret_cast<const uint2*>(kp[i] + k * 4) : make_uint2(0, 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = nt * 8 + lg;
          uint2 b = make_uint2(0, 0);
          if (r < R)
            b = *reinterpret_cast<const uint2*>(
                a.q + ((size_t(n) * a.B + r / G) * a.Hq + g * G + r % G) * D + lt * (D / 4) +
                k * 4);
          mma_bf16(s[nt], w[0].x, w[1].x, w[0].y, w[1].y, b.x, b.y);
        }
      }
      float f[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f[nt][0] = f[nt][1] = fminf(a.scale * 1.4426950408889634f, FLT_MAX);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + lg + 8 * (i >> 1) >= a.B) s[nt][i] = -INFINITY;
      }
      probabilities(s, f);
      const float iv = 1.f / a.c.v_scale;
      uint32_t p0[NT], p1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        p0[nt] = transpose8x8(pack_bf16(s[nt][0] * iv, s[nt][1] * iv));
        p1[nt] = transpose8x8(pack_bf16(s[nt][2] * iv, s[nt][3] * iv));
      }
      const uint16_t* vp[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + 2 * lt + (i & 1) + 8 * (i >> 1);
        vp[i] = j < a.B ? a.bv + ((size_t(n) * a.B + j) * a.Hkv + g) * D + lg * (D / 8) : nullptr;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {  // channels lg*D/8 + 2k, + 2k+1 of each key
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = vp[i] ? *reinterpret_cast<const uint32_t*>(vp[i] + 2 * k) : 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_bf16(o[nt][k], __byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                   __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632), p0[nt],
                   p1[nt]);
      }
    }

    // ------------------------------------------------- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
        if (lg == 0) {
          red_m[warp][nt * 8 + 2 * lt + i] = m[nt][i];
          red_l[warp][nt * 8 + 2 * lt + i] = l[nt][i];
        }
        float* dst = red + (size_t(warp) * RT + nt * 8 + 2 * lt + i) * (D + 4) + lg * (D / 8);
#pragma unroll
        for (int k = 0; k < KS; ++k)  // channels 2k, 2k+1 of this lane's run
          *reinterpret_cast<float2*>(dst + 2 * k) = make_float2(o[nt][k][i], o[nt][k][i + 2]);
      }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == units;  // no other piece of this segment
    const int slot = int(blockIdx.x) + seg;
    for (int i = threadIdx.x; i < RT * (D / 4); i += kKv4Threads) {
      // (neighbouring threads write neighbouring channels of out, rows of a partial)
      const int rr = whole ? i / (D / 4) : i % RT, c4 = whole ? i % (D / 4) : i / RT;
      const int r = rr;
      if (r >= R) continue;
      float M = -FLT_MAX;
#pragma unroll
      for (int w = 0; w < kKv4Warps; ++w) M = fmaxf(M, red_m[w][rr]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kKv4Warps; ++w) {
        const float mw = red_m[w][rr];
        const float f = fast_exp2(mw - M);
        const float4 x =
            *reinterpret_cast<const float4*>(red + (size_t(w) * RT + rr) * (D + 4) + c4 * 4);
        L += f * red_l[w][rr];
        acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
      }
      if (whole) {
        const float inv = L == 0.f ? 0.f : a.c.v_scale / L;
        *reinterpret_cast<uint2*>(a.out + ((size_t(n) * a.B + r / G) * a.Hq + g * G + r % G) * D +
                                  c4 * 4) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      } else {
        reinterpret_cast<float4*>(a.opart)[(size_t(slot) * (D / 4) + c4) * a.R16 + r] = acc;
        if (c4 == 0) a.ml[size_t(slot) * a.R16 + r] = make_float2(M, L);
      }
    }
    __syncthreads();  // the reduction buffers are free for the next piece
    at = seg0 + u1;
  }
}

// Joins the pieces of every segment that has more than one, and writes zeros
// for segments without keys.  grid (N*Hkv, ceil(R / 8)), 1024 threads: eight
// rows' chunks of four channels per D/4 * 8 threads, and kKv4JoinThreads over
// that many groups, each with every such-and-suchth partial, four in flight, so
// that the pieces of a long context travel at once; the groups are added in
// order.  subs: partials per piece (slots subs*p ...); with more than one,
// single pieces are joined here too.
constexpr int kKv4JoinThreads = 1024, kKv4JoinRows = 8;
template <int D>
__global__ void __launch_bounds__(kKv4JoinThreads)
    kv4_join_kernel(const Kv4AttnArgs a, int unit, int blk_units, int min_share, int subs) {
  constexpr int TPG = kKv4JoinRows * (D / 4), GR = kKv4JoinThreads / TPG;
  __shared__ float4 part[GR][TPG];
  __shared__ float part_m[GR][kKv4JoinRows], part_l[GR][kKv4JoinRows];
  griddep_enter();
  const int seg = blockIdx.x, n = seg / a.Hkv, g = seg - n * a.Hkv;
  const int G = a.Hq / a.Hkv, R = a.B * G;
  const int grp = threadIdx.x / TPG, item = threadIdx.x % TPG;
  const int rr = item % kKv4JoinRows, c4 = item / kKv4JoinRows;
  const int r = int(blockIdx.y) * kKv4JoinRows + rr, rc = min(r, R - 1);
  const Kv4Split split = kv4_split(kv4_total_units(a.ctx, a.N, a.L_max, unit, blk_units), a.Hkv,
                                   a.ctas, min_share);
  const int units = kv4_units(a.ctx[n], a.L_max, unit, blk_units);
  const int first =
      a.Hkv * kv4_total_units(a.ctx, n, a.L_max, unit, blk_units) + g * units;
  uint2* out = reinterpret_cast<uint2*>(
      a.out + ((size_t(n) * a.B + rc / G) * a.Hq + g * G + rc % G) * D + c4 * 4);
  if (units == 0) {
    if (grp == 0 && r < R) *out = make_uint2(0, 0);
    return;
  }
  int c0 = first / split.share, c1 = (first + units - 1) / split.share;
  if (c0 == c1 && subs == 1) return;  // one piece: written by the attention kernel
  c0 = (c0 + seg) * subs, c1 = (c1 + seg) * subs + subs - 1;  // its partials
  const float4* op = reinterpret_cast<const float4*>(a.opart) + size_t(c4) * a.R16 + rc;
  float M = -FLT_MAX, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kFly = 4;
  for (int c = c0 + grp; c <= c1; c += kFly * GR) {
    float2 p[kFly];
    float4 x[kFly];
#pragma unroll
    for (int i = 0; i < kFly; ++i) {
      const int ci = min(c + i * GR, c1);
      p[i] = a.ml[size_t(ci) * a.R16 + rc];
      x[i] = op[size_t(ci) * (D / 4) * a.R16];
      if (c + i * GR > c1) p[i] = make_float2(-FLT_MAX, 0.f), x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float M1 = M;
#pragma unroll
    for (int i = 0; i < kFly; ++i) M1 = fmaxf(M1, p[i].x);
    const float w = fast_exp2(M - M1);
    L *= w, acc.x *= w, acc.y *= w, acc.z *= w, acc.w *= w;
    M = M1;
#pragma unroll
    for (int i = 0; i < kFly; ++i) {
      const float f = fast_exp2(p[i].x - M);
      L += f * p[i].y;
      acc.x += f * x[i].x, acc.y += f * x[i].y, acc.z += f * x[i].z, acc.w += f * x[i].w;
    }
  }
  part[grp][item] = acc;
  if (c4 == 0) part_m[grp][rr] = M, part_l[grp][rr] = L;
  __syncthreads();
  if (grp != 0 || r >= R) return;
#pragma unroll
  for (int i = 0; i < GR; ++i) M = fmaxf(M, part_m[i][rr]);
  L = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < GR; ++i) {
    const float f = fast_exp2(part_m[i][rr] - M);
    const float4 x = part[i][item];
    L += f * part_l[i][rr];
    acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
  }
  const float inv = L == 0.f ? 0.f : a.c.v_scale / L;
  *out = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

// ------------------------------------------------------------------- host

template <int D, int NT>
static cudaError_t launch_rows(const Kv4AttnArgs& a, cudaStream_t st) {
  constexpr size_t smem = size_t(kKv4Warps) * 8 * NT * (D + 4) * 4;
  HERALD_CHECK_LAUNCH(ensure_smem(kv4_attn_kernel<D, NT>, smem));
  return launch_k("kv4_attn_kernel", kv4_attn_kernel<D, NT>,
                  dim3(unsigned(a.ctas)), dim3(kKv4Threads), smem, st, a);
}

// Workspace: error word, then (m, l) and O of every partial.
struct Kv4Ws {
  size_t ml, opart, total;
  int R16;
};
static Kv4Ws kv4_ws(const herald_dims& dm) {
  Kv4Ws w;
  w.R16 = cdiv(dm.B * (dm.Hq / dm.Hkv), 16) * 16;
  const size_t slots = 2 * (size_t(kKv4MaxCtas) + size_t(dm.N) * dm.Hkv);
  w.ml = 256;
  w.opart = align_up(w.ml + slots * w.R16 * 8, 256);
  w.total = w.opart + slots * w.R16 * size_t(dm.d) * 4;
  return w;
}
size_t kv4_attn_workspace(const herald_dims& dm) { return kv4_ws(dm).total; }

cudaError_t launch_kv4_attn(const herald_dims& dm, const uint16_t* q, const Kv4Dev& c,
                            const int32_t* ctx, const uint16_t* bk, const uint16_t* bv,
                            uint16_t* out, float scale, void* ws, int num_sms, cudaStream_t st) {
  const int G = dm.Hq / dm.Hkv, R = dm.B * G;
  const Kv4Ws w = kv4_ws(dm);
  char* p = static_cast<char*>(ws);
  Kv4AttnArgs a{};
  a.q = q, a.bk = bk, a.bv = bv, a.ctx = ctx, a.out = out;
  a.ml = reinterpret_cast<float2*>(p + w.ml);
  a.opart = reinterpret_cast<float*>(p + w.opart);
  a.scale = scale;
  a.N = dm.N, a.Hq = dm.Hq, a.Hkv = dm.Hkv, a.B = dm.B, a.L_max = dm.L_max, a.R16 = w.R16;
  a.c = c;
  const bool tc = R > kKv4MmaRows;
  const int nt = R <= 8 ? 1 : 2;
  a.ctas = std::min(kKv4MaxCtas, tc ? num_sms : (nt == 1 ? 2 : 1) * num_sms);
  if (tc)
    HERALD_CHECK_LAUNCH(launch_kv4_attn_tc(dm.d, R, a, reinterpret_cast<uint32_t*>(p), st));
  else if (dm.d == 128)
    HERALD_CHECK_LAUNCH((nt == 1 ? launch_rows<128, 1>(a, st) : launch_rows<128, 2>(a, st)));
  else
    HERALD_CHECK_LAUNCH((nt == 1 ? launch_rows<64, 1>(a, st) : launch_rows<64, 2>(a, st)));
  const int unit = tc ? kKv4TcKeys : kKv4Unit;
  const int blk_units = bk ? cdiv(dm.B, unit) : 0, min_share = tc ? 1 : kKv4MinShare;
  const int subs = tc && R <= kTileM ? 2 : 1;
  const dim3 grid(unsigned(dm.N * dm.Hkv), unsigned(cdiv(R, kKv4JoinRows)));
  if (dm.d == 128)
    HERALD_CHECK_LAUNCH(launch_k("kv4_join_kernel", kv4_join_kernel<128>, grid,
                                 dim3(kKv4JoinThreads), 0, st, a, unit, blk_units, min_share, subs));
  else
    HERALD_CHECK_LAUNCH(launch_k("kv4_join_kernel", kv4_join_kernel<64>, grid,
                                 dim3(kKv4JoinThreads), 0, st, a, unit, blk_units, min_share, subs));
  return cudaGetLastError();
}

HERALD_DEBUG_WORD_READER(debug_take_kv4_attn)

}  // namespace herald
