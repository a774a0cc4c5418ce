// kv8_move.cu -- rows in and out of the paged 8-bit KV cache:
//   append  rotates a block's (or a prompt's) queries and keys by their
//           positions, quantises keys and values by blocks of positions and
//           writes them into the sequences' pages
//   pool    the means of the key blocks an append touched (the block-granular
//           stage 1's input), from the rows as the cache holds them
//   gather  held rows at given positions as bf16 (sparse pool, candidates)
#include "kv8.cuh"

namespace herald {

// All three are bound by memory where there is much to do and by one launch and a chain of
// dependent loads where there is not.  Measured (per call in a graph, 32 + 2 x 8 heads of 128
// channels): append of ragged prompts, 4 x <= 4096 tokens, interleaved, 35.7 us for 222 MB (93%
// of the copy rate); of 64 tokens 3.7; of 32 tokens with block means 7.6, two launches; gather
// of 4096 rows of 32 heads 6.9 us from L2 (11.2 from DRAM) for 51 MB (with 8 channels a lane,
// and so twice the indexes, pages, scales and addresses, 8.9), of a pool of 4 x 1344 rows 2.0.
constexpr int kKv8MoveThreads = 256;
// Query heads of an item: they share a lane's angles, and their loads are in flight
// together.  Prompts of 4 x 4096 tokens, 32 + 2 x 8 heads, with 2 / 4 / 8: 74 / 63 / 61 us;
// below 512 tokens the three (and 1) are alike, 5 to 7 us.
constexpr int kQueryHeads = 8;

// The smallest exponent e with top <= 448 2^e (448 = 1.75 2^8), of a bf16 magnitude's
// bits, within the scales' range.
HERALD_DEV int kv8_need(uint32_t top) {
  const int e = int(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
  return min(max(e, kKv8MinExp), kKv8MaxExp);
}

// Eight rotated or plain channels: x (bf16 pairs) and the pairs' partners in the
// half-split form (px), each product and sum rounded to fp32 as the definition has
// them, then to bf16.  cs, sn: the lane's angles; first: this lane has the pairs'
// first channels.
template <bool Interleaved>
HERALD_DEV uint4 turn8(const uint4& x, const uint4& px, const float* cs, const float* sn,
                       bool first) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w}, pw[4] = {px.x, px.y, px.z, px.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = bf16lo(w[j]), b = bf16hi(w[j]);
    if constexpr (Interleaved) {
      o[j] = pack_bf16(__fsub_rn(__fmul_rn(a, cs[j]), __fmul_rn(b, sn[j])),
                       __fadd_rn(__fmul_rn(b, cs[j]), __fmul_rn(a, sn[j])));
    } else {
      const float p0 = __fmul_rn(bf16lo(pw[j]), sn[2 * j]),
                  p1 = __fmul_rn(bf16hi(pw[j]), sn[2 * j + 1]);
      const float y0 = __fmul_rn(a, cs[2 * j]), y1 = __fmul_rn(b, cs[2 * j + 1]);
      o[j] = first ? pack_bf16(__fsub_rn(y0, p0), __fsub_rn(y1, p1))
                   : pack_bf16(__fadd_rn(y0, p0), __fadd_rn(y1, p1));
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

struct Kv8AppendArgs {
  const uint16_t *q, *k, *v;
  int64_t q_ld, k_ld, v_ld;
  const int32_t *n_tok, *ctx;
  const float* cos_sin;  // [n_pos][rot/2][2]
  int rot;
  uint16_t *q_rot, *k_rot;
  int Hq, Hkv, T, L_max;
  int kv_ctas;               // CTAs of keys and values; those of queries follow
  int units;                 // of a sequence: touched blocks x kinds x KV heads
  int kinds;                 // 2: keys and values, 1: keys only
  int block_log2;            // of the units (the cache's, 16 without one)
  int q_chunks, tok_log2;    // queries: chunks of kQueryHeads heads, tokens of a CTA
  Kv8Dev c;                  // (kc null: rotate only)
};

// Where a lane stands in its row of D channels: D/8 neighbouring lanes hold a row,
// eight channels (16 bytes) each.  In the half-split form channel i < rot/2 pairs with
// i + rot/2: the same channels of the lane rot/16 lanes on; else 2i with 2i+1.
struct Kv8Lane {
  int c, partner;
  bool turns, first;
  HERALD_DEV Kv8Lane(int lane, int lpr, int rot) {
    c = lane % lpr;
    const int half = rot / 16;
    turns = c * 8 < rot;
    first = c < half;
    partner = (lane - c) + (!turns ? c : first ? c + half : c - half);
  }
};
template <bool Interleaved>
HERALD_DEV void load_angles(const Kv8AppendArgs& a, const Kv8Lane& l, int pos, float* cs,
                            float* sn) {
  constexpr int A = Interleaved ? 4 : 8;  // angles of a lane
  const float* p = a.cos_sin + size_t(pos) * a.rot +
                   (Interleaved || l.first ? l.c : l.c - a.rot / 16) * (2 * A);
#pragma unroll
  for (int i = 0; i < A; i += 2) {
    const float4 w = *reinterpret_cast<const float4*>(p + 2 * i);
    cs[i] = w.x, sn[i] = w.y, cs[i + 1] = w.z, sn[i + 1] = w.w;
  }
}
HERALD_DEV uint4 shfl4(const uint4& x, int src) {
  return make_uint4(__shfl_sync(0xffffffffu, x.x, src), __shfl_sync(0xffffffffu, x.y, src),
                    __shfl_sync(0xffffffffu, x.z, src), __shfl_sync(0xffffffffu, x.w, src));
}

// grid (CTAs of keys and values, then of queries; sequences).
// A unit is one touched block of one KV head's keys or values; 16 of its rows are one
// warp's (all loads first), so block/16 warps share a unit and its maximum.  Where
// the first block holds older rows and its scale grows, the same warps hold those
// anew.  A CTA has the units of neighbouring heads: rows of a token lie side by side.
// (Registers: the half-split form has twice the angles; with four CTAs an SM, 64 registers a
// lane, it takes 14.0 us for 1024 tokens instead of 12.5 with three, 80 (79 used); the other
// with three 64 us for the prompts of 4 x 4096 instead of 61 with four.)
template <int D, bool Interleaved>
__global__ void __launch_bounds__(kKv8MoveThreads, Interleaved ? 4 : 3)
    kv8_append_kernel(const Kv8AppendArgs a) {
  constexpr int Per = kQueryHeads;
  constexpr int LPR = D / 8, RPP = 32 / LPR, P = 16 / RPP;  // rows per pass of a warp, passes
  __shared__ uint32_t tops[kKv8MoveThreads / 32];
  griddep_enter();
  const int n = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ctx_raw = a.ctx[n];
  debug_flag(threadIdx.x == 0 && (ctx_raw < 0 || ctx_raw > a.L_max), DEV_BAD_COUNT);
  const int L0 = min(max(ctx_raw, 0), a.L_max);
  int toks = a.T;
  if (a.n_tok) {
    const int raw = a.n_tok[n];
    debug_flag(threadIdx.x == 0 && (raw < 0 || raw > a.T), DEV_BAD_COUNT);
    toks = min(max(raw, 0), a.T);
  }
  toks = min(toks, a.L_max - L0);  // tokens at or past L_max are ignored
  const Kv8Lane l(lane, LPR, a.rot);

  if (int(blockIdx.x) >= a.kv_ctas) {  // ------------------------------- queries
    constexpr int Rows = kKv8MoveThreads / LPR;
    const int slot = threadIdx.x / LPR, q_per_cta = Rows >> a.tok_log2;
    const int ctas = (a.q_chunks + q_per_cta - 1) / q_per_cta;
    const int i = int(blockIdx.x) - a.kv_ctas, tt = i / ctas;
    const int t = (tt << a.tok_log2) + (slot & ((1 << a.tok_log2) - 1));
    const int chunk = (i - tt * ctas) * q_per_cta + (slot >> a.tok_log2);
    const bool live = t < toks && chunk < a.q_chunks;
    if (!__any_sync(0xffffffffu, live)) return;
    const int64_t tok = int64_t(n) * a.T + t;
    const int h0 = chunk * Per;
    const uint16_t* src = a.q + tok * a.q_ld + h0 * D + l.c * 8;
    uint4 u[Per];
#pragma unroll
    for (int j = 0; j < Per; ++j)
      u[j] = live && h0 + j < a.Hq ? *reinterpret_cast<const uint4*>(src + j * D)
                                   : make_uint4(0, 0, 0, 0);
    float cs[Interleaved ? 4 : 8], sn[Interleaved ? 4 : 8];
    if (live && l.turns) load_angles<Interleaved>(a, l, L0 + t, cs, sn);
    uint16_t* dst = a.q_rot + (tok * a.Hq + h0) * D + l.c * 8;
#pragma unroll
    for (int j = 0; j < Per; ++j) {
      const uint4 px = Interleaved ? u[j] : shfl4(u[j], l.partner);
      if (l.turns) u[j] = turn8<Interleaved>(u[j], px, cs, sn, l.first);
      if (live && h0 + j < a.Hq) *reinterpret_cast<uint4*>(dst + j * D) = u[j];
    }
    return;
  }

  // ------------------------------------------------------- keys and values
  const int w_log2 = a.block_log2 - 4;                       // warps of a unit
  const int unit = (int(blockIdx.x) << (3 - w_log2)) + (warp >> w_log2);
  const int sub = warp & ((1 << w_log2) - 1);
  const int g = unit % a.Hkv, bk = unit / a.Hkv;
  const bool is_v = a.kinds == 2 && (bk & 1);
  const int pos0 = ((L0 >> a.block_log2) + bk / a.kinds) << a.block_log2;  // the block's first
  const bool on = unit < a.units && toks > 0 && pos0 < L0 + toks;
  // (with one warp a unit there is no barrier ahead, and an idle warp may leave)
  if (w_log2 == 0 && !on) return;
  const int row0 = pos0 + sub * 16 + lane / LPR;  // this lane's rows: row0 + pass * RPP
  const uint16_t* src = (is_v ? a.v : a.k) + g * D + l.c * 8;
  const int64_t ld = is_v ? a.v_ld : a.k_ld, tok0 = int64_t(n) * a.T - L0;
  uint4 u[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int pos = row0 + p * RPP;
    u[p] = on && pos >= L0 && pos < L0 + toks
               ? *reinterpret_cast<const uint4*>(src + (tok0 + pos) * ld)
               : make_uint4(0, 0, 0, 0);
  }
  int phys = -1, old = kKv8MinExp;
  size_t scale_at = 0;
  if (on && a.c.kc) {
    phys = kv8_page(a.c, n, pos0 >> a.c.page_log2);
    debug_flag(phys < 0, DEV_BAD_INDEX);  // tokens without a page
    if (phys >= 0) {
      scale_at = kv8_scale(a.c, phys, a.Hkv, g, pos0);
      if (pos0 < L0) old = kv8_exp((is_v ? a.c.vs : a.c.ks)[scale_at]);
    }
  }
  if (!is_v && a.rot) {
    // (the angles of a row ahead would spill: 37.2 us for the prompts instead of 35.8)
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int pos = row0 + p * RPP;
      const bool live = on && pos >= L0 && pos < L0 + toks;
      float cs[Interleaved ? 4 : 8], sn[Interleaved ? 4 : 8];
      if (live && l.turns) load_angles<Interleaved>(a, l, pos, cs, sn);
      const uint4 px = Interleaved ? u[p] : shfl4(u[p], l.partner);
      if (live && l.turns) u[p] = turn8<Interleaved>(u[p], px, cs, sn, l.first);
    }
  }
  if (!is_v && a.k_rot) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int pos = row0 + p * RPP;
      if (on && pos >= L0 && pos < L0 + toks)
        *reinterpret_cast<uint4*>(a.k_rot + ((tok0 + pos) * a.Hkv + g) * D + l.c * 8) = u[p];
    }
  }
  if (!a.c.kc) return;
  // the unit's largest finite magnitude
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < P; ++p)
    m = max_bf16x2_abs(max_bf16x2_abs(max_bf16x2_abs(max_bf16x2_abs(m, u[p].x), u[p].y), u[p].z),
                       u[p].w);
  uint32_t top = max(m & 0xFFFFu, m >> 16);
  if (top >= 0x7F80u) {  // infinities do not count
    top = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t w[4] = {u[p].x, u[p].y, u[p].z, u[p].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = w[j] & 0x7FFFu, y = w[j] >> 16 & 0x7FFFu;
        top = max(top, max(x < 0x7F80u ? x : 0u, y < 0x7F80u ? y : 0u));
      }
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (w_log2 > 0) {  // (also: every warp of the unit has read the old scale)
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    const int w0 = warp & ~((1 << w_log2) - 1);
    for (int i = 0; i < 1 << w_log2; ++i) top = max(top, tops[w0 + i]);
  }
  if (!on || phys < 0) return;
  const int e = max(kv8_need(top), old);
  uint8_t* codes = (is_v ? a.c.vc : a.c.kc) + kv8_row(a.c, phys, a.Hkv, g, pos0) * D + l.c * 8;
  const float inv = exp2_int(-e);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int pos = row0 + p * RPP;
    if (pos < L0 || pos >= L0 + toks) continue;
    const uint32_t w[4] = {u[p].x, u[p].y, u[p].z, u[p].w};
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = float2_to_e4m3(bf16lo(w[j]) * inv, bf16hi(w[j]) * inv);
    *reinterpret_cast<uint2*>(codes + size_t(pos - pos0) * D) =
        make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  }
  if (pos0 < L0 && e > old) {  // older rows under the larger scale
    const float down = exp2_int(old - e);
    uint2 w[P];
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (row0 + p * RPP < L0)
        w[p] = *reinterpret_cast<const uint2*>(codes + size_t(row0 + p * RPP - pos0) * D);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int pos = row0 + p * RPP;
      if (pos >= L0) continue;
      uint32_t h[4], o[4];
      e4m3x4_to_half2(w[p].x, h[0], h[1]);
      e4m3x4_to_half2(w[p].y, h[2], h[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        o[j] = float2_to_e4m3(f.x * down, f.y * down);
      }
      *reinterpret_cast<uint2*>(codes + size_t(pos - pos0) * D) =
          make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
    }
  }
  if (sub == 0 && lane == 0) (is_v ? a.c.vs : a.c.ks)[scale_at] = uint8_t(e + 127);
}

// Eight held channels (two words of codes) times 2^e, as fp32.
HERALD_DEV void held8(const uint2& w, float s, float (&x)[8]) {
  uint32_t h[4];
  e4m3x4_to_half2(w.x, h[0], h[1]);
  e4m3x4_to_half2(w.y, h[2], h[3]);
  const uint64_t s2 = f2_pack(s, s);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    f2_unpack(f2_mul(f2_pack(f.x, f.y), s2), x[2 * j], x[2 * j + 1]);
  }
}

// grid (blocks, N*Hkv): the means of the blocks that tokens [ctx, ctx + tokens) fall
// into, over the rows below ctx + tokens.  D/8 lanes per row, the block's rows dealt
// over the rest of the CTA; the threads' sums are added in a fixed tree.  A row
// without a page counts as zeros.
template <int D>
__global__ void __launch_bounds__(kKv8MoveThreads)
    kv8_pool_kernel(const Kv8Dev c, const int32_t* __restrict__ ctx,
                    const int32_t* __restrict__ n_tok, int T, int Hkv, int L_max, int Bk,
                    int nb_max, float* __restrict__ pooled) {
  constexpr int LPR = D / 8, RPC = kKv8MoveThreads / LPR;
  __shared__ float sums[RPC][D + 4];
  griddep_enter();
  const int seg = blockIdx.y, n = seg / Hkv, g = seg - n * Hkv;
  const int L0 = min(max(ctx[n], 0), L_max);
  const int end = min(L0 + (n_tok ? min(max(n_tok[n], 0), T) : T), L_max);
  const int b = L0 / Bk + int(blockIdx.x);
  if (end == L0 || b * int64_t(Bk) >= end) return;
  const int r0 = b * Bk, r1 = min(end, r0 + min(Bk, L_max - r0));
  const int ch = threadIdx.x % LPR, rr = threadIdx.x / LPR;
  float acc[8] = {};
  constexpr int F = 4;  // rows in flight
  for (int r = r0 + rr; r < r1; r += F * RPC) {
    int phys[F];
    uint2 w[F];
    uint32_t s[F];
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const int rj = r + j * RPC;
      phys[j] = rj < r1 ? kv8_page(c, n, rj >> c.page_log2) : -1;
      debug_flag(rj < r1 && phys[j] < 0, DEV_BAD_INDEX);
    }
#pragma unroll
    for (int j = 0; j < F; ++j)
      if (phys[j] >= 0) {
        const int rj = r + j * RPC;
        w[j] = *reinterpret_cast<const uint2*>(c.kc + kv8_row(c, phys[j], Hkv, g, rj) * D + ch * 8);
        s[j] = c.ks[kv8_scale(c, phys[j], Hkv, g, rj)];
      }
#pragma unroll
    for (int j = 0; j < F; ++j)
      if (phys[j] >= 0) {
        float x[8];
        held8(w[j], exp2_int(kv8_exp(s[j])), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += x[i];
      }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[rr][ch * 8 + i] = acc[i];
  for (int half = RPC / 2; half > 0; half >>= 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < half * D; i += kKv8MoveThreads)
      sums[i / D][i % D] += sums[i / D + half][i % D];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kKv8MoveThreads)
    pooled[(size_t(seg) * nb_max + b) * D + e] = sums[0][e] / float(r1 - r0);
}

// grid (row groups, N*Hkv): D/16 lanes per row, 16 channels each (16 bytes in, 32 out),
// Rows rows a thread.
template <int D, int Rows>
__global__ void __launch_bounds__(kKv8MoveThreads)
    kv8_gather_kernel(const Kv8Dev c, const int32_t* __restrict__ idx,
                      const int32_t* __restrict__ n_sel, int P_max, int Hkv, int L_max,
                      uint16_t* __restrict__ pk, uint16_t* __restrict__ pv) {
  constexpr int LPR = D / 16, RPC = kKv8MoveThreads / LPR;
  griddep_enter();
  const int seg = blockIdx.y, n = seg / Hkv, g = seg - n * Hkv;
  const int ch = threadIdx.x % LPR, r0 = blockIdx.x * (RPC * Rows) + threadIdx.x / LPR;
  const int ns = n_sel[seg];
  debug_flag(ns < 0 || ns > P_max, DEV_BAD_COUNT);
  int pos[Rows], phys[Rows];
#pragma unroll
  for (int i = 0; i < Rows; ++i) {
    const int r = r0 + i * RPC;
    pos[i] = r < P_max ? idx[size_t(seg) * P_max + r] : -1;
    if (r >= ns) pos[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < Rows; ++i) {
    phys[i] = pos[i] >= 0 && pos[i] < L_max ? kv8_page(c, n, pos[i] >> c.page_log2) : -1;
    debug_flag(r0 + i * RPC < min(ns, P_max) && phys[i] < 0, DEV_BAD_INDEX);  // outside the cache
  }
  uint4 w[2][Rows];
  uint32_t s[2][Rows];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < Rows; ++i) {
      w[kv][i] = make_uint4(0, 0, 0, 0), s[kv][i] = 0;
      if (phys[i] >= 0 && (kv == 0 || pv)) {
        w[kv][i] = *reinterpret_cast<const uint4*>(
            (kv ? c.vc : c.kc) + kv8_row(c, phys[i], Hkv, g, pos[i]) * D + ch * 16);
        s[kv][i] = (kv ? c.vs : c.ks)[kv8_scale(c, phys[i], Hkv, g, pos[i])];
      }
    }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint16_t* out = kv ? pv : pk;
    if (!out) continue;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;  // (arrays are aligned to 16)
#pragma unroll
    for (int i = 0; i < Rows; ++i) {
      const int r = r0 + i * RPC;
      const float f = exp2_int(kv8_exp(s[kv][i]));
      float x[2][8];
      held8(make_uint2(w[kv][i].x, w[kv][i].y), f, x[0]);
      held8(make_uint2(w[kv][i].z, w[kv][i].w), f, x[1]);
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = pack_bf16(x[j / 4][2 * (j % 4)], x[j / 4][2 * (j % 4) + 1]);
      if (r >= P_max) continue;
      uint16_t* dst = out + (size_t(seg) * P_max + r) * D + ch * 16;
      if (wide) {
        store8(dst, o);
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + 8) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

// ------------------------------------------------------------------- host

cudaError_t launch_kv8_append(const herald_dims& dm, int T, const int32_t* n_tok,
                              const uint16_t* q, int64_t q_ld, const uint16_t* k, int64_t k_ld,
                              const uint16_t* v, int64_t v_ld, const herald_rope* rope,
                              int32_t* ctx, const Kv8Dev* cache, uint16_t* q_rot, uint16_t* k_rot,
                              float* pooled, int Bk, bool advance, cudaStream_t st) {
  Kv8AppendArgs a{};
  a.q = q, a.k = k, a.v = v;
  a.q_ld = q_ld, a.k_ld = k_ld, a.v_ld = v_ld;
  a.n_tok = n_tok, a.ctx = ctx;
  if (rope) a.cos_sin = rope->cos_sin, a.rot = rope->rot;
  a.q_rot = q_rot, a.k_rot = k_rot;
  a.Hq = dm.Hq, a.Hkv = dm.Hkv, a.T = T, a.L_max = dm.L_max;
  a.block_log2 = 4;
  if (cache) a.c = *cache, a.block_log2 = cache->block_log2;
  a.kinds = cache ? 2 : 1;
  int64_t kv_ctas = 0;
  if (k) {
    // T tokens fall into at most this many blocks, wherever they begin
    const int64_t blocks = ((int64_t(T) - 1 + (1 << a.block_log2) - 1) >> a.block_log2) + 1;
    const int64_t units = blocks * a.kinds * dm.Hkv;
    if (units >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    a.units = int(units);
    const int upc = 8 >> (a.block_log2 - 4);  // units per CTA
    kv_ctas = (units + upc - 1) / upc;
  }
  a.kv_ctas = int(kv_ctas);
  int64_t q_ctas = 0;
  const int rpc = kKv8MoveThreads / (dm.d / 8);  // query rows of a CTA and load
  if (q) {
    a.q_chunks = cdiv(dm.Hq, kQueryHeads);
    while ((1 << a.tok_log2) < T && (2 << a.tok_log2) <= rpc) ++a.tok_log2;
    q_ctas = int64_t(cdiv(T, 1 << a.tok_log2)) * cdiv(a.q_chunks, rpc >> a.tok_log2);
  }
  if (kv_ctas + q_ctas >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  const dim3 grid(unsigned(kv_ctas + q_ctas), unsigned(dm.N));
  const bool il = rope && rope->interleaved;
  auto* kernel = dm.d == 128 ? (il ? kv8_append_kernel<128, true> : kv8_append_kernel<128, false>)
                             : (il ? kv8_append_kernel<64, true> : kv8_append_kernel<64, false>);
  HERALD_CHECK_LAUNCH(
      launch_k("kv8_append_kernel", kernel, grid, dim3(kKv8MoveThreads), 0, st, a));
  if (pooled) {
    const dim3 pg(unsigned(cdiv(T - 1, Bk) + 1), unsigned(dm.N * dm.Hkv));
    HERALD_CHECK_LAUNCH(launch_k("kv8_pool_kernel",
                                 dm.d == 128 ? kv8_pool_kernel<128> : kv8_pool_kernel<64>, pg,
                                 dim3(kKv8MoveThreads), 0, st, *cache, ctx, n_tok, T, dm.Hkv,
                                 dm.L_max, Bk, cdiv(dm.L_max, Bk), pooled));
  }
  if (advance) HERALD_CHECK_LAUNCH(launch_kv_advance(dm, T, n_tok, ctx, st));
  return cudaGetLastError();
}

cudaError_t launch_kv8_gather(const herald_dims& dm, const int32_t* idx, const int32_t* n_sel,
                              int P_max, const Kv8Dev& c, uint16_t* pk, uint16_t* pv, int num_sms,
                              cudaStream_t st) {
  const int rpc = kKv8MoveThreads / (dm.d / 16), segs = dm.N * dm.Hkv;
  // Two rows a thread, both rows' loads out before one is converted, where only keys are read
  // and the launch is more than one wave; keys and values are two loads already.  With one and
  // two, in us: 4096 candidate keys of 8, 16 and 32 heads (1024 to 4096 CTAs of one row a thread)
  // 3.4 / 4.7 / 7.7 and 3.3 / 4.4 / 6.9; pools of 1344 keys and values of 4, 32 and 64 heads 2.4 /
  // 5.0 / 8.1 and 2.5 / 5.1 / 8.3.
  const bool many = !pv && int64_t(segs) * cdiv(P_max, rpc) > int64_t(num_sms) * 8;
  const dim3 grid(unsigned(cdiv(P_max, many ? 2 * rpc : rpc)), unsigned(segs));
  auto* kernel = dm.d == 128 ? (many ? kv8_gather_kernel<128, 2> : kv8_gather_kernel<128, 1>)
                             : (many ? kv8_gather_kernel<64, 2> : kv8_gather_kernel<64, 1>);
  return launch_k("kv8_gather_kernel", kernel, grid, dim3(kKv8MoveThreads), 0, st, c, idx, n_sel,
                  P_max, dm.Hkv, dm.L_max, pk, pv);
}

HERALD_DEBUG_WORD_READER(debug_take_kv8_move)

}  // namespace herald
