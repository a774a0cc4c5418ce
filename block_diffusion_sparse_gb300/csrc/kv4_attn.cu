// kv4_attn.cu -- attention of a block's queries over the whole paged 4-bit
// cache and the block's own bf16 keys, for few query rows per KV head (one
// token, a short draft): bound by the cache's bytes and by the instructions that
// turn codes into numbers.  One token over 128K (8 KV heads, 151 MB) takes 37 us, of
// which it streams for 29 at 5.2 TB/s; its copies alone, without a product, 31.  Per
// 16 keys a warp issues some 345 instructions, 64 of them conversions and 64 products
// with scales, each at half rate; at 96 registers (two CTAs an SM) d = 128 spills 10
// bytes.  64 ragged tokens of up to 8K (327 MB): 75 us.
//
// A CTA walks its share of the keys (kv4_split) in tiles of 128.  Its last warp
// copies each tile's codes and scales from the pages into a ring of stages (bulk
// copies, the tile's pages in parallel lanes); each of the first eight takes 16
// of the tile's keys, and the ninth the block's own keys, beside them (with one
// of the eight doing that first, a ragged batch of single tokens took 114 us
// instead of 97: the ring waited for it).  With rows = the group's query rows,
//   S^T [16 keys x 8 rows] = K [16 x d] Q^T [d x 8]        (mma m16n8k16)
//   O^T [d x 8 rows]      += V^T [d x 16 keys] P^T [16 x 8] (mma m16n8k16)
// The keys are the M side of both products, so eight query rows fill an
// instruction (with the queries as M, half of every instruction would be
// padding).  The contraction index of an mma may be permuted as long as
// both operands agree, and so may the M rows, so each lane's share of a key row
// is a run of consecutive codes and dequantised registers are operands at once:
//   K: lane (g = lane/4, t = lane%4) holds channels [t d/4, (t+1) d/4) of two
//      keys, as the A fragments of d/16 steps;
//   V: lane (g, t) holds channels [g d/8, (g+1) d/8) of four keys.  A V^T
//      fragment pairs two keys in a register, so the nibbles of two keys'
//      words are interleaved (a shift and a bit select per four codes) and one
//      conversion yields the pair.
// The mma's key index j = 8h + 2t + o stands for key 8h + 4o + (t ^ o) of the 16:
// then neither the K nor the V reads meet more than two-way bank conflicts.
// code * scale is exact in fp16 (kv4.cuh).  Queries become fp16 scaled per
// row by a power of two that brings the row's largest value to [2^14, 2^15):
// exact for every value within 2^-31 of the largest (below, off by at most
// 2^-39 of the largest), the power undone in the fp32 scores.  P is fp16 (11
// bits against bf16's 8; over the block's keys two bf16 numbers, take_bf16);
// scores, row sums and O are fp32.  P^T needs the
// scores transposed: one movmatrix per 8x8 tile.
//
// A row's exponent base is set 11 (log2) below its largest score so far and
// stays while no score exceeds it by 15: P lies in fp16's [0, 2^15], weights
// down to 2^-25 of the largest keep 11 bits, and most tiles need one vote and
// no exchange between lanes.
#include <float.h>
#include <math.h>

#include "kv4.cuh"

namespace herald {

constexpr int kKv4Warps = 8;        // warps of cache keys
constexpr int kKv4Parts = kKv4Warps + 1;  // and one of the block's keys
constexpr int kKv4Threads = (kKv4Parts + 1) * 32;
constexpr int kKv4Unit = 16;        // keys per warp and tile
// Most rows per KV head of this kernel.  16 rows here and on the tensor cores'
// 128-row products: 18.3 and 24.5 us at 1 x 32K, 53 and 68 us at 16 x 8K (8 KV heads).
// (24 here spill: 32 and 99 us where the tensor cores take 25 and 68.)
constexpr int kKv4MmaRows = 16;
// What a piece costs beside its tiles, in tiles (kv4_units).  64 ragged tokens with 0 /
// 2 / 3 / 4 / 5: 88.7 / 78.7 / 74.7 / 75.7 / 76.4 us.  Tensor-core kernel with 0 / 3 / 5 /
// 7 / 9 / 12: drafts of 5 25.6 / 23.2 / 22.0 / 22.1 / 22.9 / 22.9, 32 tokens at 32K 35.1 /
// 29.2 / 28.2 / 28.0 / 27.7 / 28.9, 12 ragged blocks of 32 tokens 115 / 84 / 71.6 / 70.3 /
// 70.7 / 71.5.
constexpr int kKv4PadRows = 3, kKv4PadTc = 7;
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

HERALD_DEV void product_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(kKv4Parts * 32) : "memory");
}

// Waits of the kernel (bits 16-31 of the error word).
enum : uint32_t { W_STAGE_FREE = 1, W_STAGE_FULL = 2 };

// Dynamic shared memory: the ring of stages (codes and scales of 128 keys and
// values), then the warps' partial outputs.
template <int D, int NT>
struct RowsSmem {
  static constexpr int kStages = NT == 1 ? 3 : 5;
  static constexpr int kCodes = kKv4Tile * D / 2, kScales = kKv4Tile * D / 16;
  static constexpr int kStage = 2 * (kCodes + kScales);
  static constexpr int kRed = kStages * kStage;
  static constexpr int kTotal = kRed + kKv4Parts * 8 * NT * (D + 4) * 4;
};

// at most 8*NT query rows per KV head
template <int D, int NT>
__global__ void __launch_bounds__(kKv4Threads, NT == 1 ? 2 : 1)
    kv4_attn_kernel(const Kv4AttnArgs a, uint32_t* err) {
  using S = RowsSmem<D, NT>;
  constexpr int KS = D / 16;  // k steps of S, and M tiles of O^T
  constexpr int RT = 8 * NT;  // rows of a tile
  constexpr int kRowC = D / 2, kRowS = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[S::kStages], empty[S::kStages];
  __shared__ uint32_t failed;
  __shared__ uint8_t counts[S::kStages][kKv4Warps];  // keys of each 16 that count
  __shared__ float red_m[kKv4Parts][RT], red_l[kKv4Parts][RT];
  float* red = reinterpret_cast<float*>(smem + S::kRed);  // [parts][RT][D + 4]
  const int warp = warp_same(int(threadIdx.x) >> 5), lane = threadIdx.x & 31;
  const int lg = lane >> 2, lt = lane & 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], kKv4Warps);
    failed = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_enter();
  const Kv4Wait wait{&failed};
  const int G = a.Hq / a.Hkv, R = a.B * G;
  const int blk_units = a.bk ? kKv4BlkJoined : 0;
  const Kv4Share sh = kv4_share(a, blk_units, int(blockIdx.x));
  const int end = sh.end;
  if (sh.at >= end) return;

  // Both roles walk the same pieces: body(n, g, seg, ctx, units, u0, u1), cache
  // tiles u0 <= u < min(u1, tiles of ctx), the block's keys with tile 0.
  auto pieces = [&](auto&& body) {
    int at = sh.at, first = sh.first, n = sh.n;
    while (at < end) {
      const int ctx = warp_same(min(max(a.ctx[n], 0), a.L_max));
      const int units = kv4_units(ctx, a.L_max, blk_units, a.pad);
      if (units == 0 || at >= first + a.Hkv * units) {  // the next sequence
        first += a.Hkv * units;
        ++n;
        continue;
      }
      const int g = (at - first) / units;
      const int seg0 = first + g * units;
      const int u0 = max(at - seg0 - a.pad, 0), u1 = min(units, end - seg0) - a.pad;
      if (u1 > 0) body(n, g, n * a.Hkv + g, ctx, units - a.pad, u0, u1);
      at = seg0 + a.pad + u1;
    }
  };

  if (warp == kKv4Parts) {
    // ------------------------------------------------------------ copies
    const int sub = min(1 << a.c.page_log2, kKv4Tile);  // keys of a tile in one page
    const int k0 = lane * sub;                          // lane i: sub-chunk i of the tile
    uint32_t t = 0;
    bool ok = true;
    pieces([&](int n, int g, int, int ctx, int, int u0, int u1) {
      debug_flag(lane == 0 && a.ctx[n] != ctx, DEV_BAD_COUNT);
      const int32_t* table = a.c.table + size_t(n) * a.c.max_pages;
      int pos = u0 * kKv4Tile + k0;
      const int stop = k0 < kKv4Tile ? min(ctx, u1 * kKv4Tile) : 0;
      // the table's entry is read a tile ahead
      int next = pos < stop ? table[pos >> a.c.page_log2] : -1;
      const int tiles = min(u1, (ctx + kKv4Tile - 1) / kKv4Tile);
      for (int u = u0; u < tiles && ok; ++u, ++t, pos += kKv4Tile) {
        const int phys = next;
        if (pos + kKv4Tile < stop) next = table[(pos + kKv4Tile) >> a.c.page_log2];
        const bool on = pos < stop, have = on && phys >= 0 && phys < a.c.n_pages;
        debug_flag(on && !have, DEV_BAD_INDEX);  // positions below the length without a page
        const int keys = have ? min(sub, ctx - pos) : 0;
        const uint32_t rows = uint32_t(keys + 15) & ~15u;  // whole groups of 16: inside the page
        const uint32_t total = __reduce_add_sync(0xffffffffu, rows);
        const int mine = __shfl_sync(0xffffffffu, keys, lane * 16 / sub) - lane * 16 % sub;
        const uint32_t st = t % S::kStages;
        ok = t < uint32_t(S::kStages) || wait(&empty[st], (t / S::kStages - 1) & 1, W_STAGE_FREE);
        if (!ok) break;
        if (lane < kKv4Warps)
          *(volatile uint8_t*)&counts[st][lane] = uint8_t(min(max(mine, 0), kKv4Unit));
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[st], total * uint32_t(2 * (kRowC + kRowS)));
        __syncwarp();
        if (rows) {
          const size_t row = kv4_row(a.c, phys, a.Hkv, g, pos);
          uint8_t* d = smem + st * S::kStage;
          bulk_load(d + k0 * kRowC, a.c.kc + row * kRowC, rows * kRowC, &full[st]);
          bulk_load(d + S::kCodes + k0 * kRowC, a.c.vc + row * kRowC, rows * kRowC, &full[st]);
          bulk_load(d + 2 * S::kCodes + k0 * kRowS, a.c.ks + row * kRowS, rows * kRowS, &full[st]);
          bulk_load(d + 2 * S::kCodes + S::kScales + k0 * kRowS, a.c.vs + row * kRowS,
                    rows * kRowS, &full[st]);
        }
      }
    });
    // every copy has landed before the CTA may leave (where a wait has run out, nobody
    // else waits for it)
    for (uint32_t i = t > uint32_t(S::kStages) ? t - S::kStages : 0; i < t; ++i)
      mbar_wait(&full[i % S::kStages], (i / S::kStages) & 1);
  } else {
    // ------------------------------------------------------------ products
    // (after a failed wait the warps go on without waiting: their barriers
    // below stay in step, the results are worthless and the error is recorded)
    uint32_t t = 0;
    bool lost = false;  // a wait has run out
    const uint32_t base = smem_u32(smem);
    // this lane's keys of the warp's 16: the two of its scores, the four of V
    const int key_s = 4 * (lg & 1) + ((lg >> 1) ^ (lg & 1));  // and + 8
    auto key_v = [&](int i) { return 8 * (i >> 1) + 4 * (i & 1) + (lt ^ (i & 1)); };
    // where they start in a stage
    const uint32_t row_s = uint32_t(warp * kKv4Unit + key_s);
    const uint32_t k_off = row_s * kRowC + uint32_t(lt) * (kRowC / 4);
    const uint32_t ks_off = uint32_t(2 * S::kCodes) + row_s * kRowS + uint32_t(lt) * (kRowS / 4);
    uint32_t v_off[2], vs_off[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t r = uint32_t(warp * kKv4Unit + key_v(i));
      v_off[i] = uint32_t(S::kCodes) + r * kRowC + uint32_t(lg) * (kRowC / 8);
      vs_off[i] = uint32_t(2 * S::kCodes + S::kScales) + r * kRowS + uint32_t(lg) * kRowS / 8;
    }
    pieces([&](int n, int g, int seg, int ctx, int units, int u0, int u1) {
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
        for (int s = 0; s < KS; s += 2) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (on) w = *reinterpret_cast<const uint4*>(qp + s * 4);
          qf[nt][s][0] = w.x, qf[nt][s][1] = w.y, qf[nt][s + 1][0] = w.z, qf[nt][s + 1][1] = w.w;
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mx = fmaxf(mx, fmaxf(fabsf(bf16lo(qf[nt][s][i])), fabsf(bf16hi(qf[nt][s][i]))));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        float up, f;
        kv4_query_scale(mx, a.sc, a.sc_e, &up, &f);
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
          move |= fmaxf(fmax3f(x[nt][0], x[nt][1], x[nt][2]), x[nt][3]) > kKv4Above;
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float mx = fmaxf(s[nt][i], s[nt][i + 2]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
              float b = mx * f[nt][i];
              b = fabsf(b) > kKv4Far ? __fadd_rd(__fmul_rd(mx, f[nt][i]), -kKv4Below) : b - kKv4Below;
              b = fmaxf(m[nt][i], b);
              const float w = fast_exp2(m[nt][i] - b);
              m[nt][i] = b;
              l[nt][i] *= w;
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                o[nt][k][i] *= w;
                o[nt][k][i + 2] *= w;
              }
#pragma unroll
              for (int j = i; j < 4; j += 2) {
                x[nt][j] = fmaf(s[nt][j], f[nt][i], -b);
                if (x[nt][j] > kKv4Above) x[nt][j] = kKv4Above;  // (kKv4Far; a NaN stays)
              }
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

      // ---------------- the block's own keys, in bf16 (at most 16): the ninth warp
      // (P in units of v_scale so that O has one unit for all keys)
      if (a.bk && u0 == 0 && warp == kKv4Warps) {
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
        // every load first: the lane's runs of its two keys, its four values
        uint32_t kw[2][KS][2], vw[4][KS];
        auto run = [&](const uint16_t* base, int j, int off, uint32_t* to, int chunks) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= chunks) break;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (j < a.B)
              w = *reinterpret_cast<const uint4*>(base + ((size_t(n) * a.B + j) * a.Hkv + g) * D +
                                                  off + i * 8);
            to[4 * i] = w.x, to[4 * i + 1] = w.y, to[4 * i + 2] = w.z, to[4 * i + 3] = w.w;
          }
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) run(a.bk, key_s + 8 * i, lt * (D / 4), &kw[i][0][0], D / 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) run(a.bv, key_v(i), lg * (D / 8), vw[i], D / 64);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = nt * 8 + lg;
          const uint16_t* qp =
              a.q + ((size_t(n) * a.B + (r < R ? r / G : 0)) * a.Hq + g * G + (r < R ? r % G : 0)) * D +
              lt * (D / 4);
          uint32_t qb[KS][2];
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (r < R) w = *reinterpret_cast<const uint4*>(qp + k * 4);
            qb[k][0] = w.x, qb[k][1] = w.y, qb[k + 1][0] = w.z, qb[k + 1][1] = w.w;
          }
#pragma unroll
          for (int k = 0; k < KS; ++k)
            mma_bf16(s[nt], kw[0][k][0], kw[1][k][0], kw[0][k][1], kw[1][k][1], qb[k][0], qb[k][1]);
        }
        float f[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f[nt][0] = f[nt][1] = a.scale * 1.4426950408889634f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key_s + 8 * (i >> 1) >= a.B) s[nt][i] = -INFINITY;
        }
        probabilities(s, f);
        const float iv = 1.f / a.c.v_scale;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[nt][i] *= iv;
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {  // P as the sum of two bf16 numbers
          uint32_t p0[NT], p1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            p0[nt] = transpose8x8(take_bf16(s[nt][0], s[nt][1]));
            p1[nt] = transpose8x8(take_bf16(s[nt][2], s[nt][3]));
          }
#pragma unroll
          for (int k = 0; k < KS; ++k)  // channels lg*D/8 + 2k, + 2k+1 of each key
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_bf16(o[nt][k], __byte_perm(vw[0][k], vw[1][k], 0x5410),
                       __byte_perm(vw[0][k], vw[1][k], 0x7632),
                       __byte_perm(vw[2][k], vw[3][k], 0x5410),
                       __byte_perm(vw[2][k], vw[3][k], 0x7632), p0[nt], p1[nt]);
        }
      }

      // ------------------------------------------------------ cache tiles
      const int tiles = min(u1, (ctx + kKv4Tile - 1) / kKv4Tile);
#pragma unroll 1
      for (int u = u0; u < tiles && warp < kKv4Warps; ++u, ++t) {
        const uint32_t st = t % S::kStages, sm = base + st * uint32_t(S::kStage);
        if (!lost) lost = !wait(&full[st], (t / S::kStages) & 1, W_STAGE_FULL);
        // (every read first, not after the count: a tile of which the warp has no key
        // is rare)
        const int valid_lane = int(*(volatile uint8_t*)&counts[st][warp]);
        const uint32_t ka = sm + k_off, ksa = sm + ks_off;
        uint32_t kw[2][D / 32], ksc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (D == 128) {
            const uint4 w = lds128(ka + uint32_t(i * 8 * kRowC));
            kw[i][0] = w.x, kw[i][1] = w.y, kw[i][2] = w.z, kw[i][3] = w.w;
            ksc[i] = lds_u16(ksa + uint32_t(i * 8 * kRowS));
          } else {
            const uint2 w = lds64(ka + uint32_t(i * 8 * kRowC));
            kw[i][0] = w.x, kw[i][1] = w.y;
            ksc[i] = lds_u8(ksa + uint32_t(i * 8 * kRowS));
          }
        }
        uint32_t vw[4][D / 64], vsc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t va = sm + v_off[i & 1] + uint32_t((i >> 1) * 8 * kRowC);
          if constexpr (D == 128) {
            const uint2 w = lds64(va);
            vw[i][0] = w.x, vw[i][1] = w.y;
          } else {
            vw[i][0] = lds32(va);
          }
          vsc[i] = lds_u8(sm + vs_off[i & 1] + uint32_t((i >> 1) * 8 * kRowS));
        }
        const int valid = warp_same(valid_lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (valid > 0) {
          float s[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
          const uint32_t s0 = e4m3x2_to_half2(ksc[0]), s1 = e4m3x2_to_half2(ksc[1]);
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {  // a word of codes per key: two k steps
            uint32_t h0[4], h1[4];
            e2m1x8_to_half2(kw[0][w], h0);
            e2m1x8_to_half2(kw[1][w], h1);
            const uint32_t f0 = bcast16(s0, w >> 1), f1 = bcast16(s1, w >> 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              h0[i] = hmul2(h0[i], f0);
              h1[i] = hmul2(h1[i], f1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(s[nt], h0[0], h1[0], h0[1], h1[1], qf[nt][2 * w][0], qf[nt][2 * w][1]);
              mma_f16(s[nt], h0[2], h1[2], h0[3], h1[3], qf[nt][2 * w + 1][0],
                      qf[nt][2 * w + 1][1]);
            }
          }
          if (valid < kKv4Unit) {  // keys past the length
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (key_s + 8 * (i >> 1) >= valid) s[nt][i] = -INFINITY;
            // such a row may hold any bytes: 0 * NaN must not arise
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key_v(i) >= valid) vsc[i] = 0;
          }
          probabilities(s, rs);
          uint32_t p0[NT], p1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            p0[nt] = transpose8x8(pack_half2(s[nt][0], s[nt][1]));
            p1[nt] = transpose8x8(pack_half2(s[nt][2], s[nt][3]));
          }
          const uint32_t f0 = e4m3x2_to_half2(vsc[0] | vsc[1] << 8),
                         f1 = e4m3x2_to_half2(vsc[2] | vsc[3] << 8);
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            uint32_t e0[4], d0[4], e1[4], d1[4];  // even, odd channels of the two key pairs
            e2m1x8_to_half2((vw[0][w] & 0x0F0F0F0Fu) | ((vw[1][w] << 4) & 0xF0F0F0F0u), e0);
            e2m1x8_to_half2(((vw[0][w] >> 4) & 0x0F0F0F0Fu) | (vw[1][w] & 0xF0F0F0F0u), d0);
            e2m1x8_to_half2((vw[2][w] & 0x0F0F0F0Fu) | ((vw[3][w] << 4) & 0xF0F0F0F0u), e1);
            e2m1x8_to_half2(((vw[2][w] >> 4) & 0x0F0F0F0Fu) | (vw[3][w] & 0xF0F0F0F0u), d1);
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
          float* dst = red + (warp * RT + nt * 8 + 2 * lt + i) * (D + 4) + lg * (D / 8);
#pragma unroll
          for (int k = 0; k < KS; ++k)  // channels 2k, 2k+1 of this lane's run
            *reinterpret_cast<float2*>(dst + 2 * k) = make_float2(o[nt][k][i], o[nt][k][i + 2]);
        }
      product_bar();
      const bool whole = u0 == 0 && u1 == units;  // no other piece of this segment
      const int slot = int(blockIdx.x) + seg;
      for (int i = threadIdx.x; i < RT * (D / 4); i += kKv4Parts * 32) {
        // (neighbouring threads write neighbouring channels of out, rows of a partial)
        const int r = whole ? i / (D / 4) : i % RT, c4 = whole ? i % (D / 4) : i / RT;
        if (r >= R) continue;
        float M = -FLT_MAX;
#pragma unroll
        for (int w = 0; w < kKv4Parts; ++w) M = fmaxf(M, red_m[w][r]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < kKv4Parts; ++w) {
          const float f = fast_exp2(red_m[w][r] - M);
          const float4 x =
              *reinterpret_cast<const float4*>(red + (w * RT + r) * (D + 4) + c4 * 4);
          L += f * red_l[w][r];
          acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
        }
        if (whole) {
          const float inv = L == 0.f ? 0.f : a.c.v_scale / L;
          *reinterpret_cast<uint2*>(
              a.out + ((size_t(n) * a.B + r / G) * a.Hq + g * G + r % G) * D + c4 * 4) =
              make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        } else {
          reinterpret_cast<float4*>(a.opart)[(size_t(slot) * (D / 4) + c4) * a.R16 + r] = acc;
          if (c4 == 0) a.ml[size_t(slot) * a.R16 + r] = make_float2(M, L);
        }
      }
      product_bar();  // the reduction buffers are free for the next piece
    });
  }
  __syncthreads();
  if (threadIdx.x == 0 && failed)
    record_error(err, DEV_TIMEOUT_TMA | DEV_K_KV4_ROWS | (failed << 16));
}

// Joins the pieces of every segment that has more than one, and writes zeros
// for segments without keys.  grid (N*Hkv, ceil(R / Rows)): Rows rows' chunks of
// four channels per D/4 * Rows threads, and Threads over that many groups, each with
// every such-and-suchth partial, five in flight, so that the pieces of a long
// context travel at once; the groups are added in order.
template <int D, int Rows, int Threads>
__global__ void __launch_bounds__(Threads)
    kv4_join_kernel(const Kv4AttnArgs a, int blk_units) {
  constexpr int TPG = Rows * (D / 4), GR = Threads / TPG;
  __shared__ float4 part[GR][TPG];
  __shared__ float part_m[GR][Rows], part_l[GR][Rows];
  const int seg = blockIdx.x, n = seg / a.Hkv, g = seg - n * a.Hkv;
  const int G = a.Hq / a.Hkv, R = a.B * G;
  const int grp = threadIdx.x / TPG, item = threadIdx.x % TPG;
  const int rr = item % Rows, c4 = item / Rows;
  const int r = int(blockIdx.y) * Rows + rr, rc = min(r, R - 1);
  const Kv4Split split = kv4_split(kv4_total_units(a.ctx, a.N, a.L_max, blk_units, a.pad), a.Hkv, a.ctas);
  const int units = kv4_units(a.ctx[n], a.L_max, blk_units, a.pad);
  const int first =
      a.Hkv * kv4_total_units(a.ctx, n, a.L_max, blk_units, a.pad) + g * units;
  // The lengths were read before the grid-dependency wait: they were written
  // before the attention kernel's own wait ended, and it lets this kernel start
  // only after that.
  griddep_enter();
  uint2* out = reinterpret_cast<uint2*>(
      a.out + ((size_t(n) * a.B + rc / G) * a.Hq + g * G + rc % G) * D + c4 * 4);
  if (units == 0) {
    if (grp == 0 && r < R) *out = make_uint2(0, 0);
    return;
  }
  int c0 = (first + a.pad) / split.share, c1 = (first + units - 1) / split.share;
  if (c0 == c1) return;  // one piece: written by the attention kernel
  c0 += seg, c1 += seg;  // its partials
  const float4* op = reinterpret_cast<const float4*>(a.opart) + size_t(c4) * a.R16 + rc;
  float M = -FLT_MAX, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kFly = 5;
  for (int c = c0 + grp; c <= c1; c += kFly * GR) {
    float2 p[kFly];
    float4 x[kFly];
#pragma unroll
    for (int i = 0; i < kFly; ++i) {
      const int ci = c + i * GR;
      p[i] = make_float2(-FLT_MAX, 0.f), x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ci <= c1) {
        p[i] = a.ml[size_t(ci) * a.R16 + rc];
        x[i] = op[size_t(ci) * (D / 4) * a.R16];
      }
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

// Self-test of Kv4Wait: a warp waits on a completed barrier, then on one that nothing
// completes, and reports as the attention kernels do.
__global__ void kv4_wait_kernel(uint32_t tries, uint32_t* err) {
  __shared__ uint64_t done, open;
  __shared__ uint32_t failed;
  if (threadIdx.x == 0) {
    mbar_init(&done, 1);
    mbar_init(&open, 1);
    failed = 0;
    fence_mbar_init();
    mbar_arrive(&done);
  }
  __syncthreads();
  const Kv4Wait wait{&failed, tries};
  if (wait(&done, 0, W_STAGE_FREE)) wait(&open, 0, W_STAGE_FULL);
  __syncthreads();
  if (threadIdx.x == 0 && failed)
    record_error(err, DEV_TIMEOUT_TMA | DEV_K_KV4_ROWS | (failed << 16));
}

// ------------------------------------------------------------------- host

cudaError_t launch_kv4_wait(uint32_t tries, uint32_t* err, cudaStream_t st) {
  kv4_wait_kernel<<<1, 32, 0, st>>>(tries, err);
  return cudaGetLastError();
}

template <int D, int NT>
static cudaError_t launch_rows(const Kv4AttnArgs& a, uint32_t* err, cudaStream_t st) {
  const size_t smem = RowsSmem<D, NT>::kTotal;
  HERALD_CHECK_LAUNCH(ensure_smem(kv4_attn_kernel<D, NT>, smem));
  return launch_k("kv4_attn_kernel", kv4_attn_kernel<D, NT>, dim3(unsigned(a.ctas)),
                  dim3(kKv4Threads), smem, st, a, err);
}

template <int D>
static cudaError_t launch_join(const Kv4AttnArgs& a, int blk_units, int R, int num_sms,
                               cudaStream_t st) {
  auto go = [&](auto* kernel, int rows, int threads) {
    return launch_k("kv4_join_kernel", kernel, dim3(unsigned(a.N * a.Hkv), unsigned(cdiv(R, rows))),
                    dim3(unsigned(threads)), 0, st, a, blk_units);
  };
  const int64_t segs = int64_t(a.N) * a.Hkv;
  // While one wave holds them, CTAs of 1024 threads keep more partials of a row in
  // flight; more CTAs than that want small ones, several to an SM.  Us per call with
  // only (4, 1024) and (8, 1024) / as chosen / only (8, 256): token at 128K 39 / 38.6
  // / 41.6, 32 tokens at 32K 29 / 29 / 39, 64 ragged tokens 83 / 77 / 77, 32 tokens at
  // 4 x 64K 134 / 127 / 128, 12 ragged blocks of 64 167 / 119 / 120.
  if (segs * cdiv(R, 4) <= num_sms) return go(kv4_join_kernel<D, 4, 1024>, 4, 1024);
  if (segs * cdiv(R, 8) <= num_sms) return go(kv4_join_kernel<D, 8, 1024>, 8, 1024);
  return go(kv4_join_kernel<D, 8, 256>, 8, 256);
}

// Workspace: error word, then (m, l) and O of every partial.
struct Kv4Ws {
  size_t ml, opart, total;
  int R16;
};
static Kv4Ws kv4_ws(const herald_dims& dm) {
  Kv4Ws w;
  w.R16 = cdiv(dm.B * (dm.Hq / dm.Hkv), 16) * 16;
  const size_t slots = size_t(kKv4MaxCtas) + size_t(dm.N) * dm.Hkv;
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
  int es, ek, ep;
  const float ms = frexpf(scale, &es), mk = frexpf(c.k_scale, &ek);
  a.sc = 2.f * frexpf(ms * mk * 1.4426950408889634f, &ep);
  a.sc_e = es + ek + ep - 1;
  a.N = dm.N, a.Hq = dm.Hq, a.Hkv = dm.Hkv, a.B = dm.B, a.L_max = dm.L_max, a.R16 = w.R16;
  a.c = c;
  const bool tc = R > kKv4MmaRows;
  uint32_t* err = reinterpret_cast<uint32_t*>(p);
  a.ctas = std::min(kKv4MaxCtas, (!tc && R <= 8 ? 2 : 1) * num_sms);
  a.pad = tc ? kKv4PadTc : kKv4PadRows;
  if (tc)
    HERALD_CHECK_LAUNCH(launch_kv4_attn_tc(dm.d, R, a, err, st));
  else if (dm.d == 128)
    HERALD_CHECK_LAUNCH(
        (R <= 8 ? launch_rows<128, 1>(a, err, st) : launch_rows<128, 2>(a, err, st)));
  else
    HERALD_CHECK_LAUNCH((R <= 8 ? launch_rows<64, 1>(a, err, st) : launch_rows<64, 2>(a, err, st)));
  const int blk_units = !bk ? 0 : tc ? cdiv(dm.B, kKv4Tile) : kKv4BlkJoined;
  HERALD_CHECK_LAUNCH(dm.d == 128 ? launch_join<128>(a, blk_units, R, num_sms, st)
                                  : launch_join<64>(a, blk_units, R, num_sms, st));
  return cudaGetLastError();
}

HERALD_DEBUG_WORD_READER(debug_take_kv4_attn)

}  // namespace herald
