// kv8_rows.cu -- attention over the paged 8-bit cache on the 5th-generation tensor
// cores for few query rows per KV head (one token, a short draft): bound by the
// cache's bytes.
//
// The codes are operands as they are held: e4m3 tiles of 128 keys go from the pages to
// shared memory by TMA, swizzled on the way, and no instruction touches them after
// that.  The keys are the M side of both products, so that few query rows fill few
// columns and not a 128-row tile:
//   S^T [128 keys x rows] = K [128 x d] Q^T [d x rows]       (K's rows as they lie)
//   O^T [d x rows]       += V^T [d x 128 keys] P [128 x rows] (V's rows read as columns)
// The other operands are made e4m3 too, without losing their bits, as sums of numbers
// of 4 bits in columns of their own:
//   q = (q0 + q1/16) 2^x: a bf16 has 8 bits; x brings the row's largest to [2^7, 2^8)
//   p = p0 + p1/2^5 + p2/2^10 + p3/2^15 (kKv8Parts), with p at most 2^8: what a number leaves
//   is then at most 2^3, and 2^5 times that 2^8 again; the last one's step is 2^-24 (with
//   steps of 2^4 between them it was 2^-21, and weights of 2^-26 of a row's largest and less,
//   many of which may make its output beside a sink without value, were 0)
// and the columns are added in fp32 afterwards.  A key's scale (its block's) multiplies its
// scores.  A value's exponent e_v goes into the weight's own, p = 2^(x + e_v - m), and
// out of the row's sum again, l += p 2^-e_v: O has one unit.  p's steps end at 2^-24, where
// a row's largest p is 2^4 at least: keys 2^-29 and less below it (values of so small a
// scale, or weights) count in the sum only.
//
// One CTA per SM walks its share of the keys (kv4_split):
//   warps 0-3, 4-7  softmax: two streams that take the tiles in turn, a thread per key of
//              the tile (its TMEM lane), rows in registers; each keeps the sum of its own
//              keys' weights, each stream its own base m and O, added up at a piece's end
//   warp 8     the issuer of both products, S two tiles ahead of P V
//   warps 9, 10  copy tiles of keys and of values into a ring each, and look up pages and
//              scales, four tiles of them (32 lanes: 8 groups of 16 keys each) ahead.  A tile's
//              keys leave after its scores; its values wait for the weights, some tiles longer
//   warp 11    stages the queries of the next piece (the first piece's: the softmax warps)
// A row's exponent base m is set 4 below its largest exponent and stays while no p passes
// 2^8; a stream's four warps vote on that in one barrier a tile.  Else the tile's row maxima
// are exchanged, O is scaled once the products before it are done, and l follows.
//
// What bounds it: with up to 8 rows the cache's bytes; 64 ragged sequences of up to 8K tokens
// 93.4 us for 580 MB (6.2 TB/s, 93% of the copy rate), one of 128K 46.5 us for 268 MB, of which 6
// are launch, lengths, the first tile and the join.  With 16 rows a tile's softmax (four
// conversions and their remainders a weight) takes 1,060 cycles, a little more than its copies,
// and a piece's start and end 2 to 3 us: 102 us.  One stream took 121 there: a thread's steps wait on
// one another, and the two streams fill each other's waits.
#include <float.h>

#include "kv8.cuh"
#include "tc_common.cuh"

namespace herald {

constexpr int kKv8Parts = 4;               // e4m3 numbers of a weight
constexpr float kKv8At = 4.f, kKv8Most = 8.f;  // log2 p of a new base's row, and the largest
constexpr int kKv8RowsThreads = 384;       // 12 warps
constexpr int kKv8Metas = 16;              // tiles whose scales are held

// Waits of the kernel (bits 16-31 of the error word).
enum : uint32_t {
  W8_K_FREE = 1, W8_K_FULL = 2, W8_Q_FREE = 4, W8_Q_FULL = 8, W8_S_FULL = 0x10,
  W8_P_FULL = 0x20, W8_PV_DONE = 0x40, W8_V_FREE = 0x80, W8_V_FULL = 0x100, W8_META = 0x200
};

template <int D, int RP>
struct Kv8Rows {
  static constexpr int kNs = 2 * RP;                // columns of S: q0 rows, q1 rows
  static constexpr int kNo = kKv8Parts * RP;        // columns of O, bytes of a key's P
  static constexpr uint32_t kTile = 128u * D;       // bytes of 128 keys
  // Stages of 128 keys and of 128 values.  160 KB in flight an SM: more only makes pages of
  // other rows meet in DRAM (64 sequences of up to 8K tokens, 1 and 16 rows: 5 and 5 stages
  // 93.6 and 104.7 us, 4 and 5 93.6 and 105.7, 3 and 4 95.3 and 102.7, 4 and 7 93.4 and 116.1,
  // 6 and 7 97.9 and, 5 and 7, 112.7; one sequence of 128K 46.9 / 46.8 / 47.8 / 48.0 / 49.6).
  static constexpr int kKs = D == 64 ? 10 : 5, kVs = kKs;
  static constexpr uint32_t kQ = uint32_t(kNs) * D, kP = 128u * kNo;
  static constexpr uint32_t kSmem = (kKs + kVs) * kTile + 2 * kQ + 2 * kP + 1024;
  static constexpr int kSBufs = 4;
  static constexpr uint32_t kCols = kSBufs * kNs + 2 * kNo;  // of tensor memory
  // scales are written with a tile's keys, which wait for the products of kKs before; the
  // weights of three before those have been made by then
  static_assert(kKs + 3 <= kKv8Metas, "scales outlive their reader");
};

// What the softmax needs of 16 keys: 2^e_k, e_v, 2^-e_v and how many of them count.
struct __align__(16) Kv8Meta {
  float sk, ev, iv;
  int keys;
};

// x -> 32 (x - e4m3(x)) for a pair, returning the codes: what the next number holds.
HERALD_DEV uint32_t split_e4m3(float& a, float& b) {
  const uint32_t w = float2_to_e4m3(a, b);
  const uint32_t h = e4m3x2_to_half2(w);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  a = fmaf(f.x, -32.f, a * 32.f);
  b = fmaf(f.y, -32.f, b * 32.f);
  return w;
}

HERALD_DEV bool soft_any(int g, bool x) {  // any of a stream's threads
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(x)), "r"(1 + g)
      : "memory");
  return r != 0;
}
HERALD_DEV void soft_bar(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }
HERALD_DEV void both_bar() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

template <int N>
HERALD_DEV void tmem_load(uint32_t at, float (&v)[N]) {
  if constexpr (N == 16) {
    tmem_ld16(at, v);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 32)
      tmem_ld32(at + uint32_t(c), *reinterpret_cast<float(*)[32]>(v + c));
  }
}

// N = 4 or 8 columns of this thread's lane at each of four places.
HERALD_DEV void tmem_ld_parts(uint32_t at, uint32_t step, uint32_t (&r)[4][4]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%4, %5, %6, %7}, [%17];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%8, %9, %10, %11}, [%18];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%12, %13, %14, %15}, [%19];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0][0]), "=r"(r[0][1]), "=r"(r[0][2]), "=r"(r[0][3]), "=r"(r[1][0]), "=r"(r[1][1]),
        "=r"(r[1][2]), "=r"(r[1][3]), "=r"(r[2][0]), "=r"(r[2][1]), "=r"(r[2][2]), "=r"(r[2][3]),
        "=r"(r[3][0]), "=r"(r[3][1]), "=r"(r[3][2]), "=r"(r[3][3])
      : "r"(at), "r"(at + step), "r"(at + 2 * step), "r"(at + 3 * step)
      : "memory");
}
HERALD_DEV void tmem_ld_parts(uint32_t at, uint32_t step, uint32_t (&r)[4][8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%33];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%34];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%24, %25, %26, %27, %28, %29, %30, %31}, [%35];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0][0]), "=r"(r[0][1]), "=r"(r[0][2]), "=r"(r[0][3]), "=r"(r[0][4]), "=r"(r[0][5]),
        "=r"(r[0][6]), "=r"(r[0][7]), "=r"(r[1][0]), "=r"(r[1][1]), "=r"(r[1][2]), "=r"(r[1][3]),
        "=r"(r[1][4]), "=r"(r[1][5]), "=r"(r[1][6]), "=r"(r[1][7]), "=r"(r[2][0]), "=r"(r[2][1]),
        "=r"(r[2][2]), "=r"(r[2][3]), "=r"(r[2][4]), "=r"(r[2][5]), "=r"(r[2][6]), "=r"(r[2][7]),
        "=r"(r[3][0]), "=r"(r[3][1]), "=r"(r[3][2]), "=r"(r[3][3]), "=r"(r[3][4]), "=r"(r[3][5]),
        "=r"(r[3][6]), "=r"(r[3][7])
      : "r"(at), "r"(at + step), "r"(at + 2 * step), "r"(at + 3 * step)
      : "memory");
}

// All N rows' values over a warp's lanes at once: each step halves the rows a lane holds.
// Lane i < N returns row i's, as do lanes i + N and so on.
template <int N, typename Op>
HERALD_DEV float warp_rows(float (&v)[N], Op&& op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = N / 2; h >= 1; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, h));
    }
  }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

// Queries of a piece: D/8 lanes hold a row, eight channels each; a warp takes passes of
// 32 / (D/8) rows.
template <int D>
struct Kv8Query {
  static constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // of a row, of a pass
  static constexpr int passes(int rows) { return rows / kRows; }
  uint4 x;
  HERALD_DEV void load(const Kv8AttnArgs& a, int n, int g, int pass, int lane) {
    const int G = a.Hq / a.Hkv, r = pass * kRows + lane / kLanes;
    x = make_uint4(0, 0, 0, 0);
    if (r < a.B * G)
      x = *reinterpret_cast<const uint4*>(
          a.q + ((size_t(n) * a.B + r / G) * a.Hq + g * G + r % G) * D + lane % kLanes * 8);
  }
};
// Passes pass0 to pass0 + P as operands and their score factors.
template <int D, int RP, int P>
HERALD_DEV void stage_queries(const Kv8Query<D> (&q)[P], int pass0, int lane, float scale,
                              uint8_t* dst, float* row_f) {
  constexpr int LPR = Kv8Query<D>::kLanes;
  const int c = lane % LPR;
  float mx[P];  // (the rows' maxima side by side: their steps wait on one another)
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint4& x = q[p].x;
    const uint32_t m = max_bf16x2_abs(
        max_bf16x2_abs(max_bf16x2_abs(max_bf16x2_abs(0, x.x), x.y), x.z), x.w);
    mx[p] = fmaxf(bf16lo(m), bf16hi(m));
  }
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
    for (int p = 0; p < P; ++p) mx[p] = fmaxf(mx[p], __shfl_xor_sync(0xffffffffu, mx[p], o));
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t r = uint32_t((pass0 + p) * Kv8Query<D>::kRows + lane / LPR);
    const uint32_t half = uint32_t(c & 1) * 8u;
    float up, f;
    kv8_query_scale(mx[p], scale, &up, &f);
    const uint32_t w[4] = {q[p].x.x, q[p].x.y, q[p].x.z, q[p].x.w};
    uint32_t v0[4], v1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = pack_half2(bf16lo(w[i]) * up, bf16hi(w[i]) * up);
      v0[i] = half2_to_e4m3(h);
      const uint32_t rest = hsub2(h, e4m3x2_to_half2(v0[i]));  // what q0 left, times 16
      v1[i] = half2_to_e4m3(hmul2(rest, 0x4C004C00u));
    }
    *reinterpret_cast<uint2*>(dst + rows_off<D>(r, uint32_t(c >> 1)) + half) =
        make_uint2(v0[0] | v0[1] << 16, v0[2] | v0[3] << 16);
    *reinterpret_cast<uint2*>(dst + rows_off<D>(uint32_t(RP) + r, uint32_t(c >> 1)) + half) =
        make_uint2(v1[0] | v1[1] << 16, v1[2] | v1[3] << 16);
    if (c == 0) row_f[r] = f;
  }
}

template <int D, int RP>
__global__ void __launch_bounds__(kKv8RowsThreads, 1)
    kv8_rows_kernel(const Kv8AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, uint32_t* err) {
  using S = Kv8Rows<D, RP>;
  constexpr int NS = S::kNs, NO = S::kNo, KS = S::kKs, VS = S::kVs, SB = S::kSBufs;
  constexpr int MB = kKv8Metas;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t k_full[KS], k_free[KS], v_full[VS], v_free[VS], m_full[MB], q_full[2],
      q_free[2], s_full[SB], p_full[2], pv_done[2], all_done;
  __shared__ uint32_t tmem_base, failed;
  __shared__ Kv8Share share;
  __shared__ Kv8Meta meta[MB][8];
  __shared__ __align__(16) float row_f[2][RP];  // score factors of the rows
  __shared__ __align__(16) float red[2][4][RP];  // row maxima of a stream's warps
  // a piece's bases and the warps' sums of both streams
  __shared__ __align__(16) float row_m[2][RP];
  __shared__ float row_l[2][4][RP];
  uint8_t* base = align1024(smem_raw);
  uint8_t *Vs = base + KS * S::kTile, *Qs = Vs + VS * S::kTile, *Ps = Qs + 2 * S::kQ;
  const int warp = warp_same(int(threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) mbar_init(&k_full[i], 1), mbar_init(&k_free[i], 1);
    for (int i = 0; i < VS; ++i) mbar_init(&v_full[i], 1), mbar_init(&v_free[i], 1);
    for (int i = 0; i < MB; ++i) mbar_init(&m_full[i], 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(&q_full[i], 1), mbar_init(&q_free[i], 9), mbar_init(&p_full[i], 4),
          mbar_init(&pv_done[i], 1);
    for (int i = 0; i < SB; ++i) mbar_init(&s_full[i], 1);
    mbar_init(&all_done, 1);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 9 && lane == 0) tma_prefetch_desc(&kmap);
  if (warp == 10 && lane == 0) tma_prefetch_desc(&vmap);
  tmem_setup(&tmem_base, S::kCols);
  const uint32_t tm = tmem_base, to = tm + SB * NS;  // S buffers, then both streams' O
  griddep_enter();
  const Kv4Wait wait{&failed};
  const int G = a.Hq / a.Hkv, R = a.B * G;
  if (warp == 0) {
    const Kv8Share mine = kv8_share(a, int(blockIdx.x));
    if (lane == 0) share = mine;
  }
  __syncthreads();

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    // (after a failed wait these warps go on without waiting: the barriers among them
    // stay in step, the results are worthless and the error is recorded)
    bool lost = false;
    auto await = [&](uint64_t* bar, uint32_t parity, uint32_t which) {
      if (!lost) lost = !wait(bar, parity, which);
    };
    const int w = warp >> 2, wq = warp & 3, key = int(threadIdx.x) & 127;  // stream, quarter, key
    const uint32_t lanes = uint32_t(wq * 32) << 16, tow = to + lanes + uint32_t(w) * NO;
    uint32_t t0 = 0, np = 0;  // tiles and pieces of the CTA
    kv8_pieces(a, share, [&](int n, int g, int seg, int ctx, int u0, int u1) -> bool {
      debug_flag(threadIdx.x == 0 && a.ctx[n] != ctx, DEV_BAD_COUNT);
      const uint32_t qb = np & 1;
      if (np == 0) {  // a pass for each warp: one warp alone takes 4,300 cycles for 16 rows
        if (warp < Kv8Query<D>::passes(RP)) {
          Kv8Query<D> x[1];
          x[0].load(a, n, g, warp, lane);
          stage_queries<D, RP, 1>(x, warp, lane, a.scale, Qs, row_f[0]);
          fence_proxy_async_smem();
        }
        both_bar();
        if (threadIdx.x == 0) mbar_arrive(&q_full[0]);
      }
      await(&q_full[qb], (np >> 1) & 1, W8_Q_FULL);
      float f[RP], m[RP], l[RP];
#pragma unroll
      for (int r = 0; r < RP; r += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&row_f[qb][r]);
        f[r] = x.x, f[r + 1] = x.y, f[r + 2] = x.z, f[r + 3] = x.w;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_free[qb]);
      ++np;
#pragma unroll
      for (int r = 0; r < RP; ++r) m[r] = -FLT_MAX, l[r] = 0.f;
      const uint32_t t1 = t0 + uint32_t(u1 - u0), mine = t0 + ((t0 ^ uint32_t(w)) & 1);
#pragma unroll 1
      for (uint32_t t = mine; t < t1; t += 2) {
        await(&m_full[t % MB], (t / MB) & 1, W8_META);
        await(&s_full[t % SB], (t / SB) & 1, W8_S_FULL);
        tc_fence_after();
        const Kv8Meta mt = meta[t % MB][key >> 4];
        const bool on = (key & 15) < mt.keys;
        float s[RP], p[RP];
        {
          float x[NS];
          tmem_load<NS>(tm + lanes + t % SB * NS, x);
          // (times the key's scale, an exact step, before the row's factor: the two factors'
          // product might leave fp32 where the score does not)
#pragma unroll
          for (int r = 0; r < RP; ++r) s[r] = fmaf(x[RP + r], 0.0625f, x[r]) * mt.sk;
        }
        bool move = false;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          p[r] = on ? fmaf(s[r], f[r], mt.ev - m[r]) : -INFINITY;
          move |= p[r] > kKv8Most;
        }
        move = soft_any(w, move);
        // P of the stream's tile before has been read, and is in O
        if (t >= 2) await(&pv_done[w], ((t >> 1) - 1) & 1, W8_PV_DONE);
        if (move) {
          // row maxima of the tile, rounded down: where scores are so large that fp32's
          // steps are no longer small, a base above them all would leave no weight
          float z[RP];
#pragma unroll
          for (int r = 0; r < RP; ++r)
            z[r] = on ? __fadd_rd(__fmul_rd(s[r], f[r]), mt.ev) : -INFINITY;
          const float mx = warp_rows(z, [](float x, float y) { return fmaxf(x, y); });
          if (lane < RP) red[w][wq][lane] = mx;
          soft_bar(w);
          float k[RP];
#pragma unroll
          for (int r = 0; r < RP; r += 4) {
            float4 x = *reinterpret_cast<const float4*>(&red[w][0][r]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
              const float4 y = *reinterpret_cast<const float4*>(&red[w][i][r]);
              x.x = fmaxf(x.x, y.x), x.y = fmaxf(x.y, y.y), x.z = fmaxf(x.z, y.z), x.w = fmaxf(x.w, y.w);
            }
            k[r] = x.x, k[r + 1] = x.y, k[r + 2] = x.z, k[r + 3] = x.w;
          }
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const float m1 = fmaxf(__fadd_rd(k[r], -kKv8At), m[r]);
            k[r] = fast_exp2(m[r] - m1);
            m[r] = m1;
            l[r] *= k[r];
            const float x = fmaf(s[r], f[r], mt.ev - m1);
            p[r] = !on ? -INFINITY : x > kKv8Most ? kKv8Most : x;  // (a NaN stays)
          }
          if (t > mine) {
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < NO; c += 32) {
              float o[32];
              tmem_ld32(tow + uint32_t(c), o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= k[(c + i) % RP];
              tmem_st32(tow + uint32_t(c), o);
            }
            tmem_wait_st();
          }
          soft_bar(w);  // (the maxima have been read)
        }
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          p[r] = fast_exp2(p[r]);
          l[r] = fmaf(p[r], mt.iv, l[r]);
        }
        uint8_t* dst = Ps + uint32_t(w) * S::kP;
        uint32_t pk[NO / 4];
#pragma unroll
        for (int i = 0; i < kKv8Parts; ++i)
#pragma unroll
          for (int r = 0; r < RP; r += 4)
            pk[(i * RP + r) / 4] = split_e4m3(p[r], p[r + 1]) | split_e4m3(p[r + 2], p[r + 3]) << 16;
#pragma unroll
        for (int c = 0; c < NO / 16; ++c)
          *reinterpret_cast<uint4*>(dst + rows_off<NO>(uint32_t(key), uint32_t(c))) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        if (__any_sync(0xffffffffu, !on)) {  // a row without a key may hold any bytes: 0 * NaN
          await(&v_full[t % VS], (t / VS) & 1, W8_V_FULL);  // must not arise
          if (!on) {
            uint4* v = reinterpret_cast<uint4*>(Vs + t % VS * S::kTile + uint32_t(key) * D);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) v[c] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      // the piece's partials: l over the stream's keys, then, once both streams' last
      // products are done, each stream adds up both O for half of the rows
      const float sum = warp_rows(l, [](float x, float y) { return x + y; });
      if (lane < RP) row_l[w][wq][lane] = sum;
      if (key == 0)
#pragma unroll
        for (int r = 0; r < RP; r += 4)
          *reinterpret_cast<float4*>(&row_m[w][r]) = make_float4(m[r], m[r + 1], m[r + 2], m[r + 3]);
      both_bar();
      const bool two = u1 - u0 > 1;  // both streams had a tile; else that of the piece's first
      await(&pv_done[(t1 - 1) & 1], ((t1 - 1) >> 1) & 1, W8_PV_DONE);
      if (two) await(&pv_done[t1 & 1], ((t1 - 2) >> 1) & 1, W8_PV_DONE);
      tc_fence_after();
      const size_t slot = size_t(blockIdx.x) + seg;
      // (with d = 64 an M = 64 product's rows lie in the first 16 lanes of each warp's 32)
      const int ch = D == 128 ? key : wq * 16 + lane;
      constexpr int RH = RP / 2;
      float w0[RH], w1[RH];
#pragma unroll
      for (int r = 0; r < RH; r += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&row_m[0][w * RH + r]);
        const float4 y = *reinterpret_cast<const float4*>(&row_m[1][w * RH + r]);
        const float m0[4] = {x.x, x.y, x.z, x.w}, m1[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mm = fmaxf(m0[i], m1[i]);
          w0[r + i] = fast_exp2(m0[i] - mm), w1[r + i] = fast_exp2(m1[i] - mm);
        }
      }
      float x[RH] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (two || (t0 & 1) == uint32_t(h)) {
          uint32_t o[4][RH];
          tmem_ld_parts(to + lanes + uint32_t(h * NO + w * RH), RP, o);
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            float y = 0.f;
#pragma unroll
            for (int i = kKv8Parts - 1; i >= 0; --i) y = fmaf(y, 0.03125f, __uint_as_float(o[i][r]));
            x[r] = fmaf(y, h ? w1[r] : w0[r], x[r]);
          }
        }
      if (D == 128 || lane < 16) {
        float* dst = a.opart + (slot * a.R16 + w * RH) * D + ch;
#pragma unroll
        for (int r = 0; r < RH; ++r)
          if (w * RH + r < R) dst[r * D] = x[r];
      }
      if (key < RH && w * RH + key < R) {
        const int row = w * RH + key;
        const float m0 = row_m[0][row], m1 = row_m[1][row], mm = fmaxf(m0, m1);
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) l0 += row_l[0][i][row], l1 += row_l[1][i][row];
        a.ml[slot * a.R16 + row] =
            make_float2(mm, fast_exp2(m0 - mm) * l0 + fast_exp2(m1 - mm) * l1);
      }
      tc_fence_before();
      both_bar();  // (O, the sums and maxima have been read)
      t0 = t1;
      return true;
    });
  } else if (warp == 8) {
    // ------------------------------------------------------------- products
    const uint64_t kd = make_sdesc_rows<D>(smem_u32(base)), vd = make_sdesc_rows<D>(smem_u32(Vs));
    const uint64_t qd = make_sdesc_rows<D>(smem_u32(Qs)), pd = make_sdesc_rows<NO>(smem_u32(Ps));
    constexpr uint32_t ids = make_idesc_e4m3(128, NS, false, false);
    constexpr uint32_t ido = make_idesc_e4m3(D, NO, true, true);
    uint32_t t = 0, np = 0;
    // P V of tile x, its stream's first in the piece or not
    auto pv = [&](uint32_t x, bool first) -> bool {
      const uint32_t b = x & 1, st = x % VS;
      if (!wait(&v_full[st], (x / VS) & 1, W8_V_FULL)) return false;
      if (!wait(&p_full[b], (x >> 1) & 1, W8_P_FULL)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma_e4m3(to + b * NO, vd + ((st * S::kTile + uint32_t(ks) * 32u * D) >> 4),
                    pd + ((b * S::kP + uint32_t(ks) * 32u * NO) >> 4), ido, !first || ks > 0);
        umma_commit(&pv_done[b]);
        umma_commit(&v_free[st]);
      }
      __syncwarp();
      return true;
    };
    kv8_pieces(a, share, [&](int, int, int, int, int u0, int u1) -> bool {
      const uint32_t qb = np & 1, t1 = t + uint32_t(u1 - u0), t0 = t;
      if (!wait(&q_full[qb], (np >> 1) & 1, W8_Q_FULL)) return false;
      for (; t < t1 + 2; ++t) {
        // (S of four tiles before has been read: its P was waited for)
        if (t < t1) {
          const uint32_t st = t % KS;
          if (!wait(&k_full[st], (t / KS) & 1, W8_K_FULL)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
              umma_e4m3(tm + t % SB * NS, kd + ((st * S::kTile + uint32_t(ks) * 32u) >> 4),
                        qd + ((qb * S::kQ + uint32_t(ks) * 32u) >> 4), ids, ks > 0);
            umma_commit(&s_full[t % SB]);
            umma_commit(&k_free[st]);
            if (t + 1 == t1) umma_commit(&q_free[qb]);
          }
          __syncwarp();
        }
        if (t >= t0 + 2 && !pv(t - 2, t - 2 < t0 + 2)) return false;
      }
      t = t1;
      ++np;
      return true;
    });
    // every product and commit is done before the tensor memory is given back
    if (t > 0 && elect_one()) {
      umma_commit(&all_done);
      mbar_wait(&all_done, 0);
    }
  } else if (warp == 9 || warp == 10) {
    // --------------------------------------------------------------- copies
    // (a warp for the keys and the scales, another for the values, which wait longer)
    const bool keys = warp == 9;
    const int page = 1 << a.c.page_log2;
    const int ti = lane >> 3, gr = (lane & 7) * 16;  // this lane's tile of four, its 16 keys
    const uint32_t stages = keys ? KS : VS;
    uint64_t *full = keys ? k_full : v_full, *free = keys ? k_free : v_free;
    uint8_t* ring = keys ? base : Vs;
    const CUtensorMap* map = keys ? &kmap : &vmap;
    uint32_t t = 0, st = 0, round = 0;  // the next tile, its stage and the stage's use
    kv8_pieces(a, share, [&](int n, int g, int, int ctx, int u0, int u1) -> bool {
      const int32_t* table = a.c.table + size_t(n) * a.c.max_pages;
      const int stop = min(ctx, u1 * 128);
      int pos = (u0 + ti) * 128 + gr;
      auto look = [&](int p) { return p < stop ? table[p >> a.c.page_log2] : -1; };
      auto scales = [&](int p, int phys, int& ek, int& ev) {
        ek = ev = 127;
        if (keys && p < stop && phys >= 0 && phys < a.c.n_pages) {
          const size_t at = kv8_scale(a.c, phys, a.Hkv, g, p);
          ek = a.c.ks[at], ev = a.c.vs[at];
        }
      };
      // (the table is read two groups of four tiles ahead, the scales one)
      int phys = look(pos), next = look(pos + 512), ek, ev;
      scales(pos, phys, ek, ev);
      for (int u = u0; u < u1; u += 4, pos += 512) {
        const int after = look(pos + 1024);
        int ek1, ev1;
        scales(pos + 512, next, ek1, ev1);
        const bool on = pos < stop, have = on && phys >= 0 && phys < a.c.n_pages;
        debug_flag(on && !have, DEV_BAD_INDEX);
        const bool head = have && (gr & (page - 1)) == 0;  // this lane copies the page
        const uint32_t heads = __ballot_sync(0xffffffffu, head);
        const int tiles = min(4, u1 - u);
        auto publish = [&](int i) {  // of tile i: its keys and scales
          const uint32_t x = (t + uint32_t(i)) % MB;
          if (ti == i) {
            Kv8Meta mt;
            const int e_k = kv8_exp(uint32_t(ek)), e_v = kv8_exp(uint32_t(ev));
            mt.sk = exp2_int(e_k), mt.ev = float(e_v), mt.iv = exp2_int(-e_v);
            mt.keys = have ? min(16, ctx - pos) : 0;
            meta[x][lane & 7] = mt;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&m_full[x]);
        };
        for (int i = 0; i < tiles; ++i) {
          if (round > 0 && !wait(&free[st], (round - 1) & 1, keys ? W8_K_FREE : W8_V_FREE))
            return false;
          if (lane == 0)
            mbar_arrive_expect_tx(&full[st],
                                  uint32_t(__popc(heads >> (8 * i) & 0xFFu) * page) * D);
          __syncwarp();
          if (head && ti == i)
            tma_load_3d(ring + st * S::kTile + uint32_t(gr) * D, map, &full[st], 0,
                        g << a.c.page_log2, phys);
          if (++st == stages) st = 0, ++round;
          if (keys && u > u0) publish(i);  // (its scales came while the four before were copied)
        }
        if (keys && u == u0)
          for (int i = 0; i < tiles; ++i) publish(i);
        phys = next, next = after, ek = ek1, ev = ev1;
        t += uint32_t(tiles);
      }
      return true;
    });
    // every copy has landed before the CTA may leave (where a wait has run out, nobody
    // else waits for it)
    for (uint32_t i = 0; i < stages; ++i) {
      const uint32_t uses = round + (i < st ? 1 : 0);
      if (uses > 0) mbar_wait(&full[i], (uses - 1) & 1);
    }
  } else {
    // -------------------------------------------------------------- queries
    uint32_t np = 0;
    kv8_pieces(a, share, [&](int n, int g, int, int, int, int) -> bool {
      if (np >= 1) {
        const uint32_t qb = np & 1;
        constexpr int P = Kv8Query<D>::passes(RP);
        Kv8Query<D> x[P];
#pragma unroll
        for (int p = 0; p < P; ++p) x[p].load(a, n, g, p, lane);
        if (np >= 2 && !wait(&q_free[qb], ((np >> 1) - 1) & 1, W8_Q_FREE)) return false;
        stage_queries<D, RP, P>(x, 0, lane, a.scale, Qs + qb * S::kQ, row_f[qb]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[qb]);
      }
      ++np;
      return true;
    });
  }
  __syncthreads();
  if (threadIdx.x == 0 && failed)
    record_error(err, DEV_TIMEOUT_MMA | DEV_K_KV8_ROWS | (failed << 16));
  tmem_teardown(tm, S::kCols);
}

// ------------------------------------------------------------------- host

template <int D, int RP>
static cudaError_t launch_rows(const Kv8AttnArgs& a, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, uint32_t* err, cudaStream_t st) {
  constexpr size_t smem = Kv8Rows<D, RP>::kSmem;
  HERALD_CHECK_LAUNCH(ensure_smem(kv8_rows_kernel<D, RP>, smem));
  return launch_k("kv8_rows_kernel", kv8_rows_kernel<D, RP>, dim3(unsigned(a.ctas)),
                  dim3(kKv8RowsThreads), smem, st, a, kmap, vmap, err);
}
cudaError_t launch_kv8_rows(int d, int rows, const Kv8AttnArgs& a, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, uint32_t* err, cudaStream_t st) {
  if (d == 128)
    return rows <= 8    ? launch_rows<128, 8>(a, kmap, vmap, err, st)
                        : launch_rows<128, 16>(a, kmap, vmap, err, st);
  return rows <= 8    ? launch_rows<64, 8>(a, kmap, vmap, err, st)
                      : launch_rows<64, 16>(a, kmap, vmap, err, st);
}

HERALD_DEBUG_WORD_READER(debug_take_kv8_rows)

}  // namespace herald
