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
//   p = p0 + p1/16 + p2/256 + p3/4096 (kKv8Parts), with p at most 2^8
// and the columns are added in fp32 afterwards.  A key's scale (its block's) multiplies its
// scores.  A value's exponent e_v goes into the weight's own, p = 2^(x + e_v - m), and
// out of the row's sum again, l += p 2^-e_v: O has one unit, and weights keep their bits
// whatever their values' scales.
//
// One CTA per SM walks its share of the keys (kv4_split):
//   warps 0-3  softmax, a thread per key of the tile (its TMEM lane), rows in registers;
//              each keeps the sum of its own keys' weights
//   warp 4     the issuer of both products, S a tile ahead of P V
//   warp 5     copies tiles into a ring and looks up pages and scales, four tiles of
//              page table and scales (32 lanes: 8 groups of 16 keys each) ahead
//   warp 6     stages the queries of the next piece
// A row's exponent base m is set 4 below its largest exponent and stays while no p passes
// 2^8; all four warps vote on that in one barrier a tile.  Else the tile's row maxima are
// exchanged, O is scaled once the products before it are done, and l follows.
#include <float.h>

#include "kv8.cuh"
#include "tc_common.cuh"

namespace herald {

constexpr int kKv8Parts = 4;               // e4m3 numbers of a weight
constexpr float kKv8At = 4.f, kKv8Most = 8.f;  // log2 p of a new base's row, and the largest
constexpr int kKv8RowsThreads = 224;       // 7 warps

// Waits of the kernel (bits 16-31 of the error word).
enum : uint32_t {
  W8_STAGE_FREE = 1, W8_STAGE_FULL = 2, W8_Q_FREE = 4, W8_Q_FULL = 8, W8_S_FULL = 0x10,
  W8_P_FULL = 0x20, W8_PV_DONE = 0x40
};

template <int D, int RP>
struct Kv8Rows {
  static constexpr int kNs = 2 * RP;                // columns of S: q0 rows, q1 rows
  static constexpr int kNo = kKv8Parts * RP;        // columns of O, bytes of a key's P
  static constexpr uint32_t kTile = 128u * D;       // bytes of 128 keys
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr int kStages = D == 64 ? 8 : RP == 32 ? 5 : 6;
  static constexpr uint32_t kQ = uint32_t(kNs) * D, kP = 128u * kNo;
  static constexpr uint32_t kSmem = kStages * kStage + 2 * kQ + 2 * kP + 1024;
  static constexpr uint32_t kCols = RP == 8 ? 64 : RP == 16 ? 128 : 256;  // 2 S + O
};

// What the softmax needs of 16 keys: 2^e_k, e_v, 2^-e_v and how many of them count.
struct __align__(16) Kv8Meta {
  float sk, ev, iv;
  int keys;
};

// x -> 16 (x - e4m3(x)) for a pair, returning the codes: what the next number holds.
HERALD_DEV uint32_t split_e4m3(float& a, float& b) {
  const uint32_t w = float2_to_e4m3(a, b);
  const uint32_t h = e4m3x2_to_half2(w);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  a = fmaf(f.x, -16.f, a * 16.f);
  b = fmaf(f.y, -16.f, b * 16.f);
  return w;
}

HERALD_DEV bool soft_any(bool x) {  // any of the softmax threads
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(x))
      : "memory");
  return r != 0;
}
HERALD_DEV void soft_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

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

template <int D, int RP>
__global__ void __launch_bounds__(kKv8RowsThreads, 1)
    kv8_rows_kernel(const Kv8AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, uint32_t* err) {
  using S = Kv8Rows<D, RP>;
  constexpr int NS = S::kNs, NO = S::kNo, ST = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[ST], empty[ST], q_full[2], q_free[2], s_full[2], p_full[2], pv_done[2],
      all_done;
  __shared__ uint32_t tmem_base, failed;
  __shared__ Kv8Share share;
  __shared__ Kv8Meta meta[ST][8];
  __shared__ __align__(16) float row_f[2][RP];  // score factors of the rows
  __shared__ float red[4][RP];
  uint8_t* base = align1024(smem_raw);
  uint8_t *Qs = base + ST * S::kStage, *Ps = Qs + 2 * S::kQ;
  const int warp = warp_same(int(threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&full[i], 2), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(&q_full[i], 1), mbar_init(&q_free[i], 5), mbar_init(&s_full[i], 1),
          mbar_init(&p_full[i], 128), mbar_init(&pv_done[i], 1);
    mbar_init(&all_done, 1);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 5 && lane == 0) tma_prefetch_desc(&kmap), tma_prefetch_desc(&vmap);
  tmem_setup(&tmem_base, S::kCols);
  const uint32_t tm = tmem_base, to = tm + 2 * NS;
  griddep_enter();
  const Kv4Wait wait{&failed};
  const int G = a.Hq / a.Hkv, R = a.B * G;
  if (warp == 0) {
    const Kv8Share mine = kv8_share(a, int(blockIdx.x));
    if (lane == 0) share = mine;
  }
  __syncthreads();

  if (warp < 4) {
    // ------------------------------------------------------------ softmax
    // (after a failed wait these warps go on without waiting: the barriers among them
    // stay in step, the results are worthless and the error is recorded)
    bool lost = false;
    auto await = [&](uint64_t* bar, uint32_t parity, uint32_t which) {
      if (!lost) lost = !wait(bar, parity, which);
    };
    const int key = int(threadIdx.x);
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    uint32_t t = 0, np = 0;  // tiles and pieces of the CTA
    kv8_pieces(a, share, [&](int n, int, int seg, int ctx, int u0, int u1) -> bool {
      debug_flag(threadIdx.x == 0 && a.ctx[n] != ctx, DEV_BAD_COUNT);
      const uint32_t qb = np & 1;
      await(&q_full[qb], (np >> 1) & 1, W8_Q_FULL);
      constexpr bool kKeepF = RP < 32;  // (32 factors in registers would spill)
      float f[kKeepF ? RP : 1] = {}, m[RP], l[RP];
      if constexpr (kKeepF) {
#pragma unroll
        for (int r = 0; r < RP; r += 4) {
          const float4 x = *reinterpret_cast<const float4*>(&row_f[qb][r]);
          f[r] = x.x, f[r + 1] = x.y, f[r + 2] = x.z, f[r + 3] = x.w;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_free[qb]);
      }
      auto factor = [&](int r) { return kKeepF ? f[kKeepF ? r : 0] : *(volatile float*)&row_f[qb][r]; };
      ++np;
#pragma unroll
      for (int r = 0; r < RP; ++r) m[r] = -FLT_MAX, l[r] = 0.f;
#pragma unroll 1
      for (int u = u0; u < u1; ++u, ++t) {
        const uint32_t b = t & 1, st = t % ST;
        await(&full[st], (t / ST) & 1, W8_STAGE_FULL);  // (the meta data and V are here)
        await(&s_full[b], (t >> 1) & 1, W8_S_FULL);
        tc_fence_after();
        const Kv8Meta mt = meta[st][key >> 4];
        const bool on = (key & 15) < mt.keys;
        float s[RP], p[RP];
        {
          float x[NS];
          tmem_load<NS>(tm + lanes + b * NS, x);
#pragma unroll
          for (int r = 0; r < RP; ++r) s[r] = fmaf(x[RP + r], 0.0625f, x[r]);
        }
        bool move = false;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          p[r] = on ? fmaf(s[r], factor(r) * mt.sk, mt.ev - m[r]) : -INFINITY;
          move |= p[r] > kKv8Most;
        }
        if (soft_any(move)) {
          // row maxima of the tile, rounded down: where scores are so large that fp32's
          // steps are no longer small, a base above them all would leave no weight
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const float z = __fadd_rd(__fmul_rd(s[r], factor(r) * mt.sk), mt.ev);
            const float mx = warp_max(on ? z : -INFINITY);
            if (lane == 0) red[warp][r] = mx;
          }
          soft_bar();
          float k[RP];
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const float z = fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r]));
            const float m1 = fmaxf(__fadd_rd(z, -kKv8At), m[r]);
            k[r] = fast_exp2(m[r] - m1);
            m[r] = m1;
            l[r] *= k[r];
            const float x = fmaf(s[r], factor(r) * mt.sk, mt.ev - m1);
            p[r] = !on ? -INFINITY : x > kKv8Most ? kKv8Most : x;  // (a NaN stays)
          }
          if (u > u0) {  // O so far, once the products before this tile are in it
            await(&pv_done[b ^ 1], ((t - 1) >> 1) & 1, W8_PV_DONE);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < NO; c += 32) {
              float o[32];
              tmem_ld32(to + lanes + uint32_t(c), o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= k[(c + i) % RP];
              tmem_st32(to + lanes + uint32_t(c), o);
            }
            tmem_wait_st();
          }
          soft_bar();  // (the maxima have been read)
        }
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          p[r] = fast_exp2(p[r]);
          l[r] = fmaf(p[r], mt.iv, l[r]);
        }
        // P of two tiles before has been read
        if (t >= 2) await(&pv_done[b], ((t >> 1) - 1) & 1, W8_PV_DONE);
        uint8_t* dst = Ps + b * S::kP;
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
        if (!on) {  // such a row may hold any bytes: 0 * NaN must not arise
          uint4* v = reinterpret_cast<uint4*>(base + st * S::kStage + S::kTile + uint32_t(key) * D);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) v[c] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&p_full[b]);
      }
      if constexpr (!kKeepF) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_free[qb]);
      }
      // the piece's partials: O once the last product is done, l over all keys
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        l[r] = warp_sum(l[r]);
        if (lane == 0) red[warp][r] = l[r];
      }
      soft_bar();
      const size_t slot = size_t(blockIdx.x) + seg;
#pragma unroll
      for (int r = 0; r < RP; ++r)
        if (key == r && r < R)
          a.ml[slot * a.R16 + r] = make_float2(m[r], red[0][r] + red[1][r] + red[2][r] + red[3][r]);
      await(&pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1, W8_PV_DONE);
      tc_fence_after();
      // (with d = 64 an M = 64 product's rows lie in the first 16 lanes of each warp's 32)
      const int ch = D == 128 ? key : warp * 16 + lane;
      float* out = a.opart + slot * a.R16 * D + ch;
      float o[NO];
      tmem_load<NO>(to + lanes, o);
      if (D == 128 || lane < 16) {
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          float x = o[(kKv8Parts - 1) * RP + r];
#pragma unroll
          for (int i = kKv8Parts - 2; i >= 0; --i) x = fmaf(x, 0.0625f, o[i * RP + r]);
          if (r < R) out[r * D] = x;
        }
      }
      tc_fence_before();
      soft_bar();  // (the sums have been read)
      return true;
    });
  } else if (warp == 4) {
    // ------------------------------------------------------------- products
    const uint64_t kd = make_sdesc_rows<D>(smem_u32(base)), vd = kd + (S::kTile >> 4);
    const uint64_t qd = make_sdesc_rows<D>(smem_u32(Qs)), pd = make_sdesc_rows<NO>(smem_u32(Ps));
    constexpr uint32_t ids = make_idesc_e4m3(128, NS, false, false);
    constexpr uint32_t ido = make_idesc_e4m3(D, NO, true, true);
    uint32_t t = 0, np = 0;
    // P V of tile x, the first of its piece or not
    auto pv = [&](uint32_t x, bool first) -> bool {
      const uint32_t b = x & 1, st = x % ST;
      if (!wait(&p_full[b], (x >> 1) & 1, W8_P_FULL)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma_e4m3(to, vd + ((st * S::kStage + uint32_t(ks) * 32u * D) >> 4),
                    pd + ((b * S::kP + uint32_t(ks) * 32u * NO) >> 4), ido, !first || ks > 0);
        umma_commit(&pv_done[b]);
        umma_commit(&empty[st]);
      }
      __syncwarp();
      return true;
    };
    kv8_pieces(a, share, [&](int, int, int, int, int u0, int u1) -> bool {
      const uint32_t qb = np & 1;
      if (!wait(&q_full[qb], (np >> 1) & 1, W8_Q_FULL)) return false;
      for (int u = u0; u < u1; ++u, ++t) {
        // (S of two tiles before has been read: its P was waited for)
        const uint32_t st = t % ST;
        if (!wait(&full[st], (t / ST) & 1, W8_STAGE_FULL)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 32; ++ks)
            umma_e4m3(tm + (t & 1) * NS, kd + ((st * S::kStage + uint32_t(ks) * 32u) >> 4),
                      qd + ((qb * S::kQ + uint32_t(ks) * 32u) >> 4), ids, ks > 0);
          umma_commit(&s_full[t & 1]);
          if (u + 1 == u1) umma_commit(&q_free[qb]);
        }
        __syncwarp();
        if (u > u0 && !pv(t - 1, u == u0 + 1)) return false;
      }
      if (!pv(t - 1, u1 == u0 + 1)) return false;
      ++np;
      return true;
    });
    // every product and commit is done before the tensor memory is given back
    if (t > 0 && elect_one()) {
      umma_commit(&all_done);
      mbar_wait(&all_done, 0);
    }
  } else if (warp == 5) {
    // --------------------------------------------------------------- copies
    const int page = 1 << a.c.page_log2;
    const int ti = lane >> 3, gr = (lane & 7) * 16;  // this lane's tile of four, its 16 keys
    uint32_t t = 0, issued = 0;
    kv8_pieces(a, share, [&](int n, int g, int, int ctx, int u0, int u1) -> bool {
      const int32_t* table = a.c.table + size_t(n) * a.c.max_pages;
      const int stop = min(ctx, u1 * 128);
      int pos = (u0 + ti) * 128 + gr;
      auto look = [&](int p) { return p < stop ? table[p >> a.c.page_log2] : -1; };
      auto scales = [&](int p, int phys, int& ek, int& ev) {
        ek = ev = 127;
        if (p < stop && phys >= 0 && phys < a.c.n_pages) {
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
          const uint32_t x = (t + uint32_t(i)) % ST;
          if (ti == i) {
            Kv8Meta mt;
            const int e_k = kv8_exp(uint32_t(ek)), e_v = kv8_exp(uint32_t(ev));
            mt.sk = exp2_int(e_k), mt.ev = float(e_v), mt.iv = exp2_int(-e_v);
            mt.keys = have ? min(16, ctx - pos) : 0;
            meta[x][lane & 7] = mt;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[x]);
        };
        for (int i = 0; i < tiles; ++i) {
          const uint32_t x = t + uint32_t(i), st = x % ST;
          if (x >= uint32_t(ST) && !wait(&empty[st], (x / ST - 1) & 1, W8_STAGE_FREE)) return false;
          issued = x + 1;
          if (lane == 0)
            mbar_arrive_expect_tx(&full[st],
                                  uint32_t(__popc(heads >> (8 * i) & 0xFFu) * page) * (2u * D));
          __syncwarp();
          if (head && ti == i) {
            uint8_t* dst = base + st * S::kStage + uint32_t(gr) * D;
            tma_load_3d(dst, &kmap, &full[st], 0, g << a.c.page_log2, phys);
            tma_load_3d(dst + S::kTile, &vmap, &full[st], 0, g << a.c.page_log2, phys);
          }
          if (u > u0) publish(i);  // (its scales came while the four before were copied)
        }
        if (u == u0)
          for (int i = 0; i < tiles; ++i) publish(i);
        phys = next, next = after, ek = ek1, ev = ev1;
        t += uint32_t(tiles);
      }
      return true;
    });
    // every copy has landed before the CTA may leave (where a wait has run out, nobody
    // else waits for it)
    for (uint32_t i = issued > uint32_t(ST) ? issued - ST : 0; i < issued; ++i)
      mbar_wait(&full[i % ST], (i / ST) & 1);
  } else {
    // -------------------------------------------------------------- queries
    constexpr int LPR = D / 8, RPP = 32 / LPR, P = RP / RPP;
    const int c = lane % LPR, sub = lane / LPR;
    uint32_t np = 0;
    kv8_pieces(a, share, [&](int n, int g, int, int, int, int) -> bool {
      const uint32_t qb = np & 1;
      uint4 x[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int r = p * RPP + sub;
        x[p] = make_uint4(0, 0, 0, 0);
        if (r < R)
          x[p] = *reinterpret_cast<const uint4*>(
              a.q + ((size_t(n) * a.B + r / G) * a.Hq + g * G + r % G) * D + c * 8);
      }
      if (np >= 2 && !wait(&q_free[qb], ((np >> 1) - 1) & 1, W8_Q_FREE)) return false;
      float mx[P];  // (the rows' maxima side by side: their steps wait on one another)
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t m = max_bf16x2_abs(
            max_bf16x2_abs(max_bf16x2_abs(max_bf16x2_abs(0, x[p].x), x[p].y), x[p].z), x[p].w);
        mx[p] = fmaxf(bf16lo(m), bf16hi(m));
      }
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
        for (int p = 0; p < P; ++p) mx[p] = fmaxf(mx[p], __shfl_xor_sync(0xffffffffu, mx[p], o));
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t r = uint32_t(p * RPP + sub), half = uint32_t(c & 1) * 8u;
        float up, f;
        kv8_query_scale(mx[p], a.scale, &up, &f);
        const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
        uint32_t v0[4], v1[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t h = pack_half2(bf16lo(w[i]) * up, bf16hi(w[i]) * up);
          v0[i] = half2_to_e4m3(h);
          const uint32_t rest = hsub2(h, e4m3x2_to_half2(v0[i]));  // what q0 left, times 16
          v1[i] = half2_to_e4m3(hmul2(rest, 0x4C004C00u));
        }
        uint8_t* dst = Qs + qb * S::kQ;
        *reinterpret_cast<uint2*>(dst + rows_off<D>(r, uint32_t(c >> 1)) + half) =
            make_uint2(v0[0] | v0[1] << 16, v0[2] | v0[3] << 16);
        *reinterpret_cast<uint2*>(dst + rows_off<D>(uint32_t(RP) + r, uint32_t(c >> 1)) + half) =
            make_uint2(v1[0] | v1[1] << 16, v1[2] | v1[3] << 16);
        if (c == 0) row_f[qb][r] = f;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[qb]);
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
           : rows <= 16 ? launch_rows<128, 16>(a, kmap, vmap, err, st)
                        : launch_rows<128, 32>(a, kmap, vmap, err, st);
  return rows <= 8    ? launch_rows<64, 8>(a, kmap, vmap, err, st)
         : rows <= 16 ? launch_rows<64, 16>(a, kmap, vmap, err, st)
                      : launch_rows<64, 32>(a, kmap, vmap, err, st);
}

HERALD_DEBUG_WORD_READER(debug_take_kv8_rows)

}  // namespace herald
