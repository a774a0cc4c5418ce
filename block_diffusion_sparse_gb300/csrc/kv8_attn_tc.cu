// kv8_attn_tc.cu -- attention over the paged 8-bit cache on the 5th-generation tensor
// cores for blocks of queries (many rows per KV head).
//
// A CTA takes 128 query rows of a KV head (a row tile) and walks its share of the keys
// in tiles of 128:
//   S [128 rows x 128 keys] = Q K^T    kind::f8f6f4: K's codes as they are held, Q in
//                                      tensor memory as two e4m3 numbers a value, q0 +
//                                      q1 (a bf16 has 8 bits, e4m3 4), one product each
//   O [128 rows x d]       += P V      kind::f16: P fp16 in tensor memory, V's codes
//                                      turned into fp16 (exact)
// (P as e4m3 numbers, V as it is held, would take no conversion of V, 450 warp
// instructions a tile, but splitting 128 x 128 weights takes some 1500 more than
// packing them.)  Q in tensor memory keeps 64 KB a tile off shared memory, whose
// bandwidth would be the bound: 144 KB a tile as it is (copies 32, K twice 32, V read
// 16, written 32 and read as fp16 32).
//   warps 0-3, 4-7  softmax: two streams, a thread per row each, the first with the
//              first 64 keys of every tile, the second with the others; each has its own
//              base m, sum l and O, added up at a piece's end
//   warps 8-11 turn V tiles into fp16
//   warp 12    copies K and V tiles by TMA, looks up pages and scales four tiles ahead
//   warps 13, 14  issue S and P V, one per stream, in steps of 64 keys (warp 15 idles: registers
//              are dealt by four warps)
// Tensor memory holds, for each stream, one step's scores (64 columns), its P (32) and O
// (128), and Q (64): 512.  A step's scores are in registers before anything is done
// with them, so the next step's product runs beside its softmax.  (With P over the
// scores and three such buffers for both streams, each step waited for the product
// before it: 1,800 cycles a tile.)
// Scales: a key's multiplies its scores.  A value's exponent e_v goes into the weight's
// own, P = 2^(x + e_v - m), and out of the row's sum again, l += P 2^-e_v, so O has one
// unit and P fills fp16 whatever the values' scales.  fp16 ends at 2^-24, where a row's largest
// P is 2^5 at least: keys 2^-30 and less below it (values of so small a scale, or
// weights) count in the sum only.
//
// P = 2^(x + e_v - m) stays in fp16 as long as a step's 64 of them sum to less than
// 60000.  Where a sum does not (and at a piece's first step) the row's largest exponent
// is looked up, m set 5 below it, O and l follow, and the step is done again.
//
// fp16 rounds a weight by at most 2^-11 of it.  That shows in an output's last bf16 place now
// and then (block over 32K: 8e-4 of the outputs' norm beside the same in fp32) and not beside
// the output's own rounding (1.7e-3 from the exact values either way).  A second number a weight
// would take half as many products again and columns of tensor memory that d = 128 lacks.
//
// What bounds it: the dependent steps of a stream's warp, some 1,950 cycles a tile (scores
// from tensor memory 400, exponentials and packing 950, waiting for products 250, P to tensor
// memory 350); the tensor pipe is active 53% and DRAM 62% of the time.  Four blocks of 32 over
// 64K tokens each, 32 heads over 8: 109 us for 539 MB; one over 32K, 28 heads over 4, 24.9 us,
// half of it phases that do not grow with the keys (share 0.8 us, queries 2.6, first scores 0.6,
// partials 1.5, join 3).  S and P V from one warp a stream, so that a stream waits once a step:
// 25.2 to 24.9 us for the latter.
#include <float.h>

#include "kv8.cuh"
#include "tc_common.cuh"

namespace herald {

constexpr int kKv8TcThreads = 512;  // 16 warps
constexpr int kKv8KStages = 4, kKv8VStages = 4;
// Scales and counts of tiles, published by groups of four (fewer at a piece's end) with a
// barrier each.  The last copied tile t has S(t - 4) done, for which the scores of
// t - 5 had to be read, whose scales may still be wanted: six groups at most, of one
// tile each.
constexpr int kKv8Groups = 8;
constexpr float kKv8Below = 5.f, kKv8Top = 60000.f, kKv8TopLog2 = 15.8f;

// Waits of the kernel (bits 16-31 of the error word).
enum : uint32_t {
  X8_K_FREE = 1, X8_V_FREE = 2, X8_K_FULL = 4, X8_V_FULL = 8, X8_META = 0x10, X8_Q_FULL = 0x20,
  X8_S_FULL = 0x40, X8_P_FULL = 0x80, X8_S_READ = 0x100, X8_V16_FREE = 0x200,
  X8_V16_FULL = 0x400, X8_O_DONE = 0x800
};

struct Kv8TileMeta {  // per 16 keys: 2^e_k, e_v, 2^-e_v and how many count
  float sk[8], ev[8], iv[8];
  uint32_t keys[8];
  uint32_t whole[4];  // [0]: all of them count
};

template <int D>
struct Kv8Tc {
  static constexpr uint32_t kTile = 128u * D;          // bytes of 128 keys as held
  static constexpr uint32_t kTile16 = uint32_t(D / 64) * 16384u;  // as fp16
  static constexpr uint32_t kV = kKv8KStages * kTile, kV16 = kV + kKv8VStages * kTile;
  static constexpr uint32_t kX = kV16 + 2 * kTile16;  // 2 KB for each softmax warp's queries
  static constexpr uint32_t kSmem = kX + 8 * 2048 + 1024;
};
// Tensor memory: both streams' scores, P, then q0, q1, both streams' O.
constexpr uint32_t kKv8TmP = 128, kKv8TmQ0 = 192, kKv8TmQ1 = 224, kKv8TmO = 256;

HERALD_DEV void umma_e4m3_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// fp16 A and B (make_idesc_bf16 with formats 0)
__host__ __device__ constexpr uint32_t make_idesc_half(int M, int N, bool b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}
HERALD_DEV void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for this thread's tensor-memory loads; r (loaded before) counts as written
// here, so that no use of it moves above the wait.
HERALD_DEV void tmem_ld_done(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
                 "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
                 "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                 "+r"(r[31])
               :
               : "memory");
}
HERALD_DEV void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
HERALD_DEV void tmem_ld16_done(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
                 "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
HERALD_DEV void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

// 16 scores -> P (fp16 pairs) and their sum; two values an instruction.
HERALD_DEV float exp16(const uint32_t* x, float f, float nm, uint32_t* pk) {
  const uint64_t f2 = f2_pack(f, f), nm2 = f2_pack(nm, nm);
  uint64_t sa = f2_pack(0.f, 0.f), sb = sa;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float t0, t1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), f2, nm2), t0, t1);
    const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
    if (i & 2)
      sa = f2_add(sa, f2_pack(p0, p1));
    else
      sb = f2_add(sb, f2_pack(p0, p1));
    pk[i / 2] = pack_half2(p0, p1);
  }
  float s0, s1;
  f2_unpack(f2_add(sa, sb), s0, s1);
  return s0 + s1;
}

HERALD_DEV void tc_bar() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kKv8TcThreads, 1)
    kv8_attn_tc_kernel(const Kv8AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, uint32_t* err) {
  using S = Kv8Tc<D>;
  constexpr int KS = kKv8KStages, VS = kKv8VStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t k_full[KS], k_free[KS], v_full[VS], v_free[VS], v16_full[2], v16_free[2],
      meta_full[kKv8Groups], q_full, s_full[2], s_read[2], p_full[2], o_done[2], all_done[2];
  __shared__ uint32_t tmem_base, failed;
  __shared__ Kv8Share share;
  __shared__ __align__(16) Kv8TileMeta meta[kKv8Groups][4];
  __shared__ float2 row_ml[2][128];  // a piece's (m, l) of both streams
  __shared__ float row_f[128];       // score factors of its rows
  uint8_t* base = align1024(smem_raw);
  const int warp = warp_same(int(threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) mbar_init(&k_full[i], 1), mbar_init(&k_free[i], 2);
    for (int i = 0; i < VS; ++i) mbar_init(&v_full[i], 1), mbar_init(&v_free[i], 4);
    for (int i = 0; i < kKv8Groups; ++i) mbar_init(&meta_full[i], 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(&v16_full[i], 4), mbar_init(&v16_free[i], 2), mbar_init(&o_done[i], 1),
          mbar_init(&s_full[i], 1), mbar_init(&s_read[i], 4), mbar_init(&p_full[i], 4);
    for (int i = 0; i < 2; ++i) mbar_init(&all_done[i], 1);
    mbar_init(&q_full, 8);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 12 && lane == 0) tma_prefetch_desc(&kmap), tma_prefetch_desc(&vmap);
  tmem_setup(&tmem_base, 512);
  const uint32_t tm = tmem_base;
  griddep_enter();
  const Kv4Wait wait{&failed};
  // (through shared memory: values that all roles hold from here on would be spilled for
  // the role with the fewest registers)
  if (warp == 0) {
    const Kv8Share mine = kv8_share(a, int(blockIdx.x));
    if (lane == 0) share = mine;
  }
  __syncthreads();

  // registers: 512 threads launch with 128 each (65,536) = 128 x (2 x 200 + 64 + 48).  Each
  // role's branch begins with its own setmaxnreg, so that the compiler knows the limit
  // of the code that follows.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ------------------------------------------------------------ softmax
    // (after a failed wait these warps go on without waiting: the barriers among them
    // stay in step, the results are worthless and the error is recorded)
    bool lost = false;
    auto await = [&](uint64_t* bar, uint32_t parity, uint32_t which) {
      if (!lost) lost = !wait(bar, parity, which);
    };
    const int w = warp >> 2, lrow = (warp & 3) * 32 + lane;  // stream, TMEM lane
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t ts = tm + lanes + uint32_t(w) * 64u, tp = tm + lanes + kKv8TmP + uint32_t(w) * 32u;
    const uint32_t to = tm + lanes + kKv8TmO + uint32_t(w) * 128u, to2 = to ^ 128u;  // O, the other's
    uint8_t* xb = base + S::kX + warp * 2048;
    const int G = a.Hq / a.Hkv, R = a.B * G;
    const int per_g = 65536 / G + 1;  // r / G = r per_g / 2^16 for the rows r < 256
    uint32_t t = 0, mg = 0;  // tiles and groups of them
    kv8_pieces(a, share, [&](int n, int gt, int seg, int ctx, int u0, int u1) -> bool {
      debug_flag(threadIdx.x == 0 && a.ctx[n] != ctx, DEV_BAD_COUNT);
      const int g = gt / a.row_tiles, r0 = (gt - g * a.row_tiles) * 128;
      const bool idle = r0 + (warp & 3) * 32 >= R;  // the warp has no rows
      const int row = r0 + lrow;
      // queries: of a quarter's 32 rows each stream's warp turns 16 into q0 and q1, D/8
      // lanes a row and 8 rows at a time, and through shared memory the first stream's
      // lanes take q0 of their rows, the other's q1.  (A lane loading its row by itself
      // touched 32 lines an instruction: 6 us until the first scores.)  The scores of the
      // piece before have been read: nothing reads Q now.
      constexpr int LPR = D / 8, RPP = 32 / LPR, P = 8 / RPP, W = D / 4;
      const int c = lane % LPR, sub = lane / LPR, q_row = r0 + (warp & 3) * 32 + w * 16 + sub;
      const uint16_t* q0 = a.q + (size_t(n) * a.B * a.Hq + g * G) * D + c * 8;
      uint4 next[P];
      auto load_q = [&](int h) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int r = min(q_row + h * 8 + p * RPP, R - 1), tok = r * per_g >> 16;  // r / G
          next[p] = *reinterpret_cast<const uint4*>(q0 + (r + tok * (a.Hq - G)) * D);
        }
      };
      if (!idle) load_q(0);
      uint32_t o[W];  // this lane's row of q0 or q1
      // (a loop kept rolled: unrolled it crowds the registers of the whole role)
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (!idle) {
          uint4 x[P];
#pragma unroll
          for (int p = 0; p < P; ++p) x[p] = next[p];
          if (h == 0) load_q(1);
          float mx[P];  // (the rows' maxima side by side: their steps wait on one another)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const uint32_t m4 = max_bf16x2_abs(
                max_bf16x2_abs(max_bf16x2_abs(max_bf16x2_abs(0, x[p].x), x[p].y), x[p].z), x[p].w);
            mx[p] = fmaxf(bf16lo(m4), bf16hi(m4));
          }
#pragma unroll
          for (int i = 1; i < LPR; i <<= 1)
#pragma unroll
            for (int p = 0; p < P; ++p)
              mx[p] = fmaxf(mx[p], __shfl_xor_sync(0xffffffffu, mx[p], i));
#pragma unroll
          for (int p = 0; p < P; ++p) {
            float up, fp;
            kv8_query_scale(mx[p], a.scale, &up, &fp);
            const uint32_t wd[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
            uint32_t v0[4], v1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t h2 = pack_half2(bf16lo(wd[i]) * up, bf16hi(wd[i]) * up);
              v0[i] = half2_to_e4m3(h2);
              v1[i] = half2_to_e4m3(hsub2(h2, e4m3x2_to_half2(v0[i])));  // what q0 left
            }
            const uint32_t r = uint32_t(p * RPP + sub);
            uint8_t* dst = xb + r * D + ((uint32_t(c >> 1) ^ (r & (D / 16 - 1))) << 4) + (c & 1) * 8;
            *reinterpret_cast<uint2*>(dst) = make_uint2(v0[0] | v0[1] << 16, v0[2] | v0[3] << 16);
            *reinterpret_cast<uint2*>(dst + 8 * D) = make_uint2(v1[0] | v1[1] << 16, v1[2] | v1[3] << 16);
            if (c == 0) row_f[(warp & 3) * 32 + w * 16 + h * 8 + int(r)] = fp;
          }
        }
        tc_bar();
        if (!idle && (lane >> 3 & 1) == h) {
          const uint32_t r = uint32_t(lane) & 7u;
          const uint8_t* src = base + S::kX + ((lane >> 4) * 4 + (warp & 3)) * 2048 + w * (8 * D) + r * D;
#pragma unroll
          for (int i = 0; i < W / 4; ++i) {
            const uint4 y = *reinterpret_cast<const uint4*>(src + ((uint32_t(i) ^ (r & (D / 16 - 1))) << 4));
            o[4 * i] = y.x, o[4 * i + 1] = y.y, o[4 * i + 2] = y.z, o[4 * i + 3] = y.w;
          }
        }
        tc_bar();
      }
      float f = 0.f;
      if (!idle) {
        f = row_f[lrow];
#pragma unroll
        for (int i = 0; i < W; i += 8)
          tmem_st8(tm + lanes + (w ? kKv8TmQ1 : kKv8TmQ0) + uint32_t(i),
                   *reinterpret_cast<uint32_t(*)[8]>(o + i));
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);

      float m = -FLT_MAX, l = 0.f;
      uint32_t x[64];
      // the next scores into registers, and that they have been read
      auto begin_load = [&] {
        if (!idle) {
          tmem_ld32_async(ts, *reinterpret_cast<uint32_t(*)[32]>(x));
          tmem_ld32_async(ts + 32u, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
        }
      };
      auto end_load = [&] {
        tmem_ld_done(*reinterpret_cast<uint32_t(*)[32]>(x));
        tmem_ld_done(*reinterpret_cast<uint32_t(*)[32]>(x + 32));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_read[w]);
      };
      await(&s_full[w], t & 1, X8_S_FULL);
      tc_fence_after();
      begin_load();
      end_load();
#pragma unroll 1
      for (int u = u0; u < u1; ++u, ++t) {
        if ((u - u0) % 4 == 0 && u > u0) ++mg;
        if ((u - u0) % 4 == 0) await(&meta_full[mg % kKv8Groups], (mg / kKv8Groups) & 1, X8_META);
        const Kv8TileMeta& mt = meta[mg % kKv8Groups][(u - u0) % 4];
        uint32_t pk[32];
        float k = 1.f;
        bool moved = false;
        if (!idle) {
          const float4 a4 = *reinterpret_cast<const float4*>(&mt.sk[4 * w]);
          const float4 b4 = *reinterpret_cast<const float4*>(&mt.ev[4 * w]);
          const float4 c4 = *reinterpret_cast<const float4*>(&mt.iv[4 * w]);
          if (!mt.whole[0]) {  // keys that do not count
            const uint4 k4 = *reinterpret_cast<const uint4*>(&mt.keys[4 * w]);
            const uint32_t keys[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (uint32_t(i & 15) >= keys[i / 16]) x[i] = 0xFF800000u;  // -inf
          }
          float fk[4], ev[4], iv[4];  // P = 2^(score fk + ev - m)
          {
            fk[0] = kv8_score_factor(f, a4.x), fk[1] = kv8_score_factor(f, a4.y);
            fk[2] = kv8_score_factor(f, a4.z), fk[3] = kv8_score_factor(f, a4.w);
            ev[0] = b4.x, ev[1] = b4.y, ev[2] = b4.z, ev[3] = b4.w;
            iv[0] = c4.x, iv[1] = c4.y, iv[2] = c4.z, iv[3] = c4.w;
          }
          float add;
          float base = m;
          while (true) {
            add = 0.f;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float s = exp16(x + 16 * c, fk[c], ev[c] - base, pk + 8 * c);
              sum += s;
              add = fmaf(s, iv[c], add);
            }
            const bool high = u == u0 || !(sum <= kKv8Top);  // (a piece's first step has no base)
            if (moved || !__any_sync(0xffffffffu, high)) break;
            moved = true;
            // the largest exponent, rounded down: scores may be so large that fp32's steps
            // are no longer small
            float z = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float mx = -INFINITY;
#pragma unroll
              for (int i = 16 * c; i < 16 * c + 16; i += 2)
                mx = fmax3f(mx, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
              z = fmaxf(z, __fadd_rd(__fmul_rd(mx, fk[c]), ev[c]));
            }
            if (u == u0 || z - m > kKv8Below) {
              const float nb = fmaxf(__fadd_rd(z, -kKv8Below), -FLT_MAX);
              k = fast_exp2(m - nb);
              m = nb;
            }
            l *= k;
            base = m;
            // P of scores within a step of so large a base may pass fp16: no further than
            // its largest (the exponents themselves stand for the scores then)
            if (__any_sync(0xffffffffu, fabsf(m) > kKv4Far && m > -FLT_MAX)) {
              const bool far = fabsf(m) > kKv4Far && m > -FLT_MAX;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int i = 16 * c; i < 16 * c + 16; ++i) {
                  const float e = fmaf(__uint_as_float(x[i]), fk[c], ev[c] - m);
                  if (far) x[i] = __float_as_uint(e > kKv8TopLog2 ? kKv8TopLog2 : e);  // (a NaN stays)
                }
                if (far) fk[c] = 1.f, ev[c] = 0.f;
              }
              if (far) base = 0.f;
            }
          }
          l += add;
        }
        // the next scores; they come after the stream's product before, which has then read
        // P, and is in O (idle warps wait too: no warp arrives twice in one phase of p_full)
        if (u + 1 < u1)
          await(&s_full[w], (t + 1) & 1, X8_S_FULL);
        else if (t > 0)
          await(&o_done[w], (t - 1) & 1, X8_O_DONE);
        tc_fence_after();
        if (moved && u > u0) {
#pragma unroll 1
          for (uint32_t c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(to + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= k;
            tmem_st32(to + c, o);
          }
        }
        // the next scores come while P goes
        if (!idle) tmem_st32(tp, *reinterpret_cast<float(*)[32]>(pk));
        if (u + 1 < u1) begin_load();
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
        if (u + 1 < u1) end_load();
      }
      ++mg;
      // the piece's partials, once both streams' last products are done: each stream
      // reads both O for half of the channels and writes their sum
      row_ml[w][lrow] = make_float2(m, l);
      tc_bar();
      await(&o_done[w], (t - 1) & 1, X8_O_DONE);
      await(&o_done[w ^ 1], (t - 1) & 1, X8_O_DONE);
      tc_fence_after();
      const size_t slot = size_t(blockIdx.x) + seg;
      if (!idle) {
        const float2 o2 = row_ml[w ^ 1][lrow];
        const float mm = fmaxf(m, o2.x), w0 = fast_exp2(m - mm), w1 = fast_exp2(o2.x - mm);
        if (w == 0 && row < R) a.ml[slot * a.R16 + lrow] = make_float2(mm, w0 * l + w1 * o2.y);
        // (a lane writes whole sectors of its own row: 32 bytes an instruction.  With 16 bytes a
        // piece took 2.8 us longer, through shared memory by neighbouring lanes 1.2.)
#pragma unroll 1
        for (uint32_t c = 0; c < D / 2; c += 16) {
          uint32_t v[16], p[16];
          tmem_ld16_async(to + uint32_t(w) * (D / 2) + c, v);
          tmem_ld16_async(to2 + uint32_t(w) * (D / 2) + c, p);
          tmem_ld16_done(v);
          tmem_ld16_done(p);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = __float_as_uint(fmaf(__uint_as_float(p[i]), w1, __uint_as_float(v[i]) * w0));
          if (row < R) {
            float* dst = a.opart + (slot * a.R16 + lrow) * D + w * (D / 2) + c;
#pragma unroll
            for (int i = 0; i < 16; i += 8) store8(dst + i, v + i);
          }
        }
      }
      tc_fence_before();
      tc_bar();  // (O and row_ml have been read: the next piece may begin)
      return true;
    });
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    {
      // ------------------------------------------------- values to fp16
      // A lane turns chunks of 16 channels, one of which becomes two: eight (d = 64: four)
      // neighbouring lanes read eight chunks of one row (two rows).  With d = 128 the lanes
      // of a row's second half take the row beside it, so that in reads and writes the
      // eight lanes of a shared-memory phase meet eight different groups of banks.
      // Every load of a tile first: with two chunks under way at a time a tile took
      // 1,500 cycles, which was the longest of all roles.
      constexpr int CPR = D / 16, RPW = 32 / CPR, kTasks = 32 / RPW, kPar = 8 / RPW;
      const int c = lane % CPR, cw = warp - 8;
      // row (of the warp's 32) of task s: eight more every kPar tasks
      auto row_of = [&](int s) {
        return D == 128 ? (s >> 1) * 8 + (lane >> 3) * 2 + ((s & 1) ^ (c >> 2)) : s * 8 + (lane >> 2);
      };
      const uint32_t vs = smem_u32(base) + S::kV, v16 = smem_u32(base) + S::kV16;
      uint32_t from[kPar], to[kPar];
#pragma unroll
      for (int i = 0; i < kPar; ++i) {
        const uint32_t r = uint32_t(cw * 32 + row_of(i));
        from[i] = rows_off<D>(r, uint32_t(c));
        to[i] = uint32_t(D == 128 ? c >> 2 : 0) * 16384u + sw128_off(r, uint32_t(c & 3) * 2u);
      }
      uint32_t t = 0, mg = 0;
      kv8_pieces(a, share, [&](int, int, int, int, int u0, int u1) -> bool {
        for (int u = u0; u < u1; ++u, ++t) {
          const uint32_t st = t % VS, b = t & 1;
          if ((u - u0) % 4 == 0 && u > u0) ++mg;
          if ((u - u0) % 4 == 0 && !wait(&meta_full[mg % kKv8Groups], (mg / kKv8Groups) & 1, X8_META))
            return false;
          const Kv8TileMeta& mt = meta[mg % kKv8Groups][(u - u0) % 4];
          if (!wait(&v_full[st], (t / VS) & 1, X8_V_FULL)) return false;
          if (t >= 2 && !wait(&v16_free[b], ((t >> 1) - 1) & 1, X8_V16_FREE)) return false;
          const uint32_t src = vs + st * S::kTile, dst = v16 + b * S::kTile16;
          uint4 x[kTasks];
#pragma unroll
          for (int s = 0; s < kTasks; ++s)
            x[s] = lds128(src + from[s % kPar] + uint32_t(s / kPar) * (8u * D));
          if (!mt.whole[0]) {  // rows that do not count may hold any bytes: no 0 * NaN
            const uint32_t k0 = mt.keys[2 * cw], k1 = mt.keys[2 * cw + 1];  // of this warp's rows
#pragma unroll
            for (int s = 0; s < kTasks; ++s) {
              const uint32_t r = uint32_t(row_of(s));
              if ((r & 15u) >= (r < 16u ? k0 : k1)) x[s] = make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int s = 0; s < kTasks; ++s) {
            uint32_t h[8];
            e4m3x4_to_half2(x[s].x, h[0], h[1]);
            e4m3x4_to_half2(x[s].y, h[2], h[3]);
            e4m3x4_to_half2(x[s].z, h[4], h[5]);
            e4m3x4_to_half2(x[s].w, h[6], h[7]);
            const uint32_t at = dst + to[s % kPar] + uint32_t(s / kPar) * 1024u;
            sts128(at, h[0], h[1], h[2], h[3]);
            sts128(at ^ 16u, h[4], h[5], h[6], h[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_free[st]), mbar_arrive(&v16_full[b]);
        }
        ++mg;
        return true;
      });
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 12) {
      // ------------------------------------------------------------ copies
      const int page = 1 << a.c.page_log2;
      const int ti = lane >> 3, gr = (lane & 7) * 16;  // this lane's tile of four, its 16 keys
      uint32_t t = 0, mg = 0, k_issued = 0, v_issued = 0;
      kv8_pieces(a, share, [&](int n, int gt, int, int ctx, int u0, int u1) -> bool {
        const int g = gt / a.row_tiles;
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
          auto publish = [&] {  // the group's keys and scales
            const uint32_t x = mg % kKv8Groups;
            const int e_k = kv8_exp(uint32_t(ek)), e_v = kv8_exp(uint32_t(ev)), j = lane & 7;
            const int keys = have ? min(16, ctx - pos) : 0;
            const uint32_t some = __ballot_sync(0xffffffffu, keys < 16);
            Kv8TileMeta& m = meta[x][ti];
            m.sk[j] = exp2_int(e_k), m.ev[j] = float(e_v), m.iv[j] = exp2_int(-e_v);
            m.keys[j] = uint32_t(keys);
            if (j == 0) m.whole[0] = (some >> (8 * ti) & 0xFFu) == 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&meta_full[x]);
            ++mg;
          };
          // (a piece's first scales are still on their way: its first copies go before them)
          if (u > u0) publish();
          for (int i = 0; i < tiles; ++i) {
            const uint32_t x = t + uint32_t(i), ks = x % KS, vst = x % VS;
            const uint32_t bytes = uint32_t(__popc(heads >> (8 * i) & 0xFFu) * page) * D;
            if (x >= uint32_t(KS) && !wait(&k_free[ks], (x / KS - 1) & 1, X8_K_FREE)) return false;
            k_issued = x + 1;
            if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], bytes);
            __syncwarp();
            if (head && ti == i)
              tma_load_3d(base + ks * S::kTile + uint32_t(gr) * D, &kmap, &k_full[ks], 0,
                          g << a.c.page_log2, phys);
            if (x >= uint32_t(VS) && !wait(&v_free[vst], (x / VS - 1) & 1, X8_V_FREE)) return false;
            v_issued = x + 1;
            if (lane == 0) mbar_arrive_expect_tx(&v_full[vst], bytes);
            __syncwarp();
            if (head && ti == i)
              tma_load_3d(base + S::kV + vst * S::kTile + uint32_t(gr) * D, &vmap, &v_full[vst], 0,
                          g << a.c.page_log2, phys);
          }
          if (u == u0) publish();
          phys = next, next = after, ek = ek1, ev = ev1;
          t += uint32_t(tiles);
        }
        return true;
      });
      // every copy has landed before the CTA may leave (where a wait has run out, nobody
      // else waits for it)
      for (uint32_t i = k_issued > uint32_t(KS) ? k_issued - KS : 0; i < k_issued; ++i)
        mbar_wait(&k_full[i % KS], (i / KS) & 1);
      for (uint32_t i = v_issued > uint32_t(VS) ? v_issued - VS : 0; i < v_issued; ++i)
        mbar_wait(&v_full[i % VS], (i / VS) & 1);
    } else if (warp < 15) {
      // ----------------------------------------------------------- issuers
      // (the whole warp walks the loops, an elected lane issues)
      const uint32_t w = uint32_t(warp - 13);
      const uint64_t kd = make_sdesc_rows<D>(smem_u32(base) + w * (64u * D));
      const uint64_t vd = make_sdesc_sw128(smem_u32(base) + S::kV16 + w * 8192u, 16384u, 1024);
      constexpr uint32_t ids = make_idesc_e4m3(128, 64, false, false);
      constexpr uint32_t ido = make_idesc_half(128, D, true);
      uint32_t t = 0, np = 0;
      kv8_pieces(a, share, [&](int, int, int, int, int u0, int u1) -> bool {
        if (!wait(&q_full, np & 1, X8_Q_FULL)) return false;
        ++np;
        // S of tile u, then P V of the one before: the next S comes after that, so whoever
        // has its scores knows that P has been read
        for (int u = u0; u <= u1; ++u) {
          if (u < u1) {
            const uint32_t st = t % KS;
            if (!wait(&k_full[st], (t / KS) & 1, X8_K_FULL)) return false;
            // the stream's scores of the step before have been read
            if (t > 0 && !wait(&s_read[w], (t - 1) & 1, X8_S_READ)) return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks)
                  umma_e4m3_ts(tm + w * 64u, tm + (part ? kKv8TmQ1 : kKv8TmQ0) + uint32_t(ks) * 8u,
                               kd + ((st * S::kTile + uint32_t(ks) * 32u) >> 4), ids, part + ks > 0);
              umma_commit(&s_full[w]);
              umma_commit(&k_free[st]);
            }
            __syncwarp();
            ++t;
          }
          if (u > u0) {
            const uint32_t x = u < u1 ? t - 2 : t - 1, vb = x & 1;
            if (!wait(&v16_full[vb], (x >> 1) & 1, X8_V16_FULL)) return false;
            if (!wait(&p_full[w], x & 1, X8_P_FULL)) return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                umma_bf16_ts(tm + kKv8TmO + w * 128u, tm + kKv8TmP + w * 32u + uint32_t(ks) * 8u,
                             vd + ((vb * S::kTile16) >> 4) + uint32_t(ks) * 128u, ido,
                             u - 1 > u0 || ks > 0);
              umma_commit(&o_done[w]);
              umma_commit(&v16_free[vb]);
            }
            __syncwarp();
          }
        }
        return true;
      });
      // every product and commit is done before the tensor memory is given back
      if (t > 0 && elect_one()) {
        umma_commit(&all_done[w]);
        mbar_wait(&all_done[w], 0);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (threadIdx.x == 0 && failed)
    record_error(err, DEV_TIMEOUT_MMA | DEV_K_KV8_ATTN | (failed << 16));
  tmem_teardown(tm, 512);
}

// ------------------------------------------------------------------- host

template <int D>
static cudaError_t launch_tc(const Kv8AttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                             uint32_t* err, cudaStream_t st) {
  constexpr size_t smem = Kv8Tc<D>::kSmem;
  HERALD_CHECK_LAUNCH(ensure_smem(kv8_attn_tc_kernel<D>, smem));
  return launch_k("kv8_attn_tc_kernel", kv8_attn_tc_kernel<D>, dim3(unsigned(a.ctas)),
                  dim3(kKv8TcThreads), smem, st, a, kmap, vmap, err);
}
cudaError_t launch_kv8_attn_tc(int d, const Kv8AttnArgs& a, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, uint32_t* err, cudaStream_t st) {
  return d == 128 ? launch_tc<128>(a, kmap, vmap, err, st) : launch_tc<64>(a, kmap, vmap, err, st);
}

HERALD_DEBUG_WORD_READER(debug_take_kv8_attn_tc)

}  // namespace herald
