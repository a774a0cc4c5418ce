// kv4_attn_tc.cu -- attention over the paged 4-bit cache on the 5th-generation
// tensor cores, for blocks of queries (many rows per KV head).
//
// The tensor cores take fp16 operands from shared memory, so the codes are
// turned into fp16 there (exact, kv4.cuh), once per 128-key tile for up to 256
// query rows.  One CTA per SM walks its share of the keys (kv4_split, tiles of
// 128 keys, a segment's block keys first):
//   warps 17, 19 copy the codes and scales of a tile's K and V rows from its pages
//                into raw slots (bulk copies; the pages of a tile in parallel
//                lanes)
//   warps 8-11, 12-15 turn the K and the V slots into fp16 128-byte-swizzled
//                operand buffers
//   warps 16, 18 a tcgen05.mma issuer per stream of S = Q K^T into a score buffer
//   warps 20, 21 one per stream of O += P V with P read from tensor memory
//                (issuing an mma takes a warp about a hundred cycles: with one
//                warp per stream for both products that was the longest chain)
//   warps 0-3, 4-7 softmax of a stream, a thread per query row; together they stage
//                the queries
// Two streams run side by side: with more than 128 rows a stream is a row tile
// and takes every key tile, else both streams have the same rows and take
// alternate key tiles (at a piece's end each adds both outputs for half of the
// channels).  A stream goes in steps of 64 keys through two score buffers of 64
// TMEM columns (P, fp16, overlays the scores), so the scores of a step are
// there when the softmax of the step before is done; O takes 128 columns: the
// two streams fill the 512.
//
// A block of 32 tokens over 4 x 64K (128 rows, 8 KV heads) takes 119 us: 305 MB, 137
// GFLOP.  No unit bounds it: the tensor pipe is active for 48% of the time, memory for
// a third; 0.7 of the issue slots are taken by 5,650 warp instructions a tile, and the
// roles crowd the instruction cache: code that is unrolled more runs slower (the
// conversion by two chunks: 136 us where it was 127).
//
// A step's scores are read once: with the base m of the row as it is, P =
// 2^(s - m) stays in fp16 as long as the row's 64 of them sum to less than 60000.
// Where a sum does not (and at a piece's first step), the scores are looked at for
// their maximum, m is set 5 below it, O and l follow, and the step is done again:
// 64 P of a new base sum to 2^11 at most, and the scores must rise by 5 to 11
// (log2) before it happens again.  (Looking for the maximum in every step, as
// kv4_attn.cu does: 4 x 64K 146 us instead of 139.  With the base 9 below: 149,
// the CTAs whose keys rise late doing more steps twice than the others.)
//
// The block's own keys are bf16: their tiles come first in a segment, with
// the queries staged as bf16 (an mma's operands have one type), then the
// queries are staged again as fp16 for the cache.  P is bf16 there as well, two
// numbers a weight (take_bf16): the scores' 64 columns have room for both.
#include <float.h>

#include "kv4.cuh"
#include "tc_common.cuh"

namespace herald {

constexpr int kTcKeys = kKv4Tile;          // keys per tile
constexpr int kTcStep = 64;                // keys per step of a stream
constexpr int kTcBufs = 4;                 // operand buffers (128 keys of K or V)
// Raw slots of K and of V tiles: as many as fit beside the operands.
__host__ __device__ constexpr int tc_raw_k(int MT) { return MT == 2 ? 2 : 3; }
__host__ __device__ constexpr int tc_raw_v(int MT) { return MT == 2 ? 1 : 3; }
// Tiles whose key masks are kept for the softmax.  A K copy runs at most three slots and two
// operand buffers ahead of the scores, and the scores two steps ahead of P: the
// mask of 16 tiles back has been read by everybody.
constexpr int kTcMasks = 16;
constexpr int kTcSoft = 256;               // softmax threads
constexpr int kTcThreadsAll = 768;         // 8 + 8 + 8 warps (22, 23 only fill a warpgroup)
constexpr int kTcSWarp = 16, kTcCopyWarp = 17, kTcPvWarp = 20;  // S 16, 18; copies 17, 19; P V 20, 21
constexpr float kTcBelow = 5.f, kTcTop = 60000.f;  // base of P and largest sum (see above)
constexpr float kTcTopLog2 = 15.8727f;                // log2 of kTcTop

// Waits of the kernel (bits 16-31 of the error word).
enum : uint32_t {
  W_RAW_FREE = 1, W_RAW_FULL = 2, W_BUF_FREE = 4, W_Q_FREE = 8, W_Q_FULL = 0x10, W_K_FULL = 0x20,
  W_P_FULL = 0x40, W_V_FULL = 0x80, W_PV_DONE = 0x100, W_S_FULL = 0x200, W_MASK = 0x400,
  W_O_DONE = 0x800, W_O_READ = 0x1000
};

struct TcSmem {
  uint32_t q, buf, raw, total;
};
__host__ __device__ inline TcSmem tc_smem(int D, int MT) {
  TcSmem s;
  const uint32_t tile = uint32_t(D / 64) * 16384u;  // 128 rows of D fp16
  s.q = 0;
  s.buf = s.q + uint32_t(MT) * tile;
  s.raw = s.buf + uint32_t(kTcBufs) * tile;
  s.total = s.raw + uint32_t(tc_raw_k(MT) + tc_raw_v(MT)) * uint32_t(kTcKeys * (D / 2 + D / 16)) + 1024u;
  return s;
}

// Instruction descriptor of kind::f16 with fp16 A and B (make_idesc_bf16 with
// formats 0).
__host__ __device__ constexpr uint32_t make_idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

HERALD_DEV void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
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
// Waits for this thread's tensor-memory loads; r (loaded before) counts as
// written here, so that no use of it moves above the wait.
HERALD_DEV void tmem_wait_ld(uint32_t (&r)[32]) {
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

// Scores of keys that do not count become -inf: those without a bit in msk (two
// words), or, without msk, all but the first nk of the 64.
HERALD_DEV void mask_scores(uint32_t ts, const uint32_t* msk, int nk) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const int left = nk - 32 * c;
    const uint32_t k = msk ? msk[c] : left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u;
    if (k == ~0u) continue;
    uint32_t r[32];
    tmem_ld32_nowait(ts + uint32_t(c) * 32u, r);
    tmem_wait_ld(r);
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = (k >> i & 1) ? __uint_as_float(r[i]) : -INFINITY;
    tmem_st32(ts + uint32_t(c) * 32u, v);
  }
  tmem_wait_st();
}

// 32 scores -> probabilities 2^(s f - m), summed into *sum.
HERALD_DEV void exp32(uint32_t (&x)[32], uint64_t f2, uint64_t nm2, uint64_t* sum) {
  uint64_t sa = *sum, sb = f2_pack(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float t0, t1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), f2, nm2), t0, t1);
    const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
    if (i & 2)
      sa = f2_add(sa, f2_pack(p0, p1));
    else
      sb = f2_add(sb, f2_pack(p0, p1));
    x[i] = __float_as_uint(p0);
    x[i + 1] = __float_as_uint(p1);
  }
  *sum = f2_add(sa, sb);
}
// 32 probabilities -> 16 packed columns.  blk: bf16, times iv (P in units of
// v_scale: O has one unit for all keys; the weights' first numbers, rest_of_p has
// the second), else fp16.
HERALD_DEV void pack_p32(uint32_t* pk, const uint32_t (&x)[32], bool blk, float iv) {
  if (blk) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      pk[i] = pack_bf16(__uint_as_float(x[2 * i]) * iv, __uint_as_float(x[2 * i + 1]) * iv);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      pk[i] = pack_half2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
  }
}

HERALD_DEV void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// The second numbers of a block step's weights, from its scores at ts once more, into
// columns 32-63 (the second half's first: its own scores lie there; none without keys,
// nk, in it).  Block steps are few: kept beside P in the steps' common code these
// numbers spilled registers, and blocks took 29.1 us at 32K and 120 at 4 x 64K instead
// of 28.5 and 118.4.  (With one number a weight 27.9 and 117.1.)
HERALD_DEV void rest_of_p(uint32_t ts, uint64_t f2, uint64_t nm2, float iv, int nk) {
#pragma unroll 1
  for (int c = nk > 32 ? 1 : 0; c >= 0; --c) {
    uint32_t x[32], rest[16];
    uint64_t sum = f2_pack(0.f, 0.f);
    tmem_ld32_nowait(ts + uint32_t(c) * 32u, x);
    tmem_wait_ld(x);
    exp32(x, f2, nm2, &sum);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a = __uint_as_float(x[2 * i]) * iv, b = __uint_as_float(x[2 * i + 1]) * iv;
      take_bf16(a, b);
      rest[i] = pack_bf16(a, b);
    }
    tmem_st16(ts + 32u + uint32_t(c) * 16u, rest);
  }
}

HERALD_DEV uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Largest magnitude of 16 bf16 (a NaN does not count).
HERALD_DEV float absmax16(const uint4& a, const uint4& b) {
  constexpr uint32_t k = 0x7FFF7FFFu;
  const uint32_t m = max_bf16x2(
      max_bf16x2(max_bf16x2(a.x & k, a.y & k), max_bf16x2(a.z & k, a.w & k)),
      max_bf16x2(max_bf16x2(b.x & k, b.y & k), max_bf16x2(b.z & k, b.w & k)));
  return fmaxf(bf16lo(m), bf16hi(m));
}

template <int D, int MT>
__global__ void __launch_bounds__(kTcThreadsAll, 1)
    kv4_attn_tc_kernel(const Kv4AttnArgs a, uint32_t* err) {
  constexpr int H = D / 64, kRawK = tc_raw_k(MT), kRawV = tc_raw_v(MT);
  constexpr uint32_t kTile = uint32_t(H) * 16384u;
  constexpr int kRowC = D / 2, kRowS = D / 16;           // raw bytes of a row
  constexpr uint32_t kRawBytes = kTcKeys * (kRowC + kRowS);
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t raw_full[2][kRawK], raw_free[2][kRawK];  // [K or V][slot]
  __shared__ uint64_t buf_full[kTcBufs], buf_free[kTcBufs];
  __shared__ uint64_t q_full, q_free, s_full[2][2], p_full[2][2], pv_done[2][2], o_done[2];
  __shared__ uint64_t all_done[4], ml_full, o_read;
  __shared__ float2 row_ml[2][kTileM];              // a piece's (m, l) of both streams
  __shared__ uint64_t mask_full[kTcMasks];
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t failed;
  __shared__ uint32_t missing;                      // a position below a length had no page
  __shared__ float row_f[2 * kTileM];               // score factors of the rows (cache tiles)
  __shared__ uint32_t key_mask[kTcMasks][4];        // bit: the key counts
  __shared__ uint32_t val_mask[kRawV][4];           // the same, for the rows of a raw V slot
  const TcSmem L = tc_smem(D, MT);
  uint8_t* base = align1024(smem_raw);
  uint8_t *Qs = base + L.q, *Bs = base + L.buf, *Rs = base + L.raw;
  const uint32_t qs = smem_u32(Qs), bs = smem_u32(Bs), raw_s = smem_u32(Rs);
  const int warp = warp_same(int(threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * kRawK; ++i)
      mbar_init(&raw_full[i & 1][i >> 1], 1), mbar_init(&raw_free[i & 1][i >> 1], 4);
    for (int i = 0; i < kTcBufs; ++i) mbar_init(&buf_full[i], 4), mbar_init(&buf_free[i], MT);
    for (int i = 0; i < kTcMasks; ++i) mbar_init(&mask_full[i], 1);
    mbar_init(&q_full, 8);
    mbar_init(&ml_full, 8), mbar_init(&o_read, 8);
    mbar_init(&q_free, 2 + kTcSoft);
    for (int i = 0; i < 2; ++i)
      mbar_init(&s_full[i][0], 1), mbar_init(&s_full[i][1], 1), mbar_init(&p_full[i][0], 128),
          mbar_init(&p_full[i][1], 128), mbar_init(&pv_done[i][0], 1),
          mbar_init(&pv_done[i][1], 1), mbar_init(&o_done[i], 1), mbar_init(&all_done[i], 1),
          mbar_init(&all_done[2 + i], 1);
    failed = 0;
    missing = 0;
    fence_mbar_init();
  }
  tmem_setup(&tmem_base, 512);
  const uint32_t tm = tmem_base;
  griddep_enter();
  const Kv4Wait wait{&failed};

  const int G = a.Hq / a.Hkv, R = a.B * G;
  const int blk_units = a.bk ? (a.B + kTcKeys - 1) / kTcKeys : 0;
  const Kv4Share sh = kv4_share(a, blk_units, int(blockIdx.x));
  const int end = sh.end;

  // Every role walks the same pieces: body(n, g, seg, ctx, units, u0, u1) with
  // tiles u0 <= u < u1 of the segment, the first blk_units of them block tiles;
  // it returns false to leave (a wait ran out).
  auto pieces = [&](auto&& body) {
    int at = sh.at, first = sh.first, n = sh.n;
    while (at < end) {
      const int ctx = warp_same(min(max(a.ctx[n], 0), a.L_max));
      const int units = kv4_units(ctx, a.L_max, blk_units, a.pad);
      if (units == 0 || at >= first + a.Hkv * units) {
        first += a.Hkv * units;
        ++n;
        continue;
      }
      const int g = (at - first) / units;
      const int seg0 = first + g * units;
      const int u0 = max(at - seg0 - a.pad, 0), u1 = min(units, end - seg0) - a.pad;
      if (u1 > 0 && !body(n, g, n * a.Hkv + g, ctx, units - a.pad, u0, u1)) return;
      at = seg0 + a.pad + u1;
    }
  };
  // keys of tile u that can count
  auto tile_keys = [&](int u, int ctx) {
    return min(kTcKeys, u < blk_units ? a.B - u * kTcKeys : ctx - (u - blk_units) * kTcKeys);
  };

  // registers: 768 threads launch with 80 each (61,440) = 256 x (112 + 80 + 48).
  // Each role's branch begins with its own setmaxnreg, so that the compiler
  // knows the limit of the code that follows.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2;                  // stream
    const int lrow = (warp & 3) * 32 + lane;  // TMEM lane
    const int row = (MT == 2 ? w * kTileM : 0) + lrow;
    const bool idle = (MT == 2 ? w * kTileM : 0) + (warp & 3) * 32 >= R;  // the warp has no rows
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t ts0 = tm + lanes + uint32_t(w) * 128u, to = ts0 + 256u;
    const float iv = 1.f / a.c.v_scale;
    uint32_t tile = 0, ns = 0, mt = 0, phase = 0;  // tiles of the CTA, steps of the stream, masks
    uint32_t no = 0, np = 0;  // bit x: parity of the pieces with a step of stream x; pieces
    pieces([&](int n, int g, int seg, int ctx, int units, int u0, int u1) -> bool {
      debug_flag(threadIdx.x == 0 && a.ctx[n] != ctx, DEV_BAD_COUNT);
      const uint32_t first_tile = tile;
      float m = -FLT_MAX, l = 0.f;
      bool any = false;  // this stream has had a step of the piece
      int u = u0;
      while (u < u1) {  // a phase: block tiles, or cache tiles
        const bool blk = u < blk_units;
        const int pe = blk ? min(u1, blk_units) : u1;
        // the phase's queries: staged by these warps (the conversion starts on
        // the keys meanwhile) once the scores and factors of the phase before are
        // done with
        if (phase > 0 && !wait(&q_free, (phase - 1) & 1, W_Q_FREE)) return false;
        // queries: D/16 lanes per row, 16 channels each
        constexpr int LPR = D / 16;
        constexpr int kPass = kTcSoft / LPR, kRows = kTileM / kPass;  // rows per pass and tile
        const int c = int(threadIdx.x) % LPR;
        uint4 x4[MT * kRows][2];  // (every load first)
        {
#pragma unroll
          for (int i = 0; i < MT * kRows; ++i) {
            const int r = i * kPass + int(threadIdx.x) / LPR;
            x4[i][0] = x4[i][1] = make_uint4(0, 0, 0, 0);
            if (r < R) {
              const uint4* src = reinterpret_cast<const uint4*>(
                  a.q + ((size_t(n) * a.B + r / G) * a.Hq + g * G + r % G) * D + c * 16);
              x4[i][0] = src[0];
              x4[i][1] = src[1];
            }
          }
          float mx[MT * kRows];  // (the rows' maxima side by side: their steps wait on one another)
          if (!blk) {
#pragma unroll
            for (int i = 0; i < MT * kRows; ++i) mx[i] = absmax16(x4[i][0], x4[i][1]);
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
              for (int i = 0; i < MT * kRows; ++i)
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
          }
#pragma unroll
          for (int i = 0; i < MT * kRows; ++i) {
            const int mt2 = i / kRows, rr = i % kRows * kPass + int(threadIdx.x) / LPR;
            uint32_t x[8] = {x4[i][0].x, x4[i][0].y, x4[i][0].z, x4[i][0].w,
                             x4[i][1].x, x4[i][1].y, x4[i][1].z, x4[i][1].w};
            if (!blk) {  // fp16 scaled per row by a power of two (see kv4_attn.cu)
              float up, f;
              kv4_query_scale(mx[i], a.sc, a.sc_e, &up, &f);
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] = pack_half2(bf16lo(x[k]) * up, bf16hi(x[k]) * up);
              if (c == 0) row_f[mt2 * kTileM + rr] = f;
            }
            const uint32_t dst = qs + uint32_t(mt2) * kTile + uint32_t(c >> 2) * 16384u;
            const uint32_t c8 = uint32_t(c & 3) * 2u;
            sts128(dst + sw128_off(uint32_t(rr), c8), x[0], x[1], x[2], x[3]);
            sts128(dst + sw128_off(uint32_t(rr), c8 + 1), x[4], x[5], x[6], x[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
        if (!wait(&q_full, phase & 1, W_Q_FULL)) return false;
        const float f = blk ? a.scale * 1.4426950408889634f
                            : *(volatile float*)&row_f[row];
        const uint64_t f2 = f2_pack(f, f);
        mbar_arrive(&q_free);  // (this thread has read its factor of the phase)
        ++phase;
        const int ue = u;
        if (MT == 1 && int(tile & 1) != w) ++u;
        for (; u < pe; u += 3 - MT) {
          const uint32_t mask_no = mt + uint32_t(u - ue);
          const int keys = tile_keys(u, ctx);
#pragma unroll 1
          for (int k0 = 0; k0 < keys; k0 += kTcStep, ++ns) {
            const uint32_t b = ns & 1, ts = ts0 + b * 64u;
            if (!wait(&s_full[w][b], (ns >> 1) & 1, W_S_FULL)) return false;
            tc_fence_after();
            if (!idle) {
              if (keys < k0 + kTcStep || (!blk && *(volatile uint32_t*)&missing)) {
                const uint32_t* msk = nullptr;
                if (!blk) {
                  const uint32_t i = mask_no % kTcMasks;
                  if (!wait(&mask_full[i], (mask_no / kTcMasks) & 1, W_MASK)) return false;
                  msk = key_mask[i] + k0 / 32;
                }
                mask_scores(ts, msk, keys - k0);
              }
              float p[32], s0, s1;
              float nm = -m;  // P = 2^(score f + nm)
              bool again = false;
              while (true) {
                bool high = true;
                if (any || again) {  // (a piece's first step has no base yet)
                  const uint64_t nm2 = f2_pack(nm, nm);
                  uint64_t sum = f2_pack(0.f, 0.f);
                  uint32_t x[32], y[32];
                  tmem_ld32_nowait(ts, x);
                  tmem_ld32_nowait(ts + 32u, y);
                  tmem_wait_ld(x);
                  tmem_wait_ld(y);
                  exp32(x, f2, nm2, &sum);
                  pack_p32(reinterpret_cast<uint32_t*>(p), x, blk, iv);
                  exp32(y, f2, nm2, &sum);
                  pack_p32(reinterpret_cast<uint32_t*>(p) + 16, y, blk, iv);
                  f2_unpack(sum, s0, s1);
                  high = !(s0 + s1 <= kTcTop);
                  if (again || !__any_sync(0xffffffffu, high)) break;
                }
                again = true;
                float mx = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                  uint32_t x[32];
                  tmem_ld32_nowait(ts + uint32_t(c) * 32u, x);
                  tmem_wait_ld(x);
#pragma unroll
                  for (int i = 0; i < 32; i += 2)
                    mx = fmax3f(mx, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                }
                float k = 1.f;
                const bool far = fabsf(mx * f) > kKv4Far;
                if (high && mx * f - m > kTcBelow) {
                  const float nb =
                      far ? __fadd_rd(__fmul_rd(mx, f), -kTcBelow) : mx * f - kTcBelow;
                  k = fast_exp2(m - nb);
                  m = nb;
                  l *= k;
                }
                nm = -m;
                if (__any_sync(0xffffffffu, far)) {  // P's exponents over f as scores (kKv4Far)
                  const float per_f = 1.f / f;
#pragma unroll 1
                  for (int c = 0; c < 2; ++c) {
                    uint32_t x[32];
                    tmem_ld32_nowait(ts + uint32_t(c) * 32u, x);
                    tmem_wait_ld(x);
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                      v[i] = __uint_as_float(x[i]);
                      const float t = fmaf(v[i], f, -m);
                      if (far) v[i] = (t > kTcTopLog2 ? kTcTopLog2 : t) * per_f;  // (a NaN stays)
                    }
                    tmem_st32(ts + uint32_t(c) * 32u, v);
                  }
                  tmem_wait_st();
                  if (far) nm = 0.f;
                }
                // O so far, once the P V of the step before is in it (that of two
                // steps before is: this step's scores took its buffer)
                if (any) {
                  if (!wait(&pv_done[w][b ^ 1], ((ns - 1) >> 1) & 1, W_O_DONE)) return false;
                  tc_fence_after();
#pragma unroll 1
                  for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[32];
                    tmem_ld32_nowait(to + uint32_t(c) * 32u, r);
                    tmem_wait_ld(r);
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * k;
                    tmem_st32(to + uint32_t(c) * 32u, v);
                  }
                  tmem_wait_st();
                }
              }
              if (blk) rest_of_p(ts, f2, f2_pack(nm, nm), iv, keys - k0);
              tmem_st32(ts, p);
              l += s0 + s1;
              tmem_wait_st();
            }
            tc_fence_before();
            // (one barrier per buffer: a warp may be a step ahead of another)
            mbar_arrive(&p_full[w][b]);
            any = true;
          }
        }
        tile += uint32_t(pe - ue);
        if (!blk) mt += uint32_t(pe - ue);
        u = pe;
      }
      // the piece's rows: O once the last P V is done (pv_done would not tell: the
      // last two may both be under way).  With one row tile a row has an O in each
      // stream: both streams read both, half the channels each, and write their sum.
      const int some = MT == 1 && u1 - u0 == 1 ? 1 << (first_tile & 1) : 3;  // streams with a step
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if ((MT == 2 && x != w) || !(some >> x & 1)) continue;
        if (!wait(&o_done[x], no >> x & 1, W_O_DONE)) return false;
      }
      no ^= uint32_t(some);
      tc_fence_after();
      float w0 = 1.f, w1 = 0.f;  // weights of this stream's O and of the other's
      if (MT == 1) {
        if (!any) m = -FLT_MAX, l = 0.f;
        row_ml[w][lrow] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ml_full);
        if (!wait(&ml_full, np & 1, W_O_READ)) return false;
        const float2 o = row_ml[w ^ 1][lrow];
        const float mm = fmaxf(m, o.x);
        w0 = any ? fast_exp2(m - mm) : 0.f;
        w1 = some >> (w ^ 1) & 1 ? fast_exp2(o.x - mm) : 0.f;
        l = w0 * l + w1 * o.y;
        m = mm;
      }
      if (!idle) {
        const bool whole = u0 == 0 && u1 == units;
        const float inv = l == 0.f ? 0.f : a.c.v_scale / l;
        const int slot = int(blockIdx.x) + seg;
        const bool on = row < R;
        float4* part = reinterpret_cast<float4*>(a.opart) + size_t(slot) * (D / 4) * a.R16 + row;
        uint16_t* out =
            a.out + ((size_t(n) * a.B + (on ? row / G : 0)) * a.Hq + g * G + (on ? row % G : 0)) * D;
        const uint32_t to2 = tm + lanes + 256u + uint32_t(w ^ 1) * 128u;
        constexpr int kParts = MT == 1 ? D / 64 : D / 32;
#pragma unroll 1
        for (int cc = 0; cc < kParts; ++cc) {
          const int c = MT == 1 ? w * kParts + cc : cc;
          uint32_t r[32];
          float v[32];
          if (MT == 2 || any) {
            tmem_ld32_nowait(to + uint32_t(c) * 32u, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * w0;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
          if (MT == 1 && (some >> (w ^ 1) & 1)) {
            tmem_ld32_nowait(to2 + uint32_t(c) * 32u, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(r[i]), w1, v[i]);
          }
          if (on && whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(out + c * 32 + i) =
                  make_uint4(pack_bf16(v[i] * inv, v[i + 1] * inv),
                             pack_bf16(v[i + 2] * inv, v[i + 3] * inv),
                             pack_bf16(v[i + 4] * inv, v[i + 5] * inv),
                             pack_bf16(v[i + 6] * inv, v[i + 7] * inv));
          } else if (on) {  // neighbouring rows of a warp are neighbours in memory
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              part[size_t(c * 8 + i / 4) * a.R16] =
                  make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
          __syncwarp();
        }
        if (on && !whole && (MT == 2 || w == 0))
          a.ml[size_t(slot) * a.R16 + row] = make_float2(m, l);
        __syncwarp();
        tc_fence_before();
      }
      if (MT == 1) {  // O and (m, l) have been read: the next piece may begin
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_read);
        if (!wait(&o_read, np & 1, W_O_READ)) return false;
        ++np;
        tc_fence_after();
      }
      return true;
    });
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // ------------------------------------------------ operand conversion
    const int ct = threadIdx.x - kTcSoft;
    const int kv = (warp - 8) >> 2, cw = warp & 3;  // K or V items; warp of the four
    uint32_t tile = 0, mt = 0;
    auto publish = [&](uint64_t* bar) {  // this warp's writes are ready for the tensor cores
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    pieces([&](int n, int g, int, int, int, int u0, int u1) -> bool {
      int u = u0;
      while (u < u1) {
        const bool blk = u < blk_units;
        const int pe = blk ? min(u1, blk_units) : u1;
        for (; u < pe; ++u, ++tile) {
          const uint32_t item = 2 * tile + uint32_t(kv), b = item % kTcBufs;
          const uint32_t dst = bs + b * kTile;
          if (blk) {  // bf16 rows of the block, zeros after them
            if (item >= uint32_t(kTcBufs) &&
                !wait(&buf_free[b], (item / kTcBufs - 1) & 1, W_BUF_FREE))
              return false;
            const uint16_t* src = kv ? a.bv : a.bk;
            constexpr int CPR = D / 8;  // 16-byte chunks of a row
#pragma unroll 1
            for (int i = ct & 127; i < kTcKeys * CPR; i += 128) {
              const int r = i / CPR, c = i % CPR, j = u * kTcKeys + r;
              uint4 v = make_uint4(0, 0, 0, 0);
              if (j < a.B)
                v = *reinterpret_cast<const uint4*>(
                    src + ((size_t(n) * a.B + j) * a.Hkv + g) * D + c * 8);
              sts128(dst + uint32_t(c >> 3) * 16384u + sw128_off(uint32_t(r), uint32_t(c & 7)), v.x,
                     v.y, v.z, v.w);
            }
          } else {
            const uint32_t slots = kv ? kRawV : kRawK, rm = mt % slots;
            if (!wait(&raw_full[kv][rm], (mt / slots) & 1, W_RAW_FULL)) return false;
            const uint32_t rc = raw_s + (rm + (kv ? kRawK : 0)) * kRawBytes;
            const uint32_t rsc = rc + uint32_t(kTcKeys * kRowC);
            // A lane turns chunks of 16 bytes (32 channels): chunk j of row r.
            // Rows and chunks are dealt so that the eight lanes of a
            // shared-memory phase read eight different 16-byte bank groups
            // ((r&1)*4 + j for d = 128, (r&3)*2 + j for 64) and write eight (the
            // swizzle's XOR of r&7 with the chunk).  The loop is kept rolled, the
            // next chunk's bytes read ahead: the roles share the instruction cache.
            constexpr int kTasks = kTcKeys * (kRowC / 16) / 128;
            const int j1 = (lane >> 2) & 1;
            const int j = D == 128 ? ((lane >> 1) & 1) + 2 * j1 : lane & 1;
            auto row_of = [&](int s) {
              return D == 128 ? cw * 32 + (s >> 1) * 16 + (lane >> 3) * 4 + (lane & 1) +
                                    2 * (j1 ^ (s & 1))
                              : cw * 32 + s * 16 + (lane >> 1);
            };
            uint32_t counts = ~0u;  // keys of this warp's rows that count
            // (a value row that does not count may hold any bytes: no 0 * NaN)
            if (kv) counts = *(volatile uint32_t*)&val_mask[rm][cw];
            if (item >= uint32_t(kTcBufs) &&
                !wait(&buf_free[b], (item / kTcBufs - 1) & 1, W_BUF_FREE))
              return false;
            const uint32_t dh = dst + uint32_t(D == 128 ? j >> 1 : 0) * 16384u;
            int r = row_of(0);
            uint4 code = lds128(rc + uint32_t(r * kRowC + j * 16));
            uint32_t sc = lds_u16(rsc + uint32_t(r * kRowS + j * 2));
#pragma unroll 1
            for (int s = 0; s < kTasks; ++s) {
              const uint32_t words[4] = {code.x, code.y, code.z, code.w};
              const uint32_t s2 = (counts >> (r & 31) & 1) ? e4m3x2_to_half2(sc) : 0u;
              // chunk (j&1)*4 + k of the row: its place is the first one's, XOR k
              const uint32_t at = dh + sw128_off(uint32_t(r), uint32_t((j & 1) * 4));
              if (s + 1 < kTasks) {
                r = row_of(s + 1);
                code = lds128(rc + uint32_t(r * kRowC + j * 16));
                sc = lds_u16(rsc + uint32_t(r * kRowS + j * 2));
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t h[4];
                e2m1x8_to_half2(words[k], h);
                const uint32_t fs = __byte_perm(s2, 0, k < 2 ? 0x1010 : 0x3232);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = hmul2(h[i], fs);
                sts128(at ^ uint32_t(k << 4), h[0], h[1], h[2], h[3]);
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_free[kv][rm]);
            ++mt;
          }
          publish(&buf_full[b]);
        }
      }
      return true;
    });
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kTcCopyWarp || warp == kTcCopyWarp + 2) {
      // ------------------------------------------------------- raw copies
      const int kv = (warp - kTcCopyWarp) >> 1;
      const uint32_t slots = kv ? kRawV : kRawK;
      const uint8_t* codes = kv ? a.c.vc : a.c.kc;
      const uint8_t* scales = kv ? a.c.vs : a.c.ks;
      const int sub = min(1 << a.c.page_log2, kTcKeys);  // keys of a tile in one page
      const int k0 = lane * sub;                         // lane i: sub-chunk i of the tile
      const uint32_t dst_c = uint32_t(k0 * kRowC), dst_s = uint32_t(kTcKeys * kRowC + k0 * kRowS);
      uint32_t mt = 0;
      pieces([&](int n, int g, int, int ctx, int, int u0, int u1) -> bool {
        const int32_t* table = a.c.table + size_t(n) * a.c.max_pages;
        int pos = (max(u0, blk_units) - blk_units) * kTcKeys + k0;
        const int stop = k0 < kTcKeys ? min(ctx, (u1 - blk_units) * kTcKeys) : 0;
        // the table's entry is read a tile ahead
        int next = pos < stop ? table[pos >> a.c.page_log2] : -1;
        for (int u = max(u0, blk_units); u < u1; ++u, ++mt, pos += kTcKeys) {
          const int phys = next;
          if (pos + kTcKeys < stop) next = table[(pos + kTcKeys) >> a.c.page_log2];
          const bool on = pos < stop, have = on && phys >= 0 && phys < a.c.n_pages;
          const int keys = have ? min(sub, ctx - pos) : 0;
          debug_flag(on && !have, DEV_BAD_INDEX);
          const uint32_t rows = uint32_t(keys + 15) & ~15u;  // whole groups of 16: inside the page
          const uint32_t total = __reduce_add_sync(0xffffffffu, rows);
          const uint32_t slot = mt % slots;
          uint64_t* full = &raw_full[kv][slot];
          if (mt >= slots && !wait(&raw_free[kv][slot], (mt / slots - 1) & 1, W_RAW_FREE))
            return false;
          // lane i < 8: which of keys 16 i .. 16 i + 15 count
          const int mine = __shfl_sync(0xffffffffu, keys, lane * 16 / sub) - lane * 16 % sub;
          uint32_t* mask = kv ? val_mask[slot] : key_mask[mt % kTcMasks];
          if (lane < 8)
            reinterpret_cast<volatile uint16_t*>(mask)[lane] =
                uint16_t((1u << min(max(mine, 0), 16)) - 1u);
          if (on && !have) *(volatile uint32_t*)&missing = 1;
          __syncwarp();
          if (lane == 0) {
            if (kv == 0) mbar_arrive(&mask_full[mt % kTcMasks]);
            mbar_arrive_expect_tx(full, total * uint32_t(kRowC + kRowS));
          }
          __syncwarp();
          if (rows) {
            const size_t row = kv4_row(a.c, phys, a.Hkv, g, pos);
            uint8_t* dst = Rs + (slot + (kv ? kRawK : 0)) * kRawBytes;
            bulk_load(dst + dst_c, codes + row * kRowC, rows * kRowC, full);
            bulk_load(dst + dst_s, scales + row * kRowS, rows * kRowS, full);
          }
        }
        return true;
      });
      // every copy has landed before the CTA may leave (where a wait has run out,
      // nobody else waits for it)
      for (uint32_t i = mt > slots ? mt - slots : 0; i < mt; ++i)
        mbar_wait(&raw_full[kv][i % slots], (i / slots) & 1);
    } else if (warp == kTcSWarp || warp == kTcSWarp + 2) {
      // ------------------------------------------------------ S issuers
      // (the whole warp walks the loops, lane 0 issues)
      const int w = (warp - kTcSWarp) >> 1;
      const uint32_t ts = tm + uint32_t(w) * 128u;
      // descriptors of buffer 0; other tiles and steps add to the address field
      // (which never carries: 14 bits hold all of shared memory)
      const uint64_t qd = make_sdesc_sw128(qs + (MT == 2 ? uint32_t(w) * kTile : 0u), 16, 1024);
      const uint64_t kd = make_sdesc_sw128(bs, 16, 1024);
      uint32_t tile = 0, ns = 0, phase = 0;  // tiles of the CTA, steps of the stream
      pieces([&](int, int, int, int ctx, int, int u0, int u1) -> bool {
        int u = u0;
        while (u < u1) {
          const bool blk = u < blk_units;
          const int pe = blk ? min(u1, blk_units) : u1;
          const uint32_t ids = blk ? make_idesc_bf16(kTileM, kTcStep, false, false)
                                   : make_idesc_f16(kTileM, kTcStep, false);
          if (!wait(&q_full, phase & 1, W_Q_FULL)) return false;
          const uint32_t ns0 = ns;
          const int ue = u;
          if (MT == 1 && int(tile & 1) != w) ++u;
          for (; u < pe; u += 3 - MT) {
            const uint32_t ki = 2 * (tile + uint32_t(u - ue)), kb = ki % kTcBufs;
            if (!wait(&buf_full[kb], (ki / kTcBufs) & 1, W_K_FULL)) return false;
            const int keys = tile_keys(u, ctx);
            for (int k0 = 0; k0 < keys; k0 += kTcStep, ++ns) {
              // P of two steps before has been read: its buffer is free
              const uint32_t b = ns & 1;
              if (ns >= 2 && !wait(&pv_done[w][b], ((ns >> 1) - 1) & 1, W_PV_DONE)) return false;
              tc_fence_after();
              const uint64_t kt = kd + ((kb * kTile + uint32_t(k0) * 128u) >> 4);
              if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                  const uint32_t off = (uint32_t(ks >> 2) * 16384u + uint32_t(ks & 3) * 32u) >> 4;
                  umma_bf16(ts + b * 64u, qd + off, kt + off, ids, ks > 0 ? 1u : 0u);
                }
                umma_commit(&s_full[w][b]);
                if (k0 + kTcStep >= keys) umma_commit(&buf_free[kb]);
              }
              __syncwarp();
            }
          }
          tile += uint32_t(pe - ue);
          u = pe;
          if (lane == 0) {
            if (ns > ns0)
              umma_commit(&q_free);
            else
              mbar_arrive(&q_free);  // no product of this stream read the phase's queries
          }
          ++phase;
        }
        return true;
      });
      // every product and commit is done before the tensor memory is given back
      if (ns > 0 && lane == 0) {
        umma_commit(&all_done[w]);
        mbar_wait(&all_done[w], 0);
      }
    } else if (warp == kTcPvWarp || warp == kTcPvWarp + 1) {
      // ---------------------------------------------------- P V issuers
      const int w = warp - kTcPvWarp;
      const uint32_t ts = tm + uint32_t(w) * 128u, to = ts + 256u;
      const uint64_t vd = make_sdesc_sw128(bs, 16384u, 1024);
      uint32_t tile = 0, ns = 0;
      pieces([&](int, int, int, int ctx, int, int u0, int u1) -> bool {
        const uint32_t ns0 = ns;
        for (int u = u0; u < u1; ++u, ++tile) {
          if (MT == 1 && int(tile & 1) != w) continue;
          const uint32_t ido = u < blk_units ? make_idesc_bf16(kTileM, D, false, true)
                                             : make_idesc_f16(kTileM, D, true);
          const uint32_t vi = 2 * tile + 1, vb = vi % kTcBufs;
          if (!wait(&buf_full[vb], (vi / kTcBufs) & 1, W_V_FULL)) return false;
          const int keys = tile_keys(u, ctx);
          for (int k0 = 0; k0 < keys; k0 += kTcStep, ++ns) {
            const uint32_t b = ns & 1;
            if (!wait(&p_full[w][b], (ns >> 1) & 1, W_P_FULL)) return false;
            tc_fence_after();
            const uint64_t vt = vd + ((vb * kTile + uint32_t(k0) * 128u) >> 4);
            const uint32_t acc = ns > ns0 ? 1u : 0u;
            if (lane == 0) {
#pragma unroll
              for (int ks = 0; ks < kTcStep / 16; ++ks)
                umma_bf16_ts(to, ts + b * 64u + uint32_t(ks) * 8u, vt + uint32_t(ks) * 128u, ido,
                             ks > 0 ? 1u : acc);
              if (u < blk_units) {  // P's second numbers, of the 32-key halves with keys
#pragma unroll 1
                for (int ks = 0; ks < (keys - k0 > 32 ? 4 : 2); ++ks)
                  umma_bf16_ts(to, ts + b * 64u + 32u + uint32_t(ks) * 8u,
                               vt + uint32_t(ks) * 128u, ido, 1u);
              }
              umma_commit(&pv_done[w][b]);
              if (k0 + kTcStep >= keys) umma_commit(&buf_free[vb]);
            }
            __syncwarp();
          }
        }
        if (ns > ns0 && lane == 0) umma_commit(&o_done[w]);
        __syncwarp();
        return true;
      });
      if (ns > 0 && lane == 0) {
        umma_commit(&all_done[2 + w]);
        mbar_wait(&all_done[2 + w], 0);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (threadIdx.x == 0 && failed)
    record_error(err, DEV_TIMEOUT_MMA | DEV_K_KV4_ATTN | (failed << 16));
  tmem_teardown(tm, 512);
}

// ------------------------------------------------------------------- host

template <int D, int MT>
static cudaError_t launch_tc(const Kv4AttnArgs& a, uint32_t* err, cudaStream_t st) {
  const size_t smem = tc_smem(D, MT).total;
  HERALD_CHECK_LAUNCH(ensure_smem(kv4_attn_tc_kernel<D, MT>, smem));
  return launch_k("kv4_attn_tc_kernel", kv4_attn_tc_kernel<D, MT>, dim3(unsigned(a.ctas)),
                  dim3(kTcThreadsAll), smem, st, a, err);
}

cudaError_t launch_kv4_attn_tc(int d, int rows, const Kv4AttnArgs& a, uint32_t* err,
                               cudaStream_t st) {
  if (d == 128) return rows > kTileM ? launch_tc<128, 2>(a, err, st) : launch_tc<128, 1>(a, err, st);
  return rows > kTileM ? launch_tc<64, 2>(a, err, st) : launch_tc<64, 1>(a, err, st);
}

HERALD_DEBUG_WORD_READER(debug_take_kv4_attn_tc)

}  // namespace herald
