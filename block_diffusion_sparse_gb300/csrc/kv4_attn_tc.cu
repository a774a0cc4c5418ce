// kv4_attn_tc.cu -- attention over the paged 4-bit cache on the 5th-generation
// tensor cores, for blocks of queries (many rows per KV head).
//
// The tensor cores take fp16 operands from shared memory, so the codes are
// turned into fp16 there (exact, kv4.cuh), once per 128-key tile for up to 256
// query rows.  One CTA per SM walks its share of the keys (kv4_split, units of
// 128 keys, a segment's block keys first):
//   warp 17      copies the codes and scales of a tile's pages into a raw ring
//                (bulk copies; the pages of a tile in parallel lanes)
//   warps 8-15   turn raw items (the K or the V half of a tile) into fp16
//                128-byte-swizzled operand buffers; stage the queries
//   warps 16, 18 one tcgen05.mma issuer per stream: S = Q K^T into the stream's
//                scores, O += P V with P read from tensor memory
//   warps 0-3, 4-7 one softmax warpgroup per stream, a thread per query row
// Two streams, each with 128 TMEM columns of scores (P, fp16, overlays them)
// and 128 of output, run side by side so that one stream's products fill the
// other's softmax: with more than 128 rows a stream is a row tile and takes
// every key tile, else both streams have the same rows and take alternate key
// tiles (their partial outputs are joined like those of two CTAs).
//
// The softmax is optimistic: probabilities are formed with the row's present
// exponent base in the pass that finds the row's maximum, and only a maximum
// more than 15 (log2) above the base repeats the pass after moving the base to
// 11 below it (P stays in fp16's range, see kv4_attn.cu).
//
// The block's own keys are bf16: their tiles come first in a segment, with
// the queries staged as bf16 (an mma's operands have one type), then the
// queries are staged again as fp16 for the cache.
#include <float.h>

#include "kv4.cuh"
#include "tc_common.cuh"

namespace herald {

constexpr int kTcKeys = kKv4TcKeys;        // keys per tile
constexpr int kTcBufs = 4;                 // operand buffers (128 keys of K or V)
constexpr int kTcRaw = 3;                  // raw items
constexpr int kTcMasks = 8;                // tiles whose key masks are kept
constexpr int kTcSoft = 256, kTcConv = 256;  // softmax and conversion threads
constexpr int kTcThreadsAll = 640;         // 8 + 8 + 4 warps (warp 19 only fills its warpgroup)
constexpr int kTcMmaWarp0 = 16, kTcCopyWarp = 17, kTcIdleWarp = 19;  // (18: the other issuer)
constexpr float kTcBelow = 11.f, kTcAbove = 15.f;

// Waits of the kernel (bits 16-31 of the error word).
enum : uint32_t {
  W_RAW_FREE = 1, W_RAW_FULL = 2, W_BUF_FREE = 4, W_Q_FREE = 8, W_Q_FULL = 0x10, W_K_FULL = 0x20,
  W_P_FULL = 0x40, W_V_FULL = 0x80, W_PV_DONE = 0x100, W_S_FULL = 0x200, W_MASK = 0x400,
  W_O_DONE = 0x800
};

// Bounded wait; false when it ran out, or when another wait of the CTA has: a
// role that gets false leaves its loops at once (it touches no barrier and
// starts no copy or product any more), and the kernel returns.
struct TcWait {
  volatile uint32_t* failed;  // shared: the wait that ran out first
  HERALD_DEV bool operator()(uint64_t* bar, uint32_t parity, uint32_t which) const {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
      for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
      if (*failed) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        *failed = which;
        return false;
      }
    }
  }
  // The same answer for a whole warp, which leaves converged: lanes may see a
  // barrier complete in different polls, and the tensor-memory instructions
  // that follow (.sync.aligned) want the warp in one piece.
  HERALD_DEV bool warp(uint64_t* bar, uint32_t parity, uint32_t which) const {
    const bool ok = (*this)(bar, parity, which);
    return __all_sync(0xffffffffu, ok);
  }
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
  s.total = s.raw + uint32_t(kTcRaw) * uint32_t(kTcKeys * (D / 2 + D / 16)) + 1024u;
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
HERALD_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

template <int D, int MT>
__global__ void __launch_bounds__(kTcThreadsAll, 1)
    kv4_attn_tc_kernel(const Kv4AttnArgs a, uint32_t* err) {
  constexpr int H = D / 64;
  constexpr uint32_t kTile = uint32_t(H) * 16384u;
  constexpr int kRowC = D / 2, kRowS = D / 16;           // raw bytes of a row
  constexpr uint32_t kRawBytes = kTcKeys * (kRowC + kRowS);
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t raw_full[kTcRaw], raw_free[kTcRaw], buf_full[kTcBufs], buf_free[kTcBufs];
  __shared__ uint64_t q_full, q_free, s_full[2], p_full[2], pv_done[2], all_done[2], mask_full[kTcMasks];
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t failed;
  __shared__ float row_f[2 * kTileM];               // score factors of the rows (cache tiles)
  __shared__ uint32_t key_mask[kTcMasks][4];        // bit: the key counts
  const TcSmem L = tc_smem(D, MT);
  uint8_t* base = align1024(smem_raw);
  uint8_t *Qs = base + L.q, *Bs = base + L.buf, *Rs = base + L.raw;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTcRaw; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_free[i], 8);
    for (int i = 0; i < kTcBufs; ++i) mbar_init(&buf_full[i], 8), mbar_init(&buf_free[i], MT);
    for (int i = 0; i < kTcMasks; ++i) mbar_init(&mask_full[i], 1);
    mbar_init(&q_full, 8);
    mbar_init(&q_free, 2 + kTcSoft);
    for (int i = 0; i < 2; ++i)
      mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 128), mbar_init(&pv_done[i], 1),
          mbar_init(&all_done[i], 1);
    failed = 0;
    fence_mbar_init();
  }
  tmem_setup(&tmem_base, 512);
  const uint32_t tm = tmem_base;
  griddep_enter();
  const TcWait wait{&failed};

  const int G = a.Hq / a.Hkv, R = a.B * G;
  const int blk_units = a.bk ? (a.B + kTcKeys - 1) / kTcKeys : 0;
  const Kv4Split split = kv4_split(kv4_total_units(a.ctx, a.N, a.L_max, kTcKeys, blk_units), a.Hkv,
                                   a.ctas, 1);
  const int64_t at0 = int64_t(blockIdx.x) * split.share;
  const int64_t end = min(at0 + split.share, split.total);
  int n_first = 0;
  int64_t first0 = 0;
  if (at0 < end) kv4_find(a.ctx, a.N, a.L_max, kTcKeys, blk_units, a.Hkv, at0, &n_first, &first0);

  // Every role walks the same pieces: body(n, g, seg, ctx, units, u0, u1) with
  // tiles u0 <= u < u1 of the segment, the first blk_units of them block tiles;
  // it returns false to leave (a wait ran out).
  auto pieces = [&](auto&& body) {
    int64_t at = at0, first = first0;
    int n = n_first;
    while (at < end) {
      const int ctx = min(max(a.ctx[n], 0), a.L_max);
      const int units = kv4_units(ctx, a.L_max, kTcKeys, blk_units);
      if (units == 0 || at >= first + int64_t(a.Hkv) * units) {
        first += int64_t(a.Hkv) * units;
        ++n;
        continue;
      }
      const int g = int((at - first) / units);
      const int64_t seg0 = first + int64_t(g) * units;
      const int u0 = int(at - seg0), u1 = int(min(int64_t(units), end - seg0));
      if (!body(n, g, n * a.Hkv + g, ctx, units, u0, u1)) return;
      at = seg0 + u1;
    }
  };

  // registers: 640 threads launch with 96 each (61,440); 256 x 120 + 256 x 80 +
  // 128 x 64 = 59,392.  Each role's branch begins with its own setmaxnreg, so
  // that the compiler knows the limit of the code that follows.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2;                  // stream
    const int lrow = (warp & 3) * 32 + lane;  // TMEM lane
    const int row = (MT == 2 ? w * kTileM : 0) + lrow;
    const bool idle = (MT == 2 ? w * kTileM : 0) + (warp & 3) * 32 >= R;  // the warp has no rows
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t ts = tm + lanes + uint32_t(w) * 128u, to = tm + lanes + 256u + uint32_t(w) * 128u;
    uint32_t tile = 0, ns = 0, mt = 0, phase = 0;  // tiles of the CTA, of this stream, masks
    pieces([&](int n, int g, int seg, int ctx, int units, int u0, int u1) -> bool {
      debug_flag(threadIdx.x == 0 && a.ctx[n] != ctx, DEV_BAD_COUNT);
      float m = -FLT_MAX, l = 0.f;
      bool any = false;  // this stream has had a tile of the piece
      int u = u0;
      while (u < u1) {  // a phase: block tiles, or cache tiles
        const bool blk = u < blk_units;
        const int pe = blk ? min(u1, blk_units) : u1;
        // the phase's queries are staged (so this stream's arrivals on q_free
        // below never run into an earlier phase, with or without tiles here)
        if (!wait.warp(&q_full, phase & 1, W_Q_FULL)) return false;
        const float f = blk ? fminf(a.scale * 1.4426950408889634f, FLT_MAX)
                            : *(volatile float*)&row_f[row];
        for (; u < pe; ++u, ++tile) {
          const uint32_t mask_no = mt;
          if (!blk) ++mt;
          if (MT == 1 && int(tile & 1) != w) continue;
          if (!wait.warp(&s_full[w], ns & 1, W_S_FULL)) return false;
          tc_fence_after();
          uint32_t msk[4] = {~0u, ~0u, ~0u, ~0u};
          if (!blk) {
            const uint32_t i = mask_no % kTcMasks;
            if (!wait.warp(&mask_full[i], (mask_no / kTcMasks) & 1, W_MASK)) return false;
#pragma unroll
            for (int c = 0; c < 4; ++c) msk[c] = *(volatile uint32_t*)&key_mask[i][c];
          } else {
            const int nk = a.B - u * kTcKeys;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              msk[c] = nk >= 32 * c + 32 ? ~0u : nk <= 32 * c ? 0u : (1u << (nk - 32 * c)) - 1u;
          }
          const bool part = (msk[0] & msk[1] & msk[2] & msk[3]) != ~0u;
          if (!idle) {
            uint32_t pk[64];
            while (true) {
              float mx = -INFINITY;
              uint64_t sum2 = f2_pack(0.f, 0.f);
              const uint64_t f2 = f2_pack(f, f), nm2 = f2_pack(-m, -m);
              const float iv = 1.f / a.c.v_scale;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t r[32];
                tmem_ld32_nowait(ts + uint32_t(c) * 32u, r);
                tmem_wait_ld();
                if (part) {
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (!(msk[c] >> i & 1)) r[i] = __float_as_uint(-INFINITY);
                }
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                  mx = fmax3f(mx, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float x0, x1;
                  f2_unpack(f2_fma(f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                                   f2, nm2),
                            x0, x1);
                  const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                  sum2 = f2_add(sum2, f2_pack(p0, p1));
                  // (block tiles: P in units of v_scale, O has one unit for all keys)
                  pk[c * 16 + i] = blk ? pack_bf16(p0 * iv, p1 * iv) : pack_half2(p0, p1);
                }
              }
              const bool move = mx * f - m > kTcAbove;
              if (!__any_sync(0xffffffffu, move)) {
                float s0, s1;
                f2_unpack(sum2, s0, s1);
                l += s0 + s1;
                break;
              }
              float k = 1.f;
              if (move) {
                const float b = mx * f - kTcBelow;
                k = fast_exp2(m - b);
                m = b;
                l *= k;
              }
              __syncwarp();
              if (any) {  // (every earlier P V of the stream is done: S was issued after it)
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                  uint32_t r[32];
                  tmem_ld32_nowait(to + uint32_t(c) * 32u, r);
                  tmem_wait_ld();
                  float v[32];
#pragma unroll
                  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * k;
                  tmem_st32(to + uint32_t(c) * 32u, v);
                }
                tmem_wait_st();
              }
            }
            {
              float v[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(pk[i]);
              tmem_st32(ts, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(pk[32 + i]);
              tmem_st32(ts + 32u, v);
              tmem_wait_st();
            }
          }
          tc_fence_before();
          mbar_arrive(&p_full[w]);
          any = true;
          ++ns;
        }
        mbar_arrive(&q_free);  // (this thread has read its factor of the phase)
        ++phase;
      }
      // the piece's rows: O once the last P V is done
      if (any) {
        if (!wait.warp(&pv_done[w], (ns - 1) & 1, W_O_DONE)) return false;
        tc_fence_after();
      }
      if (!idle) {
        const bool whole = MT == 2 && u0 == 0 && u1 == units;
        const float inv = l == 0.f ? 0.f : a.c.v_scale / l;
        const int slot = MT == 2 ? int(blockIdx.x) + seg : 2 * (int(blockIdx.x) + seg) + w;
        const bool on = row < R;
        float* part = a.opart + (size_t(slot) * a.R16 + row) * D;
        uint16_t* out =
            a.out + ((size_t(n) * a.B + (on ? row / G : 0)) * a.Hq + g * G + (on ? row % G : 0)) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          if (any) {
            tmem_ld32_nowait(to + uint32_t(c) * 32u, r);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0;
          }
          if (on && whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(out + c * 32 + i) = make_uint4(
                  pack_bf16(__uint_as_float(r[i]) * inv, __uint_as_float(r[i + 1]) * inv),
                  pack_bf16(__uint_as_float(r[i + 2]) * inv, __uint_as_float(r[i + 3]) * inv),
                  pack_bf16(__uint_as_float(r[i + 4]) * inv, __uint_as_float(r[i + 5]) * inv),
                  pack_bf16(__uint_as_float(r[i + 6]) * inv, __uint_as_float(r[i + 7]) * inv));
          } else if (on) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(part + c * 32 + i) =
                  make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
          }
          __syncwarp();
        }
        if (on && !whole) a.ml[size_t(slot) * a.R16 + row] = make_float2(m, l);
        __syncwarp();
        tc_fence_before();
      }
      return true;
    });
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // --------------------------------------- queries, operand conversion
    const int ct = threadIdx.x - kTcSoft, cw = warp - 8;
    uint32_t item = 0, raw_no = 0, mt = 0, phase = 0;
    auto publish = [&](uint64_t* bar) {  // this warp's writes are ready for the tensor cores
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    pieces([&](int n, int g, int, int ctx, int, int u0, int u1) -> bool {
      (void)ctx;
      int u = u0;
      while (u < u1) {
        const bool blk = u < blk_units;
        const int pe = blk ? min(u1, blk_units) : u1;
        if (phase > 0 && !wait.warp(&q_free, (phase - 1) & 1, W_Q_FREE)) return false;
        // queries: D/16 lanes per row, 16 channels each
        constexpr int LPR = D / 16;
        for (int r0 = ct / LPR; r0 < MT * kTileM; r0 += kTcConv / LPR) {
          const int c = ct % LPR;
          uint32_t x[8] = {};
          if (r0 < R) {
            const uint4* src = reinterpret_cast<const uint4*>(
                a.q + ((size_t(n) * a.B + r0 / G) * a.Hq + g * G + r0 % G) * D + c * 16);
            const uint4 x0 = src[0], x1 = src[1];
            x[0] = x0.x, x[1] = x0.y, x[2] = x0.z, x[3] = x0.w;
            x[4] = x1.x, x[5] = x1.y, x[6] = x1.z, x[7] = x1.w;
          }
          if (!blk) {  // fp16 scaled per row by a power of two (see kv4_attn.cu)
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mx = fmaxf(mx, fmaxf(fabsf(bf16lo(x[i])), fabsf(bf16hi(x[i]))));
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            float up, f;
            kv4_query_scale(mx, a.scale * a.c.k_scale, &up, &f);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = pack_half2(bf16lo(x[i]) * up, bf16hi(x[i]) * up);
            if (c == 0) row_f[r0] = f;
          }
          uint8_t* dst = Qs + uint32_t(r0 / kTileM) * kTile + uint32_t(c >> 2) * 16384u;
          const uint32_t rr = uint32_t(r0 % kTileM), c8 = uint32_t(c & 3) * 2u;
          *reinterpret_cast<uint4*>(dst + sw128_off(rr, c8)) = make_uint4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<uint4*>(dst + sw128_off(rr, c8 + 1)) =
              make_uint4(x[4], x[5], x[6], x[7]);
        }
        publish(&q_full);
        ++phase;
        for (; u < pe; ++u) {
          const uint32_t mask_no = mt;
          if (!blk) ++mt;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++item) {
            const uint32_t b = item % kTcBufs;
            if (item >= uint32_t(kTcBufs) &&
                !wait.warp(&buf_free[b], (item / kTcBufs - 1) & 1, W_BUF_FREE))
              return false;
            uint8_t* dst = Bs + b * kTile;
            if (blk) {  // bf16 rows of the block, zeros after them
              const uint16_t* src = kv ? a.bv : a.bk;
              constexpr int CPR = D / 8;  // 16-byte chunks of a row
#pragma unroll 4
              for (int i = ct; i < kTcKeys * CPR; i += kTcConv) {
                const int r = i / CPR, c = i % CPR, j = u * kTcKeys + r;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (j < a.B)
                  v = *reinterpret_cast<const uint4*>(
                      src + ((size_t(n) * a.B + j) * a.Hkv + g) * D + c * 8);
                *reinterpret_cast<uint4*>(dst + uint32_t(c >> 3) * 16384u +
                                          sw128_off(uint32_t(r), uint32_t(c & 7))) = v;
              }
            } else {
              const uint32_t rb = raw_no % kTcRaw;
              if (!wait.warp(&raw_full[rb], (raw_no / kTcRaw) & 1, W_RAW_FULL)) return false;
              const uint8_t* rc = Rs + rb * kRawBytes;
              const uint8_t* rsc = rc + kTcKeys * kRowC;
              // A lane turns chunks of 16 bytes (32 channels): chunk j of row
              // r.  Rows and chunks are dealt so that the eight lanes of a
              // shared-memory phase read eight different 16-byte bank groups
              // ((r&1)*4 + j for d = 128, (r&3)*2 + j for 64) and write eight
              // (the swizzle's XOR of r&7 with the chunk).
              constexpr int kTasks = kTcKeys * (kRowC / 16) / kTcConv;
#pragma unroll
              for (int s = 0; s < kTasks; ++s) {
                int r, j;
                if constexpr (D == 128) {
                  const int j1 = (lane >> 2) & 1;
                  j = ((lane >> 1) & 1) + 2 * j1;
                  r = cw * 16 + (lane >> 3) * 4 + (lane & 1) + 2 * (j1 ^ s);
                } else {
                  j = lane & 1;
                  r = cw * 16 + (lane >> 1);
                }
                const uint4 cw4 = *reinterpret_cast<const uint4*>(rc + r * kRowC + j * 16);
                uint32_t sc = *reinterpret_cast<const uint16_t*>(rsc + r * kRowS + j * 2);
                // a value row that does not count may hold any bytes: 0 * NaN must not arise
                if (kv && !(*(volatile uint32_t*)&key_mask[mask_no % kTcMasks][r >> 5] >> (r & 31) & 1))
                  sc = 0;
                const uint32_t s2 = e4m3x2_to_half2(sc);
                const uint32_t words[4] = {cw4.x, cw4.y, cw4.z, cw4.w};
                uint8_t* half = dst + uint32_t(D == 128 ? j >> 1 : 0) * 16384u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  uint32_t h[4];
                  e2m1x8_to_half2(words[k], h);
                  const uint32_t fs = __byte_perm(s2, 0, k < 2 ? 0x1010 : 0x3232);
#pragma unroll
                  for (int i = 0; i < 4; ++i) h[i] = hmul2(h[i], fs);
                  *reinterpret_cast<uint4*>(half + sw128_off(uint32_t(r), uint32_t((j & 1) * 4 + k))) =
                      make_uint4(h[0], h[1], h[2], h[3]);
                }
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&raw_free[rb]);
              ++raw_no;
            }
            publish(&buf_full[b]);
          }
        }
      }
      return true;
    });
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == kTcCopyWarp) {
      // ------------------------------------------------------- raw copies
      uint32_t raw_no = 0, mt = 0;
      pieces([&](int n, int g, int, int ctx, int, int u0, int u1) -> bool {
        const int sub = min(1 << a.c.page_log2, kTcKeys);  // keys of a tile in one page
        for (int u = max(u0, blk_units); u < u1; ++u, ++mt) {
          // lane i: the tile's sub-chunk i
          const int k0 = lane * sub, pos = (u - blk_units) * kTcKeys + k0;
          int keys = 0, phys = -1;
          if (k0 < kTcKeys && pos < ctx) {
            phys = kv4_page(a.c, n, pos >> a.c.page_log2);
            debug_flag(phys < 0, DEV_BAD_INDEX);
            if (phys >= 0) keys = min(sub, ctx - pos);
          }
          const size_t row = phys >= 0 ? kv4_row(a.c, phys, a.Hkv, g, pos) : 0;
          const uint32_t rows = uint32_t(keys + 15) & ~15u;  // whole groups of 16: inside the page
          uint32_t total = rows;
  #pragma unroll
          for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  #pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++raw_no) {
            const uint32_t rb = raw_no % kTcRaw;
            if (raw_no >= uint32_t(kTcRaw) &&
                !wait.warp(&raw_free[rb], (raw_no / kTcRaw - 1) & 1, W_RAW_FREE))
              return false;
            if (kv == 0) {
              // (the masks of kTcMasks tiles back have been read: their V item
              // has left the operand ring, which is shorter)
              if (k0 < kTcKeys)
                for (int i = 0; i < sub / 16; ++i) {
                  const int v = min(max(keys - 16 * i, 0), 16);
                  reinterpret_cast<volatile uint16_t*>(key_mask[mt % kTcMasks])[k0 / 16 + i] =
                      uint16_t((1u << v) - 1u);
                }
              __syncwarp();
              if (lane == 0) mbar_arrive(&mask_full[mt % kTcMasks]);
            }
            if (lane == 0) mbar_arrive_expect_tx(&raw_full[rb], total * uint32_t(kRowC + kRowS));
            __syncwarp();
            if (rows) {
              uint8_t* dst = Rs + rb * kRawBytes;
              bulk_load(dst + k0 * kRowC, (kv ? a.c.vc : a.c.kc) + row * kRowC, rows * kRowC,
                        &raw_full[rb]);
              bulk_load(dst + kTcKeys * kRowC + k0 * kRowS, (kv ? a.c.vs : a.c.ks) + row * kRowS,
                        rows * kRowS, &raw_full[rb]);
            }
          }
        }
        return true;
      });
      // every copy has landed before the CTA may leave (only after a failed
      // wait can one still be under way)
      if (*(volatile uint32_t*)&failed)
        for (uint32_t i = raw_no > uint32_t(kTcRaw) ? raw_no - kTcRaw : 0; i < raw_no; ++i)
          mbar_wait(&raw_full[i % kTcRaw], (i / kTcRaw) & 1);
    } else if (warp != kTcIdleWarp && lane == 0) {
      // ------------------------------------------------------ MMA issuers
      const int w = warp == kTcMmaWarp0 ? 0 : 1;
      const uint32_t ts = tm + uint32_t(w) * 128u, to = tm + 256u + uint32_t(w) * 128u;
      const uint32_t qa = smem_u32(Qs) + (MT == 2 ? uint32_t(w) * kTile : 0u);
      const uint32_t ba = smem_u32(Bs);
      uint32_t tile = 0, ns = 0, phase = 0;
      bool issued = false;
      pieces([&](int, int, int, int, int, int u0, int u1) -> bool {
        bool any = false;
        int u = u0;
        while (u < u1) {
          const bool blk = u < blk_units;
          const int pe = blk ? min(u1, blk_units) : u1;
          const uint32_t ids =
              blk ? make_idesc_bf16(kTileM, kTcKeys, false, false) : make_idesc_f16(kTileM, kTcKeys, false);
          const uint32_t ido = blk ? make_idesc_bf16(kTileM, D, false, true) : make_idesc_f16(kTileM, D, true);
          if (!wait(&q_full, phase & 1, W_Q_FULL)) return false;
          const uint32_t ns0 = ns;
          for (; u < pe; ++u, ++tile) {
            if (MT == 1 && int(tile & 1) != w) continue;
            const uint32_t ki = 2 * tile, vi = ki + 1, kb = ki % kTcBufs, vb = vi % kTcBufs;
            if (!wait(&buf_full[kb], (ki / kTcBufs) & 1, W_K_FULL)) return false;
            // P of the stream's previous tile has been read
            if (ns > 0 && !wait(&pv_done[w], (ns - 1) & 1, W_PV_DONE)) return false;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = uint32_t(ks >> 2) * 16384u + uint32_t(ks & 3) * 32u;
              umma_bf16(ts, make_sdesc_sw128(qa + off, 16, 1024),
                        make_sdesc_sw128(ba + kb * kTile + off, 16, 1024), ids, ks > 0 ? 1u : 0u);
            }
            issued = true;
            umma_commit(&s_full[w]);
            umma_commit(&buf_free[kb]);
            if (!wait(&p_full[w], ns & 1, W_P_FULL)) return false;
            if (!wait(&buf_full[vb], (vi / kTcBufs) & 1, W_V_FULL)) return false;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < kTcKeys / 16; ++ks)
              umma_bf16_ts(to, ts + uint32_t(ks) * 8u,
                           make_sdesc_sw128(ba + vb * kTile + uint32_t(ks) * 2048u, 16384u, 1024),
                           ido, any || ks > 0 ? 1u : 0u);
            umma_commit(&pv_done[w]);
            umma_commit(&buf_free[vb]);
            any = true;
            ++ns;
          }
          if (ns > ns0)
            umma_commit(&q_free);
          else
            mbar_arrive(&q_free);  // no product of this stream read the phase's queries
          ++phase;
        }
        return true;
      });
      // every product and commit is done before the tensor memory is given back
      if (issued) {
        umma_commit(&all_done[w]);
        mbar_wait(&all_done[w], 0);
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
