// kv4_move.cu -- rows in and out of the paged 4-bit KV cache:
//   append  rotates a block's (or a prompt's) queries and keys by their
//           positions, quantises keys and values and writes them into the
//           sequences' pages
//   pool    the means of the key blocks an append touched (the block-granular
//           stage 1's input), from the rows as the cache holds them
//   gather  held rows at given positions as bf16 (sparse pool, candidates)
#include "kv4.cuh"

namespace herald {

// max of two numbers, NaN if either is one
HERALD_DEV float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// fp32 -> e4m3, to nearest even, past the largest to the largest, NaN stays
HERALD_DEV uint32_t float_to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}
// fp32 pair -> e2m1 codes of one byte (lo in the low half), to nearest even,
// past 6 to 6
HERALD_DEV uint32_t float2_to_e2m1(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// Eight channels of a group of 16 to codes and scale, the other eight in the
// neighbouring lane (a: the max of both).  Each step is one IEEE fp32 operation,
// so the result is defined to the bit: scale = e4m3(max|x| / (6 scale0)), code =
// e2m1(x / S) with S = scale scale0; c6 = 6 scale0.  The quotients are taken
// without dividing: with inv = 1/S rounded, q = x inv is off by an ulp or two,
// x - q S is exact in one fma, and q + (x - q S) inv is then the rounded
// quotient (P. Markstein, IBM J. Res. Dev. 34, 1990).  (The remainder's sign is
// turned so that a negative zero stays one.)  scale0 lies
// in [2^-60, 2^60], so S and 1/S are normal; a group past the largest scale, whose
// quotients may not be, divides.  (Dividing throughout made the prompts' append 7 us
// longer.)
HERALD_DEV void quantise8(const float (&x)[8], float a, float scale0, float c6, uint32_t* codes,
                          uint32_t* scale) {
  *scale = float_to_e4m3(__fdiv_rn(a, c6));
  const float S = __fmul_rn(e4m3_to_float(*scale), scale0);
  uint32_t w = 0;
  if (a < 16.f * S) {
    const float inv = __frcp_rn(S);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float q[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float q0 = __fmul_rn(x[2 * i + j], inv);
        q[j] = __fmaf_rn(__fmaf_rn(q0, S, -x[2 * i + j]), -inv, q0);
      }
      w |= float2_to_e2m1(q[0], q[1]) << (8 * i);
    }
  } else if (S > 0.f) {  // (a zero or NaN scale: codes 0)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w |= float2_to_e2m1(__fdiv_rn(x[2 * i], S), __fdiv_rn(x[2 * i + 1], S)) << (8 * i);
  }
  *codes = w;
}

constexpr int kKv4MoveThreads = 256;

// A row of D channels is handled by D/8 neighbouring lanes, eight channels (16
// bytes) each; an item is one token and Per consecutive heads of its queries, keys
// or values (a chunk).  A CTA holds `toks` = 2^tok_log2 tokens by kRows / toks
// chunks; grid (tokens, sequences, chunks).  Bound by memory for interleaved prompts
// (ragged 4 x 4096 tokens of 32 + 2 x 8 heads: 39 us, 82% of the copy rate; 42 with
// inputs that change from call to call, past L2), by instructions as well for
// half-split ones (50 and 53 us: four shuffles a head, 72 registers for 61), and by
// latency below some hundred tokens.  What counts is that an item loads its heads before it
// works on any, that queries, keys and values do not share warps (one loop over all
// three kinds: 64 us) and that no lane divides for its place.
struct Kv4AppendArgs {
  const uint16_t *q, *k, *v;
  int64_t q_ld, k_ld, v_ld;
  const int32_t *n_tok, *ctx;
  const float* cos_sin;  // [n_pos][rot/2][2]
  int rot;
  uint16_t *q_rot, *k_rot;
  int Hq, Hkv, T, L_max, q_chunks, k_chunks, chunks, tok_log2;
  Kv4Dev c;
};

template <int D, bool Interleaved, int Per>
__global__ void __launch_bounds__(kKv4MoveThreads, 3)
    kv4_append_kernel(const Kv4AppendArgs a) {
  constexpr int LPR = D / 8;
  griddep_enter();
  const int n = blockIdx.y, lane = threadIdx.x & 31, row = threadIdx.x / LPR;
  const int c = lane % LPR;  // this lane's eight channels
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
  const int t = (int(blockIdx.x) << a.tok_log2) + (row & ((1 << a.tok_log2) - 1));
  int chunk = int(blockIdx.z) * ((kKv4MoveThreads / LPR) >> a.tok_log2) + (row >> a.tok_log2);
  const bool live = t < toks && chunk < a.chunks;
  // (a warp without an item leaves whole; the others keep every lane for the
  // exchanges below)
  if (!__any_sync(0xffffffffu, live)) return;
  const int pos = live ? L0 + t : 0;
  const bool is_q = chunk < a.q_chunks;
  if (!is_q) chunk -= a.q_chunks;
  const bool is_k = !is_q && chunk < a.k_chunks;
  if (!is_q && !is_k) chunk -= a.k_chunks;
  const int H = is_q ? a.Hq : a.Hkv, h0 = chunk * Per;
  const int64_t tok = int64_t(n) * a.T + t;

  uint4 u[Per];  // every load of the item first
  {
    const uint16_t* src = (is_q ? a.q + tok * a.q_ld : is_k ? a.k + tok * a.k_ld
                                                            : a.v + tok * a.v_ld) +
                          h0 * D + c * 8;
#pragma unroll
    for (int i = 0; i < Per; ++i)
      u[i] = live && h0 + i < H ? *reinterpret_cast<const uint4*>(src + i * D)
                                : make_uint4(0, 0, 0, 0);
  }
  // angles: in the half-split form channel i < rot/2 pairs with i + rot/2
  // (the same channels of the lane rot/16 lanes on), else 2i pairs with 2i+1
  const bool turns = c * 8 < a.rot && (is_q || is_k);
  const int half = a.rot / 16;  // lanes per half
  const bool first = c < half;
  const int partner = (lane - c) + (c * 8 >= a.rot ? c : first ? c + half : c - half);
  constexpr int A = Interleaved ? 4 : 8;  // angles of a lane
  float cs[A], sn[A];
#pragma unroll
  for (int i = 0; i < A; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (turns) {
    const float* p =
        a.cos_sin + size_t(pos) * a.rot + (Interleaved || first ? c : c - half) * (2 * A);
#pragma unroll
    for (int i = 0; i < A; i += 2) {
      const float4 w = *reinterpret_cast<const float4*>(p + 2 * i);
      cs[i] = w.x, sn[i] = w.y, cs[i + 1] = w.z, sn[i + 1] = w.w;
    }
  }
  int phys = -1;
  if (!is_q && a.c.kc && live) {
    phys = kv4_page(a.c, n, pos >> a.c.page_log2);
    debug_flag(phys < 0, DEV_BAD_INDEX);  // a token without a page
  }
  uint16_t* rot = is_q ? a.q_rot : is_k ? a.k_rot : nullptr;
  if (rot) rot += (tok * H + h0) * D + c * 8;
  const float s0 = is_k ? a.c.k_scale : a.c.v_scale, c6 = __fmul_rn(6.f, s0);
  const size_t held = kv4_row(a.c, max(phys, 0), a.Hkv, h0, pos);
  uint8_t* codes = (is_k ? a.c.kc : a.c.vc) + held * (D / 2) + c * 4;
  uint8_t* scales = (is_k ? a.c.ks : a.c.vs) + held * (D / 16) + c / 2;
#pragma unroll
  for (int i = 0; i < Per; ++i) {
    const bool on = live && h0 + i < H;
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf16lo(w[j]);
      x[2 * j + 1] = bf16hi(w[j]);
    }
    // products and sums rounded one by one, as the definition has them
    if constexpr (Interleaved) {
      if (turns) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = x[2 * j], o = x[2 * j + 1];
          x[2 * j] = __fsub_rn(__fmul_rn(e, cs[j]), __fmul_rn(o, sn[j]));
          x[2 * j + 1] = __fadd_rn(__fmul_rn(o, cs[j]), __fmul_rn(e, sn[j]));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t pw = __shfl_sync(0xffffffffu, w[j], partner);
        if (turns) {
          const float p0 = __fmul_rn(bf16lo(pw), sn[2 * j]),
                      p1 = __fmul_rn(bf16hi(pw), sn[2 * j + 1]);
          const float y0 = __fmul_rn(x[2 * j], cs[2 * j]),
                      y1 = __fmul_rn(x[2 * j + 1], cs[2 * j + 1]);
          x[2 * j] = first ? __fsub_rn(y0, p0) : __fadd_rn(y0, p0);
          x[2 * j + 1] = first ? __fsub_rn(y1, p1) : __fadd_rn(y1, p1);
        }
      }
    }
    if (rot && on)
      *reinterpret_cast<uint4*>(rot + i * D) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                     pack_bf16(x[6], x[7]));
    if (__all_sync(0xffffffffu, is_q)) continue;
    float top = fabsf(x[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) top = max_nan(top, fabsf(x[j]));
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (on && phys >= 0) {
      uint32_t w8, scale;
      quantise8(x, top, s0, c6, &w8, &scale);
      *reinterpret_cast<uint32_t*>(codes + (size_t(i) << a.c.page_log2) * (D / 2)) = w8;
      if (!(c & 1)) scales[(size_t(i) << a.c.page_log2) * (D / 16)] = uint8_t(scale);
    }
  }
}

// grid (blocks, N*Hkv): the means of the blocks that tokens [ctx, ctx + tokens)
// fall into, over the rows below ctx + tokens.  D/16 lanes per row (16 channels
// each), the block's rows dealt over the rest of the CTA; the threads' sums are
// added in a fixed tree.  A row without a page counts as zeros.  (One thread per
// channel walking the rows, a page lookup and two byte loads per row, took 17 us
// for one block of 64; this 3 us.)
template <int D>
__global__ void __launch_bounds__(kKv4MoveThreads)
    kv4_pool_kernel(const Kv4Dev c, const int32_t* __restrict__ ctx,
                    const int32_t* __restrict__ n_tok, int T, int Hkv, int L_max, int Bk,
                    int nb_max, float* __restrict__ pooled) {
  constexpr int LPR = D / 16, RPC = kKv4MoveThreads / LPR;
  __shared__ float sums[RPC][D + 4];
  griddep_enter();
  const int seg = blockIdx.y, n = seg / Hkv, g = seg - n * Hkv;
  const int L0 = min(max(ctx[n], 0), L_max);
  const int end = min(L0 + (n_tok ? min(max(n_tok[n], 0), T) : T), L_max);
  const int b = L0 / Bk + int(blockIdx.x);
  if (end == L0 || b * int64_t(Bk) >= end) return;
  const int r0 = b * Bk, r1 = min(end, r0 + min(Bk, L_max - r0));
  const int ch = threadIdx.x % LPR, rr = threadIdx.x / LPR;
  float acc[16] = {};
  for (int r = r0 + rr; r < r1; r += RPC) {
    const int phys = kv4_page(c, n, r >> c.page_log2);
    if (phys < 0) {
      debug_flag(true, DEV_BAD_INDEX);
      continue;
    }
    const size_t row = kv4_row(c, phys, Hkv, g, r);
    const uint2 w = *reinterpret_cast<const uint2*>(c.kc + row * (D / 2) + ch * 8);
    const float s = e4m3_to_float(c.ks[row * LPR + ch]);
    uint32_t h[8];
    e2m1x8_to_half2(w.x, *reinterpret_cast<uint32_t(*)[4]>(h));
    e2m1x8_to_half2(w.y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      acc[2 * i] += f.x * s;
      acc[2 * i + 1] += f.y * s;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[rr][ch * 16 + i] = acc[i];
  for (int half = RPC / 2; half > 0; half >>= 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < half * D; i += kKv4MoveThreads)
      sums[i / D][i % D] += sums[i / D + half][i % D];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kKv4MoveThreads)
    pooled[(size_t(seg) * nb_max + b) * D + e] = sums[0][e] * c.k_scale / float(r1 - r0);
}

__global__ void kv4_advance_kernel(int32_t* ctx, const int32_t* n_tok, int N, int T, int L_max) {
  griddep_enter();
  const int n = blockIdx.x * blockDim.x + threadIdx.x;
  if (n >= N) return;
  const int L0 = min(max(ctx[n], 0), L_max);
  ctx[n] = min(L0 + min(n_tok ? min(max(n_tok[n], 0), T) : T, L_max - L0), L_max);
}

// grid (row groups, N*Hkv): D/16 lanes per row, each 16 channels: 8 bytes of
// codes and one scale in, 32 bytes of bf16 out.  Bound by its chain of three loads,
// 13 bytes a thread in flight: 32 x 4096 candidate keys 12.9 us, half of the copy rate,
// with inputs that change from call to call, 8.9 where the same 43.5 MB stay in L2;
// 4 x 1344 rows of K and V 3.8 and 2.8.  (Two rows per thread, on data in L2: 9.7 and
// 3.1.)
template <int D>
__global__ void __launch_bounds__(kKv4MoveThreads)
    kv4_gather_kernel(const Kv4Dev c, const int32_t* __restrict__ idx,
                      const int32_t* __restrict__ n_sel, int P_max, int Hkv, int L_max,
                      uint16_t* __restrict__ pk, uint16_t* __restrict__ pv) {
  constexpr int LPR = D / 16, RPC = kKv4MoveThreads / LPR;
  griddep_enter();
  const int seg = blockIdx.y, n = seg / Hkv, g = seg - n * Hkv;
  const int ch = threadIdx.x % LPR, r = blockIdx.x * RPC + threadIdx.x / LPR;
  if (r >= P_max) return;
  const int pos = idx[size_t(seg) * P_max + r];
  const int ns = n_sel[seg];
  debug_flag(ns < 0 || ns > P_max, DEV_BAD_COUNT);
  int phys = -1;
  if (r < ns) {
    if (pos >= 0 && pos < L_max) phys = kv4_page(c, n, pos >> c.page_log2);
    debug_flag(phys < 0, DEV_BAD_INDEX);  // a selected row outside the cache
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint16_t* out = kv ? pv : pk;
    if (!out) continue;
    uint32_t o[8] = {};
    if (phys >= 0) {
      const size_t row = kv4_row(c, phys, Hkv, g, pos);
      const uint2 w = *reinterpret_cast<const uint2*>((kv ? c.vc : c.kc) + row * (D / 2) + ch * 8);
      const float s = e4m3_to_float((kv ? c.vs : c.ks)[row * LPR + ch]);
      const float s0 = kv ? c.v_scale : c.k_scale;
      uint32_t h[8];
      e2m1x8_to_half2(w.x, *reinterpret_cast<uint32_t(*)[4]>(h));
      e2m1x8_to_half2(w.y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        // code * scale is exact; one rounding by s0 in fp32, one to bf16
        o[i] = pack_bf16(f.x * s * s0, f.y * s * s0);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(out + (size_t(seg) * P_max + r) * D + ch * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ------------------------------------------------------------------- host

cudaError_t launch_kv4_append(const herald_dims& dm, int T, const int32_t* n_tok,
                              const uint16_t* q, int64_t q_ld, const uint16_t* k, int64_t k_ld,
                              const uint16_t* v, int64_t v_ld, const herald_rope* rope,
                              int32_t* ctx, const Kv4Dev* cache, uint16_t* q_rot, uint16_t* k_rot,
                              float* pooled, int Bk, bool advance, int num_sms, cudaStream_t st) {
  Kv4AppendArgs a{};
  a.q = q, a.k = k, a.v = v;
  a.q_ld = q_ld, a.k_ld = k_ld, a.v_ld = v_ld;
  a.n_tok = n_tok, a.ctx = ctx;
  if (rope) a.cos_sin = rope->cos_sin, a.rot = rope->rot;
  a.q_rot = q_rot, a.k_rot = k_rot;
  a.Hq = dm.Hq, a.Hkv = dm.Hkv, a.T = T, a.L_max = dm.L_max;
  if (cache) a.c = *cache;
  const int hq = q ? dm.Hq : 0, hk = k ? dm.Hkv : 0, hv = cache ? dm.Hkv : 0;
  const int rpc = kKv4MoveThreads / (dm.d / 8);  // rows per CTA
  const int64_t rows = int64_t(dm.N) * T * (hq + hk + hv);
  // heads per item: 4 share a lane's angles and keep four loads in flight, 1 makes
  // more warps of a small call.  Us with 1 and 4, 48 heads: 1 x 64 tokens 2.5 and
  // 3.7, 256 tokens 3.8 and 4.1, 384 tokens 4.6 and 4.3, 1024 tokens 9.3 and 6.7
  const int per = rows <= int64_t(num_sms) * 6 * rpc ? 1 : 4;
  a.q_chunks = cdiv(hq, per), a.k_chunks = cdiv(hk, per);
  a.chunks = a.q_chunks + a.k_chunks + cdiv(hv, per);
  while ((1 << a.tok_log2) < T && (2 << a.tok_log2) <= rpc) ++a.tok_log2;
  const dim3 grid(unsigned(cdiv(T, 1 << a.tok_log2)), unsigned(dm.N),
                  unsigned(cdiv(a.chunks, rpc >> a.tok_log2)));
  auto pick = [&](auto d, auto il) {
    return per == 1 ? kv4_append_kernel<d.value, il.value, 1>
                    : kv4_append_kernel<d.value, il.value, 4>;
  };
  constexpr std::integral_constant<int, 128> d128{};
  constexpr std::integral_constant<int, 64> d64{};
  const bool il = rope && rope->interleaved;
  auto* kernel = dm.d == 128 ? (il ? pick(d128, std::true_type{}) : pick(d128, std::false_type{}))
                             : (il ? pick(d64, std::true_type{}) : pick(d64, std::false_type{}));
  HERALD_CHECK_LAUNCH(
      launch_k("kv4_append_kernel", kernel, grid, dim3(kKv4MoveThreads), 0, st, a));
  if (pooled) {
    const dim3 pg(unsigned(cdiv(T - 1, Bk) + 1), unsigned(dm.N * dm.Hkv));
    if (dm.d == 128)
      HERALD_CHECK_LAUNCH(launch_k("kv4_pool_kernel", kv4_pool_kernel<128>, pg,
                                   dim3(kKv4MoveThreads), 0, st, *cache, ctx, n_tok, T, dm.Hkv,
                                   dm.L_max, Bk, cdiv(dm.L_max, Bk), pooled));
    else
      HERALD_CHECK_LAUNCH(launch_k("kv4_pool_kernel", kv4_pool_kernel<64>, pg,
                                   dim3(kKv4MoveThreads), 0, st, *cache, ctx, n_tok, T, dm.Hkv,
                                   dm.L_max, Bk, cdiv(dm.L_max, Bk), pooled));
  }
  if (advance)
    HERALD_CHECK_LAUNCH(launch_k("kv4_advance_kernel", kv4_advance_kernel,
                                 dim3(unsigned(cdiv(dm.N, 256))), dim3(256), 0, st, ctx, n_tok,
                                 dm.N, T, dm.L_max));
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const herald_dims& dm, const int32_t* idx, const int32_t* n_sel,
                              int P_max, const Kv4Dev& c, uint16_t* pk, uint16_t* pv,
                              cudaStream_t st) {
  const int rpc = kKv4MoveThreads / (dm.d / 16);
  const dim3 grid(unsigned(cdiv(P_max, rpc)), unsigned(dm.N * dm.Hkv));
  if (dm.d == 128)
    HERALD_CHECK_LAUNCH(launch_k("kv4_gather_kernel", kv4_gather_kernel<128>, grid,
                                 dim3(kKv4MoveThreads), 0, st, c, idx, n_sel, P_max, dm.Hkv,
                                 dm.L_max, pk, pv));
  else
    HERALD_CHECK_LAUNCH(launch_k("kv4_gather_kernel", kv4_gather_kernel<64>, grid,
                                 dim3(kKv4MoveThreads), 0, st, c, idx, n_sel, P_max, dm.Hkv,
                                 dm.L_max, pk, pv));
  return cudaGetLastError();
}

HERALD_DEBUG_WORD_READER(debug_take_kv4_move)

}  // namespace herald
