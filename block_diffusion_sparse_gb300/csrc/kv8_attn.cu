// kv8_attn.cu -- attention of a block's queries over the whole paged 8-bit cache and
// the block's own bf16 keys: a kernel for few or many query rows (kv8_rows.cu,
// kv8_attn_tc.cu) writes partial results over the cache's keys (m, l, O per query row
// and piece of a segment), the join here adds the block's own keys and writes the output.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "kv8.cuh"

namespace herald {

// What a piece costs beside its tiles, in tiles (kv4_units): its first scores, its first base
// and its partials.  Few rows, with 0 / 1 / 2 / 3 / 4: 64 ragged sequences of up to 8K tokens
// 97.5 / 95.2 / 94.6 / 93.7 / 94.3 us, 16 of them with 4 tokens each 35.4 / 29.7 / 27.0 / 26.1 /
// 25.9, one of 128K (whose pieces are long) 46.3 / 46.0 / 46.0 / 46.8 / 47.1.  Many, with 5 / 6 / 7 /
// 8: seven ragged drafts of 35 rows 21.0 / 20.7 / 21.0 / 21.6, 16 ragged sequences of 32 rows 35.1 /
// 34.3 / 34.4 / 35.1, 64 of 128 rows 184 / 176 / 172 / 168, a block of 224 rows over 32K 24.7 to 24.9.
constexpr int kKv8PadRows = 3, kKv8PadTc = 7;
constexpr int kKv8MaxCtas = 304;  // most attention CTAs (workspace slots)

HERALD_DEV void join_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int Words>
HERALD_DEV void load_run(const uint16_t* p, bool on, uint32_t (&w)[Words]) {
#pragma unroll
  for (int i = 0; i < Words; i += 4) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (on) x = *reinterpret_cast<const uint4*>(p + 2 * i);
    w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
  }
}

// Whether one of two bf16 is an infinity or a NaN shows in a sum of 0 * x: t stays 0 (of
// either sign) as long as none is.
HERALD_DEV uint32_t zero_times(uint32_t w, uint32_t t) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(t) : "r"(w), "r"(0u));
  return t;
}
HERALD_DEV uint32_t finite_or_zero(uint32_t w) {  // (of two bf16)
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

// The block's own keys in the join: up to kOwnWarps warps take 16 keys at a time, for 16
// query rows (mma m16n8k16 of bf16, fp32 sums; P as two bf16 numbers, take_bf16), and
// leave (m, l, O) in shared memory.  The contraction's channels may stand in any order
// that both operands share, so a lane's share of a row is a run of channels: q and k
// [t D/4, (t+1) D/4) of lane t = lane%4, v [g D/8, (g+1) D/8) of lane group g = lane/4,
// whose n-th channel goes to column g of the product's n-th tile.
// A weight's second number may be 0 or negative, and times an infinite value that is a NaN or
// the other infinity where the weight times it is not: infinities and NaNs are left to
// the first number alone (positive, or 0 where the weight is).
constexpr int kOwnWarps = 4;
template <int D>
struct OwnKeys {
  static constexpr int kPitch = D / 32 * 36;  // (four floats after 32: runs meet all banks)
  float o[kOwnWarps][16][kPitch];
  float m[kOwnWarps][16], l[kOwnWarps][16];
};
template <int D>
HERALD_DEV void own_keys(const Kv8AttnArgs& a, OwnKeys<D>& sm, int n, int g, int r0, int warp,
                         int lane) {
  constexpr int KW = D / 8, VW = D / 16;  // words of a lane's run
  const int G = a.Hq / a.Hkv, R = a.B * G, lg = lane >> 2, lt = lane & 3;
  uint32_t q[2][KW];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = min(r0 + lg + 8 * i, R - 1);
    load_run<KW>(a.q + ((size_t(n) * a.B + r / G) * a.Hq + g * G + r % G) * D + lt * (D / 4), true,
                 q[i]);
  }
  float m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f};
#pragma unroll 1
  for (int k0 = warp * 16; k0 < a.B; k0 += kOwnWarps * 16) {
    const size_t ld = size_t(a.Hkv) * D, at = (size_t(n) * a.B + k0) * ld + size_t(g) * D;
    uint32_t v[4][VW];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 2 * lt + (i & 1) + 8 * (i >> 1);
      load_run<VW>(a.bv + at + j * ld + lg * (D / 8), k0 + j < a.B, v[i]);
    }
    float s[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t k[KW];
      load_run<KW>(a.bk + at + (lg + 8 * h) * ld + lt * (D / 4), k0 + lg + 8 * h < a.B, k);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[h][i] = 0.f;
#pragma unroll
      for (int i = 0; i < KW; i += 2)
        join_mma(s[h], q[0][i], q[1][i], q[0][i + 1], q[1][i + 1], k[i], k[i + 1]);
    }
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // rows lg, lg + 8: scores 2 i, 2 i + 1 of each half
      float mx = m[i];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = s[h][2 * i + e];
          x = k0 + 8 * h + 2 * lt + e < a.B ? x * a.scale : -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      f[i] = fast_exp2(m[i] - mx);
      m[i] = mx;
      l[i] *= f[i];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[h][2 * i + e] = fast_exp2(s[h][2 * i + e] - mx);
          l[i] += s[h][2 * i + e];
        }
    }
    uint32_t p[2][4];
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) p[part][2 * h + i] = take_bf16(s[h][2 * i], s[h][2 * i + 1]);
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < VW; ++j) t = zero_times(v[i][j], t);
    const bool odd = __any_sync(0xffffffffu, (t & 0x7FFF7FFFu) != 0);
    auto values = [&](auto odd_c) {
      constexpr bool Odd = decltype(odd_c)::value;
#pragma unroll
      for (int c = 0; c < VW; c += 2) {  // four channels of a run: four tiles
        float o[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = c + j / 2;
          const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
          uint32_t b0 = __byte_perm(v[0][i], v[1][i], sel), b1 = __byte_perm(v[2][i], v[3][i], sel);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
          join_mma(o[j], p[0][0], p[0][1], p[0][2], p[0][3], b0, b1);
          if constexpr (Odd) b0 = finite_or_zero(b0), b1 = finite_or_zero(b1);
          join_mma(o[j], p[1][0], p[1][1], p[1][2], p[1][3], b0, b1);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // row lg + 8 (e >> 1), run 2 lt + (e & 1)
          const int ch = (2 * lt + (e & 1)) * (D / 8) + 2 * c;
          float4* dst = reinterpret_cast<float4*>(&sm.o[warp][lg + 8 * (e >> 1)][ch + ch / 32 * 4]);
          float4 x = make_float4(o[0][e], o[1][e], o[2][e], o[3][e]);
          if (k0 >= kOwnWarps * 16) {
            const float4 y = *dst;
            const float w = f[e >> 1];
            x.x = fmaf(y.x, w, x.x), x.y = fmaf(y.y, w, x.y), x.z = fmaf(y.z, w, x.z), x.w = fmaf(y.w, w, x.w);
          }
          *dst = x;
        }
      }
    };
    if (odd)
      values(std::true_type{});
    else
      values(std::false_type{});
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (lt == 0) sm.m[warp][lg + 8 * i] = m[i], sm.l[warp][lg + 8 * i] = l[i];
  }
}

// The output: the pieces of a segment joined, with the block's own keys.  grid (N*Hkv,
// ceil(R / Rows)); D/4 lanes hold a row's channels, four each, a thread has Per rows, and
// GR groups of threads share the pieces: each takes every such-and-suchth, kFly rows'
// worth in flight; the groups are then added in order.  The block's keys come before the
// grid-dependency wait: they and the lengths were written before the attention
// kernel's own wait ended, and it lets this kernel start only after that.  Few of them
// (not Tc) are taken one after another by the row's lanes, every load first.
// (64 sequences of one token: 105 us by lanes and 110 by products, when the whole took that.)
constexpr int kOwnFew = 4;  // block keys at most that the lanes take
template <int D, int Rows, int Per, int GR, bool Tc>
__global__ void __launch_bounds__(D / 4 * Rows / Per * GR, Tc && GR == 1 ? 2 : 1)
    kv8_join_kernel(const Kv8AttnArgs a) {
  constexpr int TPR = D / 4, RS = Rows / Per;  // rows side by side
  static_assert(!Tc || TPR * RS * GR > 32 * kOwnWarps || GR == 1, "warps of the block's keys");
  __shared__ OwnKeys<Tc ? D : 32> own;
  __shared__ float4 part[GR][GR > 1 ? Rows : 1][TPR];
  __shared__ float part_m[GR][Rows], part_l[GR][Rows];
  __shared__ int pieces[2];
  const int seg = blockIdx.x, n = seg / a.Hkv, g = seg - n * a.Hkv;
  const int G = a.Hq / a.Hkv, R = a.B * G;
  const int c4 = threadIdx.x % TPR, rr = threadIdx.x / TPR % RS, grp = threadIdx.x / (TPR * RS);
  const int r0 = int(blockIdx.y) * Rows, warp = warp_same(int(threadIdx.x) >> 5);
  // (the rows of a CTA lie in one row tile: Rows divides 128)
  const int heads = a.Hkv * a.row_tiles, tile = r0 / a.R16;
  if (warp == int(blockDim.x) / 32 - 1) {  // slots of the segment's pieces
    const Kv4Split split = kv4_split(kv4_total_units(a.ctx, a.N, a.L_max, 0, a.pad), heads, a.ctas);
    const int units = kv4_units(a.ctx[n], a.L_max, 0, a.pad), gt = g * a.row_tiles + tile;
    const int first = heads * kv4_total_units(a.ctx, n, a.L_max, 0, a.pad) + gt * units;
    if ((threadIdx.x & 31) == 0) {
      pieces[0] = units > 0 ? (first + a.pad) / split.share + n * heads + gt : 0;
      pieces[1] = units > 0 ? (first + units - 1) / split.share + n * heads + gt : -1;
    }
  }
  float M[Per], L[Per];
  float4 acc[Per];
#pragma unroll
  for (int e = 0; e < Per; ++e) M[e] = -FLT_MAX, L[e] = 0.f, acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (Tc) {
    if (a.bk && warp < kOwnWarps) own_keys<D>(a, own, n, g, r0, warp, threadIdx.x & 31);
  } else if (a.bk) {
    static_assert(Per == 1, "one row a thread");
    const int r = min(r0 + rr, R - 1);
    const uint2 qw = *reinterpret_cast<const uint2*>(
        a.q + ((size_t(n) * a.B + r / G) * a.Hq + g * G + r % G) * D + c4 * 4);
    uint2 kw[kOwnFew], vw[kOwnFew];
#pragma unroll
    for (int j = 0; j < kOwnFew; ++j) {
      const size_t at = ((size_t(n) * a.B + min(j, a.B - 1)) * a.Hkv + g) * D + c4 * 4;
      kw[j] = *reinterpret_cast<const uint2*>(a.bk + at);
      vw[j] = *reinterpret_cast<const uint2*>(a.bv + at);
    }
    float s[kOwnFew];
#pragma unroll
    for (int j = 0; j < kOwnFew; ++j)
      s[j] = fmaf(bf16lo(qw.x), bf16lo(kw[j].x), bf16hi(qw.x) * bf16hi(kw[j].x)) +
             fmaf(bf16lo(qw.y), bf16lo(kw[j].y), bf16hi(qw.y) * bf16hi(kw[j].y));
#pragma unroll
    for (int o = 1; o < TPR; o <<= 1)
#pragma unroll
      for (int j = 0; j < kOwnFew; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
    if (grp == 0) {
#pragma unroll
      for (int j = 0; j < kOwnFew; ++j) {
        s[j] = j < a.B ? s[j] * a.scale : -INFINITY;
        M[0] = fmaxf(M[0], s[j]);
      }
#pragma unroll
      for (int j = 0; j < kOwnFew; ++j) {
        const float p = fast_exp2(s[j] - M[0]);
        if (j >= a.B) break;
        L[0] += p;
        acc[0].x = fmaf(p, bf16lo(vw[j].x), acc[0].x), acc[0].y = fmaf(p, bf16hi(vw[j].x), acc[0].y);
        acc[0].z = fmaf(p, bf16lo(vw[j].y), acc[0].z), acc[0].w = fmaf(p, bf16hi(vw[j].y), acc[0].w);
      }
    }
  }
  __syncthreads();
  const int c0 = pieces[0], c1 = pieces[1];
  if constexpr (Tc) {
    if (a.bk && grp == 0) {
      const int with = min(kOwnWarps, (a.B + 15) / 16);
#pragma unroll
      for (int e = 0; e < Per; ++e) {
        const int r = rr + e * RS;
        for (int i = 0; i < with; ++i) M[e] = fmaxf(M[e], own.m[i][r]);
        for (int i = 0; i < with; ++i) {
          const float f = fast_exp2(own.m[i][r] - M[e]);
          const float4 x = *reinterpret_cast<const float4*>(&own.o[i][r][c4 * 4 + c4 / 8 * 4]);
          L[e] += f * own.l[i][r];
          acc[e].x += f * x.x, acc[e].y += f * x.y, acc[e].z += f * x.z, acc[e].w += f * x.w;
        }
      }
    }
  }
  griddep_enter();
  {
    const int rt = r0 - tile * a.R16 + rr, top = min(a.R16, R - tile * a.R16) - 1;
    constexpr int kFly = Per > 1 ? 3 : 5;
    for (int c = c0 + grp; c <= c1; c += kFly * GR) {
      float2 p[kFly][Per];
      float4 x[kFly][Per];
#pragma unroll
      for (int i = 0; i < kFly; ++i)
#pragma unroll
        for (int e = 0; e < Per; ++e) {
          const int ci = c + i * GR;
          const size_t at = size_t(ci) * a.R16 + min(rt + e * RS, top);
          p[i][e] = make_float2(-FLT_MAX, 0.f), x[i][e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (ci <= c1) {
            p[i][e] = a.ml[at];
            x[i][e] = reinterpret_cast<const float4*>(a.opart)[at * (D / 4) + c4];
          }
        }
#pragma unroll
      for (int e = 0; e < Per; ++e) {
        float M1 = M[e];
#pragma unroll
        for (int i = 0; i < kFly; ++i) M1 = fmaxf(M1, p[i][e].x);
        const float w = fast_exp2(M[e] - M1);
        L[e] *= w, acc[e].x *= w, acc[e].y *= w, acc[e].z *= w, acc[e].w *= w;
        M[e] = M1;
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
          const float f = fast_exp2(p[i][e].x - M1);
          L[e] += f * p[i][e].y;
          acc[e].x += f * x[i][e].x, acc[e].y += f * x[i][e].y;
          acc[e].z += f * x[i][e].z, acc[e].w += f * x[i][e].w;
        }
      }
    }
  }
  if constexpr (GR > 1) {
    static_assert(Per == 1, "groups of one row a thread");
    part[grp][rr][c4] = acc[0];
    if (c4 == 0) part_m[grp][rr] = M[0], part_l[grp][rr] = L[0];
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int i = 0; i < GR; ++i) M[0] = fmaxf(M[0], part_m[i][rr]);
    L[0] = 0.f;
    acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      const float f = fast_exp2(part_m[i][rr] - M[0]);
      const float4 x = part[i][rr][c4];
      L[0] += f * part_l[i][rr];
      acc[0].x += f * x.x, acc[0].y += f * x.y, acc[0].z += f * x.z, acc[0].w += f * x.w;
    }
  }
#pragma unroll
  for (int e = 0; e < Per; ++e) {
    const int r = r0 + rr + e * RS;
    if (r >= R) break;
    const float inv = L[e] == 0.f ? 0.f : 1.f / L[e];
    *reinterpret_cast<uint2*>(a.out + ((size_t(n) * a.B + r / G) * a.Hq + g * G + r % G) * D + c4 * 4) =
        make_uint2(pack_bf16(acc[e].x * inv, acc[e].y * inv), pack_bf16(acc[e].z * inv, acc[e].w * inv));
  }
}

// ------------------------------------------------------------------- host

template <int D>
static cudaError_t launch_join(const Kv8AttnArgs& a, int R, int num_sms, cudaStream_t st) {
  auto go = [&](auto* kernel, int rows, int threads) {
    return launch_k("kv8_join_kernel", kernel, dim3(unsigned(a.N * a.Hkv), unsigned(cdiv(R, rows))),
                    dim3(unsigned(threads)), 0, st, a);
  };
  // Few rows a CTA and its groups of threads side by side on the pieces, as long as every CTA
  // is resident at once; many CTAs in a row would each pay for the pieces' place and the block's
  // keys.  The whole call in us, without products (4 rows in 4 groups / 8 in one): one segment of
  // 2K keys 7.0 / 7.8, eight of 128K 47.2 / 48.3, 512 of up to 8K 97.2 / 93.7, 128 with 16 rows
  // 29.0 / 26.4.  With products (4 rows in 4 groups / 8 in two / 16 in one): 8 segments of 20 rows
  // 15.3 / 15.5 / 18.0, 32 of 32 rows 19.8 / 17.1 / 17.0, 4 of 224 rows 28.4 / 25.8 / 28.5, 32 of
  // 128 rows 131 / 121 / 112.
  const int64_t segs = int64_t(a.N) * a.Hkv;
  if (!a.bk || a.B <= kOwnFew) {
    if (segs * cdiv(R, 4) <= num_sms) return go(kv8_join_kernel<D, 4, 1, 4, false>, 4, D * 4);
    return go(kv8_join_kernel<D, 8, 1, 1, false>, 8, D * 2);
  }
  if (segs * cdiv(R, 4) <= num_sms) return go(kv8_join_kernel<D, 4, 1, 4, true>, 4, D * 4);
  if (segs * cdiv(R, 8) <= num_sms) return go(kv8_join_kernel<D, 8, 1, 2, true>, 8, D * 4);
  return go(kv8_join_kernel<D, 16, 2, 1, true>, 16, D * 2);
}

// Workspace: error word, then (m, l) and O of every partial.
struct Kv8Ws {
  size_t ml, opart, total;
  int R16, row_tiles;
};
static Kv8Ws kv8_ws(const herald_dims& dm) {
  Kv8Ws w;
  const int R = dm.B * (dm.Hq / dm.Hkv);
  w.row_tiles = cdiv(R, kTileM);
  w.R16 = std::min(cdiv(R, 16) * 16, kTileM);
  const size_t slots = size_t(kKv8MaxCtas) + size_t(dm.N) * dm.Hkv * w.row_tiles;
  w.ml = 256;
  w.opart = align_up(w.ml + slots * w.R16 * 8, 256);
  // (O is written by 32 bytes; the workspace itself may be aligned to 16)
  w.total = w.opart + slots * w.R16 * size_t(dm.d) * 4 + 16;
  return w;
}
size_t kv8_attn_workspace(const herald_dims& dm) { return kv8_ws(dm).total; }

cudaError_t launch_kv8_attn(const herald_dims& dm, const uint16_t* q, const Kv8Dev& c,
                            const CUtensorMap& kmap, const CUtensorMap& vmap, const int32_t* ctx,
                            const uint16_t* bk, const uint16_t* bv, uint16_t* out, float scale, void* ws, int num_sms, cudaStream_t st) {
  const int G = dm.Hq / dm.Hkv, R = dm.B * G;
  const Kv8Ws w = kv8_ws(dm);
  char* p = static_cast<char*>(ws);
  Kv8AttnArgs a{};
  a.q = q, a.bk = bk, a.bv = bv, a.ctx = ctx, a.out = out;
  a.ml = reinterpret_cast<float2*>(p + w.ml);
  a.opart = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(p + w.opart) + 31) & ~uintptr_t(31));
  a.scale = scale * 1.4426950408889634f;
  a.N = dm.N, a.Hq = dm.Hq, a.Hkv = dm.Hkv, a.B = dm.B, a.L_max = dm.L_max;
  a.R16 = w.R16, a.row_tiles = w.row_tiles;
  a.c = c;
  a.ctas = std::min(kKv8MaxCtas, num_sms);
  a.pad = R <= kKv8FewRows ? kKv8PadRows : kKv8PadTc;
  uint32_t* err = reinterpret_cast<uint32_t*>(p);
  if (R <= kKv8FewRows)
    HERALD_CHECK_LAUNCH(launch_kv8_rows(dm.d, R, a, kmap, vmap, err, st));
  else
    HERALD_CHECK_LAUNCH(launch_kv8_attn_tc(dm.d, a, kmap, vmap, err, st));
  HERALD_CHECK_LAUNCH(dm.d == 128 ? launch_join<128>(a, R, num_sms, st)
                                  : launch_join<64>(a, R, num_sms, st));
  return cudaGetLastError();
}

}  // namespace herald
