// kv8_attn.cu -- attention of a block's queries over the whole paged 8-bit cache and
// the block's own bf16 keys: a kernel for few or many query rows (kv8_rows.cu,
// kv8_attn_tc.cu) writes partial results over the cache's keys (m, l, O per query row
// and piece of a segment), the join here adds the block's own keys and writes the output.
#include <float.h>
#include <math.h>

#include "kv8.cuh"

namespace herald {

constexpr int kKv8MaxCtas = 304;  // most attention CTAs (workspace slots)

// The output: the pieces of a segment joined, with the block's own keys.  grid (N*Hkv,
// ceil(R / Rows)); D/4 lanes hold a row's channels, four each, and Threads over Rows
// such groups share a row: each takes every such-and-suchth chunk of the block's own
// keys (a key per lane: q in shared memory, the whole of a dot product in one lane,
// fp32 throughout) and every such-and-suchth piece, five in flight; the groups are
// then added in order.  The block's keys come before the grid-dependency wait: they
// and the lengths were written before the attention kernel's own wait ended, and it
// lets this kernel start only after that.
template <int D, int Rows, int Threads>
__global__ void __launch_bounds__(Threads) kv8_join_kernel(const Kv8AttnArgs a) {
  constexpr int TPR = D / 4, GR = Threads / (TPR * Rows);
  __shared__ float qs[Rows][D];
  __shared__ float4 part[GR][Rows][TPR];
  __shared__ float part_m[GR][Rows], part_l[GR][Rows];
  const int seg = blockIdx.x, n = seg / a.Hkv, g = seg - n * a.Hkv;
  const int G = a.Hq / a.Hkv, R = a.B * G;
  const int c4 = threadIdx.x % TPR, rr = threadIdx.x / TPR % Rows, grp = threadIdx.x / (TPR * Rows);
  const int r = int(blockIdx.y) * Rows + rr, rc = min(r, R - 1);
  const size_t row = (size_t(n) * a.B + rc / G) * a.Hq + g * G + rc % G;
  const int heads = a.Hkv * a.row_tiles, tile = rc / a.R16, rt = rc - tile * a.R16;
  const Kv4Split split = kv4_split(kv4_total_units(a.ctx, a.N, a.L_max, 0, a.pad), heads, a.ctas);
  const int units = kv4_units(a.ctx[n], a.L_max, 0, a.pad), gt = g * a.row_tiles + tile;
  const int first = heads * kv4_total_units(a.ctx, n, a.L_max, 0, a.pad) + gt * units;
  float M = -FLT_MAX, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.bk) {
    if (grp == 0) {
      const uint2 w = *reinterpret_cast<const uint2*>(a.q + row * D + c4 * 4);
      float4 f = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
      *reinterpret_cast<float4*>(&qs[rr][c4 * 4]) = f;
    }
    __syncthreads();
    const int chunks = (a.B + TPR - 1) / TPR;
    for (int ch = grp; ch < chunks; ch += GR) {  // (grp, and so the count, is a warp's own
      const int j = ch * TPR + c4;               // or, with D = 64, a multiple of it: Rows >= 2)
      float s = -INFINITY;
      if (j < a.B) {
        const uint4* kp =
            reinterpret_cast<const uint4*>(a.bk + ((size_t(n) * a.B + j) * a.Hkv + g) * D);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 w = kp[i];
          const float4 x = *reinterpret_cast<const float4*>(&qs[rr][i * 8]);
          const float4 y = *reinterpret_cast<const float4*>(&qs[rr][i * 8 + 4]);
          s0 = fmaf(x.x, bf16lo(w.x), s0), s1 = fmaf(x.y, bf16hi(w.x), s1);
          s0 = fmaf(x.z, bf16lo(w.y), s0), s1 = fmaf(x.w, bf16hi(w.y), s1);
          s0 = fmaf(y.x, bf16lo(w.z), s0), s1 = fmaf(y.y, bf16hi(w.z), s1);
          s0 = fmaf(y.z, bf16lo(w.w), s0), s1 = fmaf(y.w, bf16hi(w.w), s1);
        }
        s = (s0 + s1) * a.scale;
      }
      float m1 = fmaxf(M, s);
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
      const float k = fast_exp2(M - m1), p = fast_exp2(s - m1);
      float sum = p;
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      M = m1, L = L * k + sum;
      acc.x *= k, acc.y *= k, acc.z *= k, acc.w *= k;
      const int here = min(TPR, a.B - ch * TPR);
      const uint16_t* vp = a.bv + ((size_t(n) * a.B + ch * TPR) * a.Hkv + g) * D + c4 * 4;
#pragma unroll 4
      for (int i = 0; i < here; ++i) {
        const float pi = __shfl_sync(0xffffffffu, p, i, TPR);
        const uint2 w = *reinterpret_cast<const uint2*>(vp + size_t(i) * a.Hkv * D);
        acc.x = fmaf(pi, bf16lo(w.x), acc.x), acc.y = fmaf(pi, bf16hi(w.x), acc.y);
        acc.z = fmaf(pi, bf16lo(w.y), acc.z), acc.w = fmaf(pi, bf16hi(w.y), acc.w);
      }
    }
  }
  griddep_enter();
  if (units > 0) {
    const int c0 = (first + a.pad) / split.share + n * heads + gt,
              c1 = (first + units - 1) / split.share + n * heads + gt;  // slots of its pieces
    const float4* op = reinterpret_cast<const float4*>(a.opart) + size_t(rt) * (D / 4) + c4;
    constexpr int kFly = 5;
    for (int c = c0 + grp; c <= c1; c += kFly * GR) {
      float2 p[kFly];
      float4 x[kFly];
#pragma unroll
      for (int i = 0; i < kFly; ++i) {
        const int ci = c + i * GR;
        p[i] = make_float2(-FLT_MAX, 0.f), x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ci <= c1) {
          p[i] = a.ml[size_t(ci) * a.R16 + rt];
          x[i] = op[size_t(ci) * a.R16 * (D / 4)];
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
  }
  if constexpr (GR > 1) {
    part[grp][rr][c4] = acc;
    if (c4 == 0) part_m[grp][rr] = M, part_l[grp][rr] = L;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int i = 0; i < GR; ++i) M = fmaxf(M, part_m[i][rr]);
    L = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      const float f = fast_exp2(part_m[i][rr] - M);
      const float4 x = part[i][rr][c4];
      L += f * part_l[i][rr];
      acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
    }
  }
  if (r >= R) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(a.out + row * D + c4 * 4) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

// ------------------------------------------------------------------- host

template <int D>
static cudaError_t launch_join(const Kv8AttnArgs& a, int R, int num_sms, cudaStream_t st) {
  auto go = [&](auto* kernel, int rows, int threads) {
    return launch_k("kv8_join_kernel", kernel, dim3(unsigned(a.N * a.Hkv), unsigned(cdiv(R, rows))),
                    dim3(unsigned(threads)), 0, st, a);
  };
  const int64_t segs = int64_t(a.N) * a.Hkv;
  if (segs * cdiv(R, 4) <= num_sms) return go(kv8_join_kernel<D, 4, 1024>, 4, 1024);
  return go(kv8_join_kernel<D, 8, D * 2>, 8, D * 2);
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
  w.total = w.opart + slots * w.R16 * size_t(dm.d) * 4;
  return w;
}
size_t kv8_attn_workspace(const herald_dims& dm) { return kv8_ws(dm).total; }

cudaError_t launch_kv8_attn(const herald_dims& dm, const uint16_t* q, const Kv8Dev& c,
                            const CUtensorMap& kmap, const CUtensorMap& vmap, const int32_t* ctx, const uint16_t* bk, const uint16_t* bv,
                            uint16_t* out, float scale, void* ws, int num_sms, cudaStream_t st) {
  const int G = dm.Hq / dm.Hkv, R = dm.B * G;
  const Kv8Ws w = kv8_ws(dm);
  char* p = static_cast<char*>(ws);
  Kv8AttnArgs a{};
  a.q = q, a.bk = bk, a.bv = bv, a.ctx = ctx, a.out = out;
  a.ml = reinterpret_cast<float2*>(p + w.ml);
  a.opart = reinterpret_cast<float*>(p + w.opart);
  a.scale = scale * 1.4426950408889634f;
  a.N = dm.N, a.Hq = dm.Hq, a.Hkv = dm.Hkv, a.B = dm.B, a.L_max = dm.L_max, a.R16 = w.R16, a.row_tiles = w.row_tiles;
  a.c = c;
  a.ctas = std::min(kKv8MaxCtas, num_sms);
  a.pad = 0;
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
