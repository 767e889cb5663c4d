// The gated feed-forward block on one weight set (a shared expert beside the
// routed ones), bf16:
//   h = bf16(silu(x Wg^T) * (x Wu^T)),  y = bf16(res + h W2^T)
// with W1p [2f, d] = [Wg; Wu] and W2 [d, f], both K-contiguous, and its
// backward.  g and u are not rounded before the activation; h is, because the
// second product takes bf16 operands.  Accumulation fp32; the residual joins
// the fp32 sum, so y is rounded once.
//
// Three forms, by the number of tokens T (choose_form says where they meet):
//  * few tokens: the weights are read once and that is the bound (HBM).  A
//    workgroup owns 16 weight rows, its wavefronts split K and go straight
//    from HBM to MFMA fragments, no LDS stage; the wavefronts' sums meet in
//    LDS in a fixed order;
//  * a moderate number: BM x BN tiles through LDS, K split over workgroups
//    until the chip is full, the fp32 partial sums added by a second kernel
//    in split order;
//  * many: the persistent 256 x 256 kernels of the grouped products
//    (gg_bf16.hip) with one group.
#include <algorithm>

#include "dense_args.h"
#include "gg_common.h"

namespace moe {
moe_status_t launch_fwd(const GGArgs& a, int epilogue, int out_f32, int b_layout, hipStream_t s);  // gg_bf16.hip
moe_status_t launch_fwd_residual(const GGArgs& a, hipStream_t s);                                   // gg_bf16.hip
moe_status_t launch_wgrad(const GGArgs& a, int out_f32, hipStream_t s);                             // gg_bf16.hip
size_t fwd_split_workspace_bytes();                                                                  // gg_bf16.hip

namespace ffn {

struct ProdArgs {
  const uint16_t* x;     // [T, K] rows, pitch ldx
  const uint16_t* w;     // [N, K] (plain) or [2N, K] (gated: N gate rows, N up rows)
  const uint16_t* res;   // plain: [T, N], pitch ldr, or NULL
  uint16_t* out;         // [T, N]
  uint16_t* aux;         // gated: [T, 2N] pre-activations, or NULL
  float* part;           // split: [S, T, N or 2N] partial sums
  int64_t ldx, ldr;
  int T, N, K;
  int S;                 // splits of K
  int mtiles, ntiles;
};

__device__ __forceinline__ f32x4_t mfma(uint4 w, uint4 x, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, x), c,
                                                 0, 0, 0);
}

// ------------------------------------------------------------------ few tokens
// 16 weight rows per workgroup (gated: 8 gate rows and the 8 matching up
// rows), MT x 16 tokens.  Wavefront w takes the 32-deep K steps w, w + NW, ...,
// U of them in flight while the U before are multiplied.
constexpr int kFewWaves = 8, kFewUnroll = 8;

template <int MT, bool GATED>
__global__ __launch_bounds__(kFewWaves * 64) void few_tokens_kernel(ProdArgs a) {
  constexpr int NW = kFewWaves, U = kFewUnroll;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r16 = lane & 15, g4 = lane >> 4;
  const int n0 = blockIdx.x * (GATED ? 8 : 16);
  int row;   // this lane's weight row; rows past the end repeat the last one and are not stored
  if constexpr (GATED) {
    row = min(n0 + (r16 & 7), a.N - 1) + (r16 < 8 ? 0 : a.N);
  } else {
    row = min(n0 + r16, a.N - 1);
  }
  const uint16_t* wp = a.w + (int64_t)row * a.K + 8 * g4;
  const uint16_t* xp[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) xp[m] = a.x + (int64_t)min(16 * m + r16, a.T - 1) * a.ldx + 8 * g4;
  const int steps = (a.K + 31) / 32;
  f32x4_t acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  struct Batch {
    uint4 w[U], x[U][MT];
  };
  auto load = [&](int s0, Batch& b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = 32 * (s0 + u * NW);
      const bool ok = k + 8 * g4 < a.K;   // K % 8 == 0: a lane's piece is whole or absent
      b.w[u] = ok ? *reinterpret_cast<const uint4*>(wp + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        b.x[u][m] = ok ? *reinterpret_cast<const uint4*>(xp[m] + k) : make_uint4(0, 0, 0, 0);
    }
  };
  auto mma = [&](const Batch& b) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m] = mfma(b.w[u], b.x[u][m], acc[m]);
  };
  Batch p, q;
  int s = wave;
  if (s < steps) load(s, p);
  while (s < steps) {
    s += U * NW;
    if (s < steps) load(s, q);
    mma(p);
    if (s >= steps) break;
    s += U * NW;
    if (s < steps) load(s, p);
    mma(q);
  }
  // sum of the wavefronts in their order; lane: token r16, rows 4 g4 + e
  __shared__ float sum[NW][MT * 16][17];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[wave][16 * m + r16][4 * g4 + e] = acc[m][e];
  __syncthreads();
  constexpr int PER = GATED ? 8 : 16;   // output columns of the workgroup
  for (int i = threadIdx.x; i < MT * 16 * PER; i += NW * 64) {
    const int t = i / PER, j = i % PER;
    if (t >= a.T || n0 + j >= a.N) continue;
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      v += sum[w][t][j];
      if constexpr (GATED) u += sum[w][t][8 + j];
    }
    if constexpr (GATED) {
      if (a.aux) {
        a.aux[(int64_t)t * 2 * a.N + n0 + j] = (uint16_t)f32_to_bf16_bits(v);
        a.aux[(int64_t)t * 2 * a.N + a.N + n0 + j] = (uint16_t)f32_to_bf16_bits(u);
      }
      v = silu_f32(v) * u;
    } else if (a.res) {
      v += bf16_bits_to_f32(a.res[t * a.ldr + n0 + j]);
    }
    a.out[(int64_t)t * a.N + n0 + j] = (uint16_t)f32_to_bf16_bits(v);
  }
}

// ------------------------------------------------------------------ tiles
// BM tokens x BN weight rows, K staged 64 at a time through two LDS buffers:
// the next stage's loads are in flight (in registers) while the present one
// is multiplied.  Four wavefronts, 2 x 2.  LDS rows of 128 bytes, 16-byte
// slots XOR-swizzled by row.  Gated: a wavefront's weight rows are BN/4 gate
// rows followed by the matching BN/4 up rows.
template <int BM, int BN, bool GATED>
__global__ __launch_bounds__(256) void tile_kernel(ProdArgs a) {
  constexpr int TM = BM / 32, TN = BN / 32;
  constexpr int XR = BM / 32, WR = BN / 32;   // 16-byte pieces per thread and stage
  __shared__ __align__(16) uint8_t lds[2][(BM + BN) * 128];
  // consecutive workgroups run on different XCDs; the m-tiles of one weight
  // tile follow each other on one XCD, so its L2 reads the weights once
  const int xcd = blockIdx.x & 7, q = blockIdx.x >> 3;
  const int mt = q % a.mtiles, unit = (q / a.mtiles) * 8 + xcd;
  if (unit >= a.ntiles * a.S) return;
  const int nt = unit % a.ntiles, split = unit / a.ntiles;
  const int m0 = mt * BM, n0 = nt * (GATED ? BN / 2 : BN);
  const int steps = (a.K + 63) / 64;
  const int s0 = (int)((int64_t)split * steps / a.S), s1 = (int)((int64_t)(split + 1) * steps / a.S);
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r16 = lane & 15, g4 = lane >> 4;
  const int wm = wave & 1, wn = wave >> 1;
  // loader: this thread's piece of row lr + 32 i
  const int lr = threadIdx.x >> 3, lc = threadIdx.x & 7;
  const uint16_t* xp[XR];
  const uint16_t* wp[WR];
#pragma unroll
  for (int i = 0; i < XR; ++i) xp[i] = a.x + (int64_t)min(m0 + lr + 32 * i, a.T - 1) * a.ldx + 8 * lc;
#pragma unroll
  for (int i = 0; i < WR; ++i) {
    const int r = lr + 32 * i;
    int row;
    if constexpr (GATED) {
      const int w = r / (BN / 2), p = r % (BN / 2);
      row = min(n0 + w * (BN / 4) + p % (BN / 4), a.N - 1) + (p < BN / 4 ? 0 : a.N);
    } else {
      row = min(n0 + r, a.N - 1);
    }
    wp[i] = a.w + (int64_t)row * a.K + 8 * lc;
  }
  uint4 xv[XR], wv[WR];
  auto load = [&](int s) {
    const int k = 64 * s;
    const bool ok = k + 8 * lc < a.K;
#pragma unroll
    for (int i = 0; i < WR; ++i) wv[i] = ok ? *reinterpret_cast<const uint4*>(wp[i] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < XR; ++i) xv[i] = ok ? *reinterpret_cast<const uint4*>(xp[i] + k) : make_uint4(0, 0, 0, 0);
  };
  auto put = [&](uint8_t* buf) {
    const int o = lr * 128 + ((lc ^ (lr & 7)) << 4);
#pragma unroll
    for (int i = 0; i < WR; ++i) *reinterpret_cast<uint4*>(buf + o + i * 32 * 128) = wv[i];
#pragma unroll
    for (int i = 0; i < XR; ++i) *reinterpret_cast<uint4*>(buf + BN * 128 + o + i * 32 * 128) = xv[i];
  };
  f32x4_t acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (s0 < s1) {
    load(s0);
    put(lds[0]);
    __syncthreads();
    for (int s = s0; s < s1; ++s) {
      const uint8_t* buf = lds[(s - s0) & 1];
      if (s + 1 < s1) load(s + 1);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int slot = ((kk * 4 + g4) ^ (r16 & 7)) << 4;
        uint4 fw[TN], fx[TM];
#pragma unroll
        for (int i = 0; i < TN; ++i)
          fw[i] = *reinterpret_cast<const uint4*>(buf + (wn * (BN / 2) + i * 16 + r16) * 128 + slot);
#pragma unroll
        for (int j = 0; j < TM; ++j)
          fx[j] = *reinterpret_cast<const uint4*>(buf + BN * 128 + (wm * (BM / 2) + j * 16 + r16) * 128 + slot);
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int j = 0; j < TM; ++j) acc[i][j] = mfma(fw[i], fx[j], acc[i][j]);
      }
      if (s + 1 < s1) put(lds[(s + 1 - s0) & 1]);
      __syncthreads();
    }
  }
  // lane: token r16 of each 16, four consecutive columns from 4 g4
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int t = m0 + wm * (BM / 2) + j * 16 + r16;
    if (t >= a.T) continue;
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < TN / 2; ++i) {
        const int c = n0 + wn * (BN / 4) + i * 16 + 4 * g4;
        if (c >= a.N) continue;
        const f32x4_t g = acc[i][j], u = acc[i + TN / 2][j];
        if (a.part) {
          float* const o = a.part + ((int64_t)split * a.T + t) * 2 * a.N;
          *reinterpret_cast<f32x4_t*>(o + c) = g;
          *reinterpret_cast<f32x4_t*>(o + a.N + c) = u;
        } else {
          uint8_t* const aux = reinterpret_cast<uint8_t*>(a.aux);
          if (aux) {
            store_sub<MOE_OUT_BF16>(aux, 2 * (int64_t)a.N, t, c, g);
            store_sub<MOE_OUT_BF16>(aux, 2 * (int64_t)a.N, t, a.N + c, u);
          }
          f32x4_t h;
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = silu_f32(g[e]) * u[e];
          store_sub<MOE_OUT_BF16>(reinterpret_cast<uint8_t*>(a.out), a.N, t, c, h);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int c = n0 + wn * (BN / 2) + i * 16 + 4 * g4;
        if (c >= a.N) continue;
        f32x4_t v = acc[i][j];
        if (a.part) {
          *reinterpret_cast<f32x4_t*>(a.part + ((int64_t)split * a.T + t) * a.N + c) = v;
        } else {
          if (a.res) {
            const uint16_t* r = a.res + t * a.ldr + c;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += bf16_bits_to_f32(r[e]);
          }
          store_sub<MOE_OUT_BF16>(reinterpret_cast<uint8_t*>(a.out), a.N, t, c, v);
        }
      }
    }
  }
}

// The partial sums of the S splits, added in split order, through the
// product's epilogue; four columns a thread.
template <bool GATED>
__global__ __launch_bounds__(256) void join_kernel(ProdArgs a) {
  const int nq = a.N / 4;
  const int64_t total = (int64_t)a.T * nq;
  const int ld = GATED ? 2 * a.N : a.N;
  const int64_t plane = (int64_t)a.T * ld;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / nq;
    const int c = 4 * (int)(i - t * nq);
    const float* p = a.part + t * ld + c;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(p), u = v;
    if constexpr (GATED) u = *reinterpret_cast<const f32x4_t*>(p + a.N);
#pragma unroll 4
    for (int s = 1; s < a.S; ++s) {
      v += *reinterpret_cast<const f32x4_t*>(p + s * plane);
      if constexpr (GATED) u += *reinterpret_cast<const f32x4_t*>(p + s * plane + a.N);
    }
    if constexpr (GATED) {
      if (a.aux) {
        uint8_t* const aux = reinterpret_cast<uint8_t*>(a.aux);
        store_sub<MOE_OUT_BF16>(aux, ld, t, c, v);
        store_sub<MOE_OUT_BF16>(aux, ld, t, a.N + c, u);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = silu_f32(v[e]) * u[e];
    } else if (a.res) {
      const uint16_t* r = a.res + t * a.ldr + c;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += bf16_bits_to_f32(r[e]);
    }
    store_sub<MOE_OUT_BF16>(reinterpret_cast<uint8_t*>(a.out), a.N, t, c, v);
  }
}

__global__ void set_rows_kernel(int32_t* p, int32_t v) { *p = v; }

// ------------------------------------------------------------------ host

enum Form { FEW, TILES, MANY };
struct Plan {
  Form form;
  int BM, S;
};

// How one product [T, K] x [N or 2N, K] runs.
Plan choose_form(int64_t T, int N, int K, bool gated, bool strided) {
  const int cus = moe_host::device_cu_count();
  if (T <= 16) return {FEW, 0, 1};
  const int64_t big = ((T + 255) / 256) * ((N + (gated ? 127 : 255)) / (gated ? 128 : 256));
  if (!strided && K % 64 == 0 && 4 * big >= 3 * (int64_t)cus) return {MANY, 0, 1};
  const int BM = T <= 64 ? 64 : 128;
  const int64_t tiles = ((T + BM - 1) / BM) * ((N + (gated ? 63 : 127)) / (gated ? 64 : 128));
  const int steps = (K + 63) / 64;
  const int S = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(16, steps / 4), 2 * cus / tiles));
  return {TILES, BM, S};
}

size_t part_bytes(const Plan& p, int64_t T, int N, bool gated) {
  if (p.form == MANY) return fwd_split_workspace_bytes();
  if (p.form == TILES && p.S > 1) return (size_t)p.S * (size_t)T * (size_t)(gated ? 2 * N : N) * 4;
  return 0;
}

moe_status_t status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

template <bool GATED>
moe_status_t run_tiles(ProdArgs a, const Plan& p, hipStream_t s) {
  constexpr int BN = 128;
  a.S = p.S;
  if (p.S == 1) a.part = nullptr;
  a.mtiles = (a.T + p.BM - 1) / p.BM;
  a.ntiles = (a.N + (GATED ? BN / 2 : BN) - 1) / (GATED ? BN / 2 : BN);
  const int64_t units = (int64_t)a.ntiles * a.S;
  const dim3 grid((unsigned)(8 * a.mtiles * ((units + 7) / 8)));
  if (p.BM == 64) {
    hipLaunchKernelGGL((tile_kernel<64, BN, GATED>), grid, dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL((tile_kernel<128, BN, GATED>), grid, dim3(256), 0, s, a);
  }
  if (status() != MOE_OK) return MOE_ERR_HIP;
  if (p.S > 1) {
    const int64_t total = (int64_t)a.T * (a.N / 4);
    const int64_t blocks = std::min<int64_t>((total + 255) / 256, 16 * (int64_t)moe_host::device_cu_count());
    hipLaunchKernelGGL((join_kernel<GATED>), dim3((unsigned)blocks), dim3(256), 0, s, a);
  }
  return status();
}

GGArgs one_group(const void* A, const void* B, void* C, void* aux, int64_t T, int N, int K, const int32_t* rows,
                 float* part) {
  GGArgs g{};
  g.A = reinterpret_cast<const uint8_t*>(A);
  g.B = reinterpret_cast<const uint8_t*>(B);
  g.C = reinterpret_cast<uint8_t*>(C);
  g.Caux = reinterpret_cast<uint8_t*>(aux);
  g.sizes = rows;
  g.m_cap = T;
  g.G = 1;
  g.N = N;
  g.K = K;
  g.part = part;
  return g;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace ffn
}  // namespace moe

using namespace moe;
using namespace moe::ffn;

// Workspace: the row count (device), h where the caller keeps none, and the
// larger of the two products' partial sums.
extern "C" size_t moe_gated_ffn_ws_impl(int64_t T, int32_t d, int32_t f, int keep, int strided) {
  const size_t a = part_bytes(choose_form(T, f, d, true, strided), T, f, true);
  const size_t b = part_bytes(choose_form(T, d, f, false, false), T, d, false);
  return 256 + (keep ? 0 : up256((size_t)T * f * 2)) + std::max(a, b);
}

extern "C" moe_status_t moe_gated_ffn_launch(const uint16_t* x, int64_t ldx, const uint16_t* w1p, const uint16_t* w2,
                                             const uint16_t* res, int64_t ldr, int64_t T, int32_t d, int32_t f,
                                             uint16_t* h, uint16_t* gu, uint16_t* y, void* ws, hipStream_t s) {
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  int32_t* const rows = reinterpret_cast<int32_t*>(w);
  w += 256;
  if (!h) {
    h = reinterpret_cast<uint16_t*>(w);
    w += up256((size_t)T * f * 2);
  }
  float* const part = reinterpret_cast<float*>(w);
  const bool strided = ldx != d;
  const Plan p1 = choose_form(T, f, d, true, strided), p2 = choose_form(T, d, f, false, false);
  if (p1.form == MANY || p2.form == MANY) {
    hipLaunchKernelGGL(set_rows_kernel, dim3(1), dim3(1), 0, s, rows, (int32_t)T);
    if (ffn::status() != MOE_OK) return MOE_ERR_HIP;
  }
  ProdArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.w = w1p;
  a.out = h;
  a.aux = gu;
  a.part = part;
  a.T = (int)T;
  a.N = f;
  a.K = d;
  moe_status_t st;
  if (p1.form == FEW) {
    hipLaunchKernelGGL((few_tokens_kernel<1, true>), dim3((unsigned)((f + 7) / 8)), dim3(kFewWaves * 64), 0, s, a);
    st = ffn::status();
  } else if (p1.form == TILES) {
    st = run_tiles<true>(a, p1, s);
  } else {
    st = launch_fwd(one_group(x, w1p, h, gu, T, 2 * f, d, rows, part), MOE_EPI_SWIGLU, 0, MOE_B_NK, s);
  }
  if (st != MOE_OK) return st;
  ProdArgs b{};
  b.x = h;
  b.ldx = f;
  b.w = w2;
  b.res = res;
  b.ldr = ldr;
  b.out = y;
  b.part = part;
  b.T = (int)T;
  b.N = d;
  b.K = f;
  if (p2.form == FEW) {
    hipLaunchKernelGGL((few_tokens_kernel<1, false>), dim3((unsigned)((d + 15) / 16)), dim3(kFewWaves * 64), 0, s, b);
    return ffn::status();
  }
  if (p2.form == TILES) return run_tiles<false>(b, p2, s);
  GGArgs g = one_group(h, w2, y, const_cast<uint16_t*>(res), T, d, f, rows, part);
  if (res) {
    g.ld_aux = ldr;
    return launch_fwd_residual(g, s);
  }
  return launch_fwd(g, MOE_EPI_NONE, 0, MOE_B_NK, s);
}

extern "C" size_t moe_gated_ffn_backward_ws_impl(void) { return 256 + fwd_split_workspace_bytes(); }

extern "C" moe_status_t moe_gated_ffn_backward_launch(const uint16_t* dy, const uint16_t* x, const uint16_t* gu,
                                                      const uint16_t* h, const uint16_t* w1p, const uint16_t* w2,
                                                      int64_t T, int32_t d, int32_t f, uint16_t* dgu, uint16_t* dx,
                                                      void* dw1p, void* dw2, int out_f32, void* ws, hipStream_t s) {
  int32_t* const rows = reinterpret_cast<int32_t*>(ws);
  float* const part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + 256);
  hipLaunchKernelGGL(set_rows_kernel, dim3(1), dim3(1), 0, s, rows, (int32_t)T);
  moe_status_t st = ffn::status();
  // dgu = swiglu'(gu, dy W2), dx = dgu W1p
  if (st == MOE_OK && T > 0)
    st = launch_fwd(one_group(dy, w2, dgu, const_cast<uint16_t*>(gu), T, f, d, rows, part), MOE_EPI_SWIGLU_BWD, 0,
                    MOE_B_KN, s);
  if (st == MOE_OK && T > 0)
    st = launch_fwd(one_group(dgu, w1p, dx, nullptr, T, d, 2 * f, rows, part), MOE_EPI_NONE, 0, MOE_B_KN, s);
  // dW1p = dgu^T x, dW2 = dy^T h
  if (st == MOE_OK) {
    GGArgs g = one_group(dgu, x, dw1p, nullptr, T, d, 0, rows, nullptr);
    g.M = 2 * f;
    st = launch_wgrad(g, out_f32, s);
  }
  if (st == MOE_OK) {
    GGArgs g = one_group(dy, h, dw2, nullptr, T, f, 0, rows, nullptr);
    g.M = d;
    st = launch_wgrad(g, out_f32, s);
  }
  return st;
}
