// Root-mean-square norm in front of the layer, with the residual's addition
// before it and MXFP8 quantisation behind it, and its backward.
//
// Forward, per row of d elements:
//   s = x + r          rounded to the residual stream's type, as it is stored
//   rstd = 1 / sqrt(mean(s^2) + eps)
//   y = bf16(s * rstd * w);  MXFP8: the codes and scales of that y
// The norm is that of the stored s, so the backward, which reads s,
// differentiates what the forward computed.  Backward, with xh = s * rstd:
//   ds = dres + rstd * (w * dy - xh * mean(w * dy * xh)),  dw = sum_rows dy * xh
//
// Bound: HBM.  A row is read once into registers by TPR threads (one
// wavefront, 256 or 1024 threads), its sum of squares taken there and its
// outputs written from there; the weight comes from L2.  All arithmetic and
// every sum is fp32.
#include "common.h"
#include "dense_args.h"

namespace moe {

__device__ __forceinline__ void load8_f32(const float* p, float* f) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8_f32(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// weight elements 8v .. 8v + 7
__device__ __forceinline__ void load_w8(const void* w, int w_f32, int v, float* f) {
  if (w_f32) {
    load8_f32(reinterpret_cast<const float*>(w) + 8 * v, f);
  } else {
    unpack8(reinterpret_cast<const uint4*>(w)[v], f);
  }
}
__device__ __forceinline__ float load_w1(const void* w, int w_f32, int e) {
  return w_f32 ? reinterpret_cast<const float*>(w)[e] : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(w)[e]);
}

// Sum of v over the TPR threads of a row (one wavefront, or the workgroup
// through one LDS word per wavefront: `slot` picks one of two such sets, so
// that two sums in a row need one barrier each).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, int slot) {
  v = wave_sum(v);
  if constexpr (TPR > kWave) {
    constexpr int NW = TPR / kWave;
    __shared__ float part[2][NW];
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) v += part[slot][i];
  }
  return v;
}

// One row's element block: 8 elements of s, as stored (bf16 pairs or floats)
template <int RT>
struct Row8 {
  uint4 b;
  __device__ __forceinline__ void get(float* f) const { unpack8(b, f); }
};
template <>
struct Row8<RES_F32> {
  float v[8];
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v[j];
  }
};

// 16-byte path: d % 8 == 0, rows and pointers 16-byte aligned.  Thread t of a
// row holds the 8-element pieces t, t + TPR, ...; the four lanes of an MXFP8
// block are neighbours.
template <int TPR, int VPT, int RT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void add_rmsnorm_kernel(NormArgs a) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
  if (row >= a.T) return;   // RPW > 1: a whole wavefront, and row_sum has no barrier
  const int nvec = a.d / 8;
  const uint4* xr = reinterpret_cast<const uint4*>(a.x + row * a.ldx);
  Row8<RT> sv[VPT];
  float sq = 0.f;
  if constexpr (RT == RES_NONE) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = t + TPR * k;
      sv[k].b = v < nvec ? xr[v] : make_uint4(0, 0, 0, 0);
    }
  } else {
    uint4 xv[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = t + TPR * k;
      xv[k] = v < nvec ? xr[v] : make_uint4(0, 0, 0, 0);
    }
    if constexpr (RT == RES_BF16) {
      const uint4* rr = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.r) + row * a.ldr);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = t + TPR * k;
        sv[k].b = v < nvec ? rr[v] : make_uint4(0, 0, 0, 0);
      }
      uint4* sr = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.s) + row * a.lds);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = t + TPR * k;
        float f[8], g[8];
        unpack8(xv[k], f);
        unpack8(sv[k].b, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += g[j];
        sv[k].b = pack8(f);
        if (v < nvec) sr[v] = sv[k].b;
      }
    } else {
      const float* rr = reinterpret_cast<const float*>(a.r) + row * a.ldr;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = t + TPR * k;
#pragma unroll
        for (int j = 0; j < 8; ++j) sv[k].v[j] = 0.f;
        if (v < nvec) load8_f32(rr + 8 * v, sv[k].v);
      }
      float* sr = reinterpret_cast<float*>(a.s) + row * a.lds;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = t + TPR * k;
        float f[8];
        unpack8(xv[k], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) sv[k].v[j] += f[j];
        if (v < nvec) store8_f32(sr + 8 * v, sv[k].v);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    float f[8];
    sv[k].get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) sq = fmaf(f[j], f[j], sq);
  }
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(sq, 0) / (float)a.d + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = t + TPR * k;
    if (v >= nvec) continue;   // the four lanes of a block stay together: nvec % 4 == 0 where codes are written
    float f[8], w[8];
    sv[k].get(f);
    load_w8(a.w, a.w_f32, v, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];
    const uint4 o = pack8(f);
    if (a.y) reinterpret_cast<uint4*>(a.y + row * a.d)[v] = o;
    if (a.q) {
      uint32_t m = max_u16x2(max_u16x2(mag_pair(o.x), mag_pair(o.y)), max_u16x2(mag_pair(o.z), mag_pair(o.w)));
      m = max_u16x2(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));   // lane ^ 1
      m = max_u16x2(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));   // lane ^ 2
      const int e = mx_exponent(amax_of_pair(m));
      uint2 c;
      if (e != kMxNaN) {
        const float sc = mx_scale_operand(e);
        const uint32_t lim2 = mx_clamp_pair(e);
        c = make_uint2(mx_codes4_pairs(o.x, o.y, sc, lim2), mx_codes4_pairs(o.z, o.w, sc, lim2));
      } else {
        c = make_uint2(mx_nan_codes4_pairs(o.x, o.y), mx_nan_codes4_pairs(o.z, o.w));
      }
      reinterpret_cast<uint2*>(a.q + row * a.d)[v] = c;
      if ((t & 3) == 0) a.qs[row * (a.d / 32) + (v >> 2)] = (uint8_t)(e + 127);
    }
  }
}

// Any d and alignment, bf16 output: thread t holds the elements t, t + TPR, ...
// (neighbouring lanes read neighbouring elements).
template <int TPR, int EPT, int RT>
__global__ __launch_bounds__(TPR) void add_rmsnorm_any_kernel(NormArgs a) {
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const uint16_t* xr = a.x + row * a.ldx;
  float s[EPT];
#pragma unroll
  for (int k = 0; k < EPT; ++k) {
    const int e = t + TPR * k;
    s[k] = e < a.d ? bf16_bits_to_f32(xr[e]) : 0.f;
  }
  if constexpr (RT == RES_BF16) {
    const uint16_t* rr = reinterpret_cast<const uint16_t*>(a.r) + row * a.ldr;
    uint16_t* sr = reinterpret_cast<uint16_t*>(a.s) + row * a.lds;
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int e = t + TPR * k;
      if (e < a.d) {
        const uint32_t b = f32_to_bf16_bits(s[k] + bf16_bits_to_f32(rr[e]));
        sr[e] = (uint16_t)b;
        s[k] = bf16_bits_to_f32(b);
      }
    }
  } else if constexpr (RT == RES_F32) {
    const float* rr = reinterpret_cast<const float*>(a.r) + row * a.ldr;
    float* sr = reinterpret_cast<float*>(a.s) + row * a.lds;
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int e = t + TPR * k;
      if (e < a.d) sr[e] = s[k] += rr[e];
    }
  }
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < EPT; ++k) sq = fmaf(s[k], s[k], sq);
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(sq, 0) / (float)a.d + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < EPT; ++k) {
    const int e = t + TPR * k;
    if (e < a.d) a.y[row * a.d + e] = (uint16_t)f32_to_bf16_bits(s[k] * rstd * load_w1(a.w, a.w_f32, e));
  }
}

// ------------------------------------------------------------------ backward

// Each workgroup walks rows blockIdx, blockIdx + grid, ... (RPW at a time)
// and keeps its share of dw in registers; the next row's loads are in flight
// while a row is reduced and written.  The workgroups' sums go to part and
// are added by norm_dw_kernel in a fixed order: no atomics.
template <int TPR, int VPT, int ST>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_backward_kernel(NormBwdArgs a) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nvec = a.d / 8;
  struct In {
    uint4 dy[VPT];
    Row8<ST> s[VPT], dr[VPT];
    float rstd;
  };
  float w[VPT][8], acc[VPT][8];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = t + TPR * k;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[k][j] = acc[k][j] = 0.f;
    if (v < nvec) load_w8(a.w, a.w_f32, v, w[k]);
  }
  auto load_s = [&](const void* p, int64_t ld, int64_t row, Row8<ST> (&o)[VPT]) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = t + TPR * k;
      if constexpr (ST == RES_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[k].v[j] = 0.f;
        if (v < nvec) load8_f32(reinterpret_cast<const float*>(p) + row * ld + 8 * v, o[k].v);
      } else {
        o[k].b = v < nvec ? reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + row * ld)[v]
                          : make_uint4(0, 0, 0, 0);
      }
    }
  };
  auto load = [&](int64_t row, In& in) {
    in.rstd = a.rstd[row];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = t + TPR * k;
      in.dy[k] = v < nvec ? reinterpret_cast<const uint4*>(a.dy + row * a.lddy)[v] : make_uint4(0, 0, 0, 0);
    }
    load_s(a.s, a.lds, row, in.s);
    if (a.dres) load_s(a.dres, a.lddres, row, in.dr);
  };
  const int64_t step = (int64_t)gridDim.x * RPW;
  int slot = 0;
  auto process = [&](int64_t row, const In& in) {
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float dy[8], s[8];
      unpack8(in.dy[k], dy);
      in.s[k].get(s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = s[j] * in.rstd;
        acc[k][j] = fmaf(dy[j], xh, acc[k][j]);
        dot = fmaf(w[k][j] * dy[j], xh, dot);
      }
    }
    const float c = row_sum<TPR>(dot, slot) / (float)a.d;
    slot ^= 1;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = t + TPR * k;
      if (v >= nvec) continue;
      float dy[8], s[8], o[8], dr[8];
      unpack8(in.dy[k], dy);
      in.s[k].get(s);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = in.rstd * fmaf(w[k][j], dy[j], -(s[j] * in.rstd) * c);
      if (a.dres) {
        in.dr[k].get(dr);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += dr[j];
      }
      if constexpr (ST == RES_F32) {
        store8_f32(a.ds + row * a.d + 8 * v, o);
      }
      reinterpret_cast<uint4*>(a.dx + row * a.d)[v] = pack8(o);
    }
  };
  int64_t row = (int64_t)blockIdx.x * RPW + sub;
  if (row < a.T) {
    In p, q;
    load(row, p);
    for (;;) {
      int64_t next = row + step;
      if (next < a.T) load(next, q);
      process(row, p);
      if (next >= a.T) break;
      row = next;
      next = row + step;
      if (next < a.T) load(next, p);
      process(row, q);
      if (next >= a.T) break;
      row = next;
    }
  }
  float* const out = a.part + (int64_t)blockIdx.x * a.d;
  if constexpr (RPW == 1) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = t + TPR * k;
      if (v < nvec) store8_f32(out + 8 * v, acc[k]);
    }
  } else {
    // the wavefronts' sums meet in LDS
    __shared__ float sum[RPW][TPR * VPT * 8];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[sub][8 * (t + TPR * k) + j] = acc[k][j];
    __syncthreads();
    for (int e = threadIdx.x; e < a.d; e += 256) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < RPW; ++i) v += sum[i][e];
      out[e] = v;
    }
  }
}

// any d and alignment
template <int TPR, int EPT, int ST>
__global__ __launch_bounds__(TPR) void rmsnorm_backward_any_kernel(NormBwdArgs a) {
  const int t = threadIdx.x;
  float acc[EPT];
#pragma unroll
  for (int k = 0; k < EPT; ++k) acc[k] = 0.f;
  auto load_s = [&](const void* p, int64_t at) {
    return ST == RES_F32 ? reinterpret_cast<const float*>(p)[at]
                         : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p)[at]);
  };
  int slot = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float dy[EPT], xh[EPT], dot = 0.f;
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int e = t + TPR * k;
      dy[k] = e < a.d ? bf16_bits_to_f32(a.dy[row * a.lddy + e]) : 0.f;
      xh[k] = e < a.d ? load_s(a.s, row * a.lds + e) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int e = t + TPR * k;
      xh[k] *= rstd;
      acc[k] = fmaf(dy[k], xh[k], acc[k]);
      dy[k] = e < a.d ? dy[k] * load_w1(a.w, a.w_f32, e) : 0.f;
      dot = fmaf(dy[k], xh[k], dot);
    }
    const float c = row_sum<TPR>(dot, slot) / (float)a.d;
    slot ^= 1;
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int e = t + TPR * k;
      if (e >= a.d) continue;
      float o = rstd * (dy[k] - xh[k] * c);
      if (a.dres) o += load_s(a.dres, row * a.lddres + e);
      if constexpr (ST == RES_F32) a.ds[row * a.d + e] = o;
      a.dx[row * a.d + e] = (uint16_t)f32_to_bf16_bits(o);
    }
  }
#pragma unroll
  for (int k = 0; k < EPT; ++k) {
    const int e = t + TPR * k;
    if (e < a.d) a.part[(int64_t)blockIdx.x * a.d + e] = acc[k];
  }
}

// dw[e] = sum over P partial rows: 32 columns x 32 row groups per workgroup
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ part, int P, int d,
                                                       float* __restrict__ dw) {
  __shared__ float sum[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + c;
  float v = 0.f;
  if (e < d) {
#pragma unroll 8
    for (int p = g; p < P; p += 32) v += part[(int64_t)p * d + e];
  }
  sum[g][c] = v;
  __syncthreads();
  if (g == 0 && e < d) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sum[i][c];
    dw[e] = v;
  }
}

namespace {

constexpr int kNormParts = 512;   // partial rows of dw at most (two workgroups per compute unit)

moe_status_t status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

template <int RT>
void launch_norm(const NormArgs& a, bool vec, hipStream_t s) {
  auto go = [&](auto kern, int tpr) {
    const int rpw = tpr < 256 ? 256 / tpr : 1;
    hipLaunchKernelGGL(kern, dim3((unsigned)((a.T + rpw - 1) / rpw)), dim3(tpr < 256 ? 256 : tpr), 0, s, a);
  };
  if (!vec) {
    if (a.d <= 1024) {
      go(add_rmsnorm_any_kernel<256, 4, RT>, 256);
    } else if (a.d <= 8192) {
      go(add_rmsnorm_any_kernel<256, 32, RT>, 256);
    } else {
      go(add_rmsnorm_any_kernel<1024, 32, RT>, 1024);
    }
    return;
  }
  const int nvec = a.d / 8;
  // few rows: many threads each, for the latency; many rows: a wavefront each
  const bool few = a.T <= 4 * (int64_t)moe_host::device_cu_count();
  if (nvec <= 64) {
    go(add_rmsnorm_kernel<64, 1, RT>, 64);
  } else if (few) {
    if (nvec <= 256) {
      go(add_rmsnorm_kernel<256, 1, RT>, 256);
    } else if (nvec <= 1024) {
      go(add_rmsnorm_kernel<1024, 1, RT>, 1024);
    } else {
      go(add_rmsnorm_kernel<1024, 4, RT>, 1024);
    }
  } else if (nvec <= 128) {
    go(add_rmsnorm_kernel<64, 2, RT>, 64);
  } else if (nvec <= 256) {
    go(add_rmsnorm_kernel<64, 4, RT>, 64);
  } else if (nvec <= 512) {
    go(add_rmsnorm_kernel<256, 2, RT>, 256);
  } else if (nvec <= 1024) {
    go(add_rmsnorm_kernel<256, 4, RT>, 256);
  } else {
    go(add_rmsnorm_kernel<1024, 4, RT>, 1024);
  }
}

template <int ST>
void launch_norm_backward(const NormBwdArgs& a, bool vec, int parts, hipStream_t s) {
  auto go = [&](auto kern, int tpr) {
    hipLaunchKernelGGL(kern, dim3((unsigned)parts), dim3(tpr < 256 ? 256 : tpr), 0, s, a);
  };
  const int nvec = a.d / 8;
  if (!vec) {
    if (a.d <= 1024) {
      go(rmsnorm_backward_any_kernel<256, 4, ST>, 256);
    } else if (a.d <= 8192) {
      go(rmsnorm_backward_any_kernel<256, 32, ST>, 256);
    } else {
      go(rmsnorm_backward_any_kernel<1024, 32, ST>, 1024);
    }
  } else if (nvec <= 64) {
    go(rmsnorm_backward_kernel<64, 1, ST>, 64);
  } else if (nvec <= 256) {
    go(rmsnorm_backward_kernel<256, 1, ST>, 256);
  } else if (nvec <= 512) {
    go(rmsnorm_backward_kernel<256, 2, ST>, 256);
  } else if (nvec <= 1024) {
    go(rmsnorm_backward_kernel<256, 4, ST>, 256);
  } else {
    go(rmsnorm_backward_kernel<1024, 4, ST>, 1024);
  }
}

}  // namespace
}  // namespace moe

// Workgroups of the backward: every one holds at least one row
extern "C" int moe_norm_backward_parts(int64_t T) {
  return (int)std::min<int64_t>(T, moe::kNormParts);
}

extern "C" moe_status_t moe_add_rmsnorm_launch(const moe::NormArgs* a, int res, int vec, hipStream_t s) {
  if (res == moe::RES_NONE) {
    moe::launch_norm<moe::RES_NONE>(*a, vec, s);
  } else if (res == moe::RES_BF16) {
    moe::launch_norm<moe::RES_BF16>(*a, vec, s);
  } else {
    moe::launch_norm<moe::RES_F32>(*a, vec, s);
  }
  return moe::status();
}

extern "C" moe_status_t moe_rmsnorm_backward_launch(const moe::NormBwdArgs* a, int s_f32, int vec, float* dw,
                                                    hipStream_t s) {
  const int parts = moe_norm_backward_parts(a->T);
  if (parts > 0) {
    if (s_f32) {
      moe::launch_norm_backward<moe::RES_F32>(*a, vec, parts, s);
    } else {
      moe::launch_norm_backward<moe::RES_BF16>(*a, vec, parts, s);
    }
    if (moe::status() != MOE_OK) return MOE_ERR_HIP;
  }
  hipLaunchKernelGGL(moe::norm_dw_kernel, dim3((unsigned)((a->d + 31) / 32)), dim3(1024), 0, s, a->part, parts, a->d,
                     dw);
  return moe::status();
}
