// One AdamW step over many tensors in one pass.
//
//   g = grad * grad_scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// Bound: HBM (28 bytes an element with fp32 states, master weights and bf16
// gradients; 10.1 with 8-bit states and bf16 weights).  A workgroup takes one
// chunk of one tensor; the tensors' addresses travel in the kernel's
// arguments.  All arithmetic is fp32.
//
// 8-bit states: m and sqrt(v) as E4M3 codes with one E8M0 scale per 32
// consecutive elements, 2^e the smallest power of two with amax <= 448 * 2^e.
// sqrt(v), not v: its range is half v's in octaves, and E4M3 spans 18.  The
// codes are rounded up or down at random in proportion to the distance: one
// step moves v by a fraction 1 - b2 of itself, far below half of a code's
// step, so that rounding to nearest would never let it decay.  bf16 weights
// without a master copy are rounded in the same way for the same reason.
// The random bits are a hash of (seed, step, tensor, element): no state, the
// same on every run, no matter how the work is split.
#include "common.h"
#include "dense_args.h"

namespace moe {

enum { PM_MASTER = 0, PM_BF16 = 1, PM_F32 = 2 };   // bf16 weight and fp32 master; bf16 alone; fp32 alone

__host__ __device__ __forceinline__ uint32_t mix32(uint32_t v) {
  v = (v ^ (v >> 16)) * 0x7FEB352Du;
  v = (v ^ (v >> 15)) * 0x846CA68Bu;
  return v ^ (v >> 16);
}

// the smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), clamped to
// [-127, 127]; kMxNaN for a NaN or infinite amax
__device__ __forceinline__ int state_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int ef = (int)(b >> 23);
  if (ef == 0) return -127;
  if (ef == 255) return kMxNaN;
  return max(-127, min(127, ef - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u)));
}

// a value scaled into [-448, 448], rounded to the E4M3 grid by 16 random
// bits: the low 20 mantissa bits are cut after the bits were added at their
// top; below the smallest normal, 2^-6 is added first so that the cut falls
// on the subnormals' grid of 2^-9
__device__ __forceinline__ float round_e4m3(float a, uint32_t rnd16) {
  const float mag = fabsf(a);
  const bool low = mag < 0.015625f;
  const float base = low ? mag + 0.015625f : mag;
  const float cut = __uint_as_float((__float_as_uint(base) + (rnd16 << 4)) & 0xFFF00000u);
  return copysignf(low ? cut - 0.015625f : cut, a);
}

__device__ __forceinline__ uint32_t round_bf16(float p, uint32_t rnd16) {
  const uint32_t u = __float_as_uint(p);
  if ((u & 0x7F800000u) == 0x7F800000u) return f32_to_bf16_bits(p);
  return (u + rnd16) >> 16;
}

__device__ __forceinline__ void ldf8(const float* p, float* f) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void stf8(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
// eight E4M3 codes times 2^e
__device__ __forceinline__ void ld_codes8(uint2 q, uint8_t scale, float* f) {
  const float s = scale == 255 ? __uint_as_float(0x7FC00000u) : mx_scale_operand((int)scale - 127);
  const float tiny = scale == 0 ? __uint_as_float(0x00400000u) : s;   // 2^-127 is subnormal
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = h ? (int)q.y : (int)q.x;
    f[4 * h + 0] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * tiny;
    f[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * tiny;
    f[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * tiny;
    f[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * tiny;
  }
}

// The codes of eight neighbouring elements of a block whose other elements
// the three neighbouring lanes hold; returns the scale byte.
__device__ __forceinline__ uint32_t st_codes8(const float* f, const uint32_t* rnd, int sh, uint2& q) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = mx_absmax(m, f[j]);
  m = mx_absmax(m, __shfl_xor(m, 1, 64));
  m = mx_absmax(m, __shfl_xor(m, 2, 64));
  const int e = state_exponent(m);
  if (e == kMxNaN) {
    q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    return 255u;
  }
  float o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = round_e4m3(scale_pow2(f[j], e), (rnd[j] >> sh) & 0xFFFFu);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(o[0], o[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(o[2], o[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(o[4], o[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(o[6], o[7], hi, true);
  q = make_uint2((uint32_t)lo, (uint32_t)hi);
  return (uint32_t)(e + 127);
}

template <bool S8, int PM, bool G32>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwArgs a) {
  // the chunk's tensor: the last one that starts at or before this workgroup
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.start[mid] <= blockIdx.x) lo = mid; else hi = mid - 1;
  }
  const AdamwTensor t = a.t[lo];
  const float gs = a.gscale ? *a.gscale : 1.0f;
  if ((__float_as_uint(gs) & 0x7F800000u) == 0x7F800000u) return;   // a step to be skipped
  const int64_t base = (int64_t)(blockIdx.x - a.start[lo]) * kAdamwChunk;
  // 1 / (1 - b1^t) and 1 / sqrt(1 - b2^t), in 64 bits once per workgroup
  __shared__ float corr[2];
  const int32_t step = *a.step + 1;
  if (threadIdx.x < 2) {
    const double c = -expm1((double)step * (threadIdx.x ? a.log_b2 : a.log_b1));
    corr[threadIdx.x] = (float)(threadIdx.x ? 1.0 / sqrt(c) : 1.0 / c);
  }
  __syncthreads();
  const float ic1 = corr[0], ic2 = corr[1];
  const uint32_t key = mix32(mix32(mix32(a.seed) ^ (uint32_t)step) ^ (uint32_t)(a.first + lo));
  const uint32_t hkey = mix32(key ^ (uint32_t)(base >> 32));   // a chunk never crosses a multiple of 2^32
  const uintptr_t bits = (uintptr_t)t.p | (uintptr_t)t.master | (uintptr_t)t.g | (S8 ? 0 : (uintptr_t)t.m | (uintptr_t)t.v);
  const uintptr_t bits8 = S8 ? (uintptr_t)t.m | (uintptr_t)t.v : 0;
  const bool vec = (bits & 15) == 0 && (bits8 & 7) == 0;
#pragma unroll 1
  for (int it = 0; it < kAdamwChunk / 2048; ++it) {
    const int64_t i0 = base + it * 2048 + threadIdx.x * 8;
    // whole wavefronts leave together where the states are 8-bit: the four
    // lanes of a block exchange their largest values
    if (i0 - (S8 ? (threadIdx.x & 63) * 8 : 0) >= t.n) break;
    const bool full = vec && i0 + 8 <= t.n;
    const int live = (int)max((int64_t)0, min((int64_t)8, t.n - i0));
    float g[8], p[8], m[8], v[8];
    if (full) {
      if constexpr (G32) {
        ldf8(reinterpret_cast<const float*>(t.g) + i0, g);
      } else {
        unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(t.g) + i0), g);
      }
      if constexpr (PM == PM_MASTER) {
        ldf8(t.master + i0, p);
      } else if constexpr (PM == PM_F32) {
        ldf8(reinterpret_cast<const float*>(t.p) + i0, p);
      } else {
        unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(t.p) + i0), p);
      }
      if constexpr (S8) {
        const uint2 qm = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(t.m) + i0);
        const uint2 qv = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(t.v) + i0);
        ld_codes8(qm, t.ms[i0 >> 5], m);
        ld_codes8(qv, t.vs[i0 >> 5], v);
      } else {
        ldf8(reinterpret_cast<const float*>(t.m) + i0, m);
        ldf8(reinterpret_cast<const float*>(t.v) + i0, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] = p[j] = m[j] = v[j] = 0.f;
        if (j < live) {
          const int64_t i = i0 + j;
          g[j] = G32 ? reinterpret_cast<const float*>(t.g)[i]
                     : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(t.g)[i]);
          p[j] = PM == PM_MASTER ? t.master[i]
                 : PM == PM_F32  ? reinterpret_cast<const float*>(t.p)[i]
                                 : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(t.p)[i]);
          if constexpr (!S8) {
            m[j] = reinterpret_cast<const float*>(t.m)[i];
            v[j] = reinterpret_cast<const float*>(t.v)[i];
          }
        }
      }
      if constexpr (S8) {
        if (live > 0) {
          uint32_t qm[2] = {0, 0}, qv[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j < live) {
              qm[j >> 2] |= (uint32_t)reinterpret_cast<const uint8_t*>(t.m)[i0 + j] << (8 * (j & 3));
              qv[j >> 2] |= (uint32_t)reinterpret_cast<const uint8_t*>(t.v)[i0 + j] << (8 * (j & 3));
            }
          }
          ld_codes8(make_uint2(qm[0], qm[1]), t.ms[i0 >> 5], m);
          ld_codes8(make_uint2(qv[0], qv[1]), t.vs[i0 >> 5], v);
        }
      }
    }
    uint32_t rnd[8];
    if constexpr (S8 || PM == PM_BF16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) rnd[j] = mix32((uint32_t)(i0 + j) + hkey);
    }
    float sv[8];   // sqrt(v)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = g[j] * gs;
      if constexpr (S8) v[j] *= v[j];
      m[j] = fmaf(a.b1, m[j], a.omb1 * gj);
      v[j] = fmaf(a.b2, v[j], a.omb2 * gj * gj);
      sv[j] = sqrtf(v[j]);
      const float upd = (m[j] * ic1) * __builtin_amdgcn_rcpf(fmaf(sv[j], ic2, a.eps));
      p[j] = fmaf(-a.lr, fmaf(a.wd, p[j], upd), p[j]);
    }
    uint2 qm, qv;
    uint32_t em = 0, ev = 0;
    if constexpr (S8) {
      em = st_codes8(m, rnd, 0, qm);
      ev = st_codes8(sv, rnd, 16, qv);
    }
    uint32_t pb[8];
    if constexpr (PM == PM_BF16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) pb[j] = round_bf16(p[j], mix32(rnd[j] + 0x9E3779B9u) & 0xFFFFu);
    }
    if constexpr (S8) {
      if ((threadIdx.x & 3) == 0 && live > 0) {
        t.ms[i0 >> 5] = (uint8_t)em;
        t.vs[i0 >> 5] = (uint8_t)ev;
      }
    }
    if (full) {
      if constexpr (PM == PM_MASTER) {
        stf8(t.master + i0, p);
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(t.p) + i0) = pack8(p);
      } else if constexpr (PM == PM_F32) {
        stf8(reinterpret_cast<float*>(t.p) + i0, p);
      } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(t.p) + i0) =
            make_uint4(pb[0] | (pb[1] << 16), pb[2] | (pb[3] << 16), pb[4] | (pb[5] << 16), pb[6] | (pb[7] << 16));
      }
      if constexpr (S8) {
        *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(t.m) + i0) = qm;
        *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(t.v) + i0) = qv;
      } else {
        stf8(reinterpret_cast<float*>(t.m) + i0, m);
        stf8(reinterpret_cast<float*>(t.v) + i0, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < live) {
          const int64_t i = i0 + j;
          if constexpr (PM == PM_MASTER) {
            t.master[i] = p[j];
            reinterpret_cast<uint16_t*>(t.p)[i] = (uint16_t)f32_to_bf16_bits(p[j]);
          } else if constexpr (PM == PM_F32) {
            reinterpret_cast<float*>(t.p)[i] = p[j];
          } else {
            reinterpret_cast<uint16_t*>(t.p)[i] = (uint16_t)pb[j];
          }
          if constexpr (S8) {
            reinterpret_cast<uint8_t*>(t.m)[i] = (uint8_t)((j < 4 ? qm.x : qm.y) >> (8 * (j & 3)));
            reinterpret_cast<uint8_t*>(t.v)[i] = (uint8_t)((j < 4 ? qv.x : qv.y) >> (8 * (j & 3)));
          } else {
            reinterpret_cast<float*>(t.m)[i] = m[j];
            reinterpret_cast<float*>(t.v)[i] = v[j];
          }
        }
      }
    }
  }
}

// after every tensor's launch: the counter moves on, unless the step was skipped
__global__ void adamw_advance_kernel(int32_t* step, const float* gscale) {
  if (gscale && (__float_as_uint(*gscale) & 0x7F800000u) == 0x7F800000u) return;
  *step += 1;
}

}  // namespace moe

extern "C" moe_status_t moe_adamw_launch(const moe::AdamwArgs* a, uint32_t chunks, int s8, int pm, int g32,
                                         hipStream_t s) {
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(chunks), dim3(256), 0, s, *a); };
  auto with_pm = [&](auto s8c, auto g32c) {
    constexpr bool S = decltype(s8c)::value, G = decltype(g32c)::value;
    if (pm == moe::PM_MASTER) {
      go(moe::adamw_kernel<S, moe::PM_MASTER, G>);
    } else if (pm == moe::PM_BF16) {
      go(moe::adamw_kernel<S, moe::PM_BF16, G>);
    } else {
      go(moe::adamw_kernel<S, moe::PM_F32, G>);
    }
  };
  using T = std::integral_constant<bool, true>;
  using F = std::integral_constant<bool, false>;
  if (s8) {
    if (g32) with_pm(T(), T()); else with_pm(T(), F());
  } else {
    if (g32) with_pm(F(), T()); else with_pm(F(), F());
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

extern "C" moe_status_t moe_adamw_advance_launch(int32_t* step, const float* gscale, hipStream_t s) {
  hipLaunchKernelGGL(moe::adamw_advance_kernel, dim3(1), dim3(1), 0, s, step, gscale);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
