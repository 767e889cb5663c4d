// Kernel arguments of the dense operators around the expert layer, shared by
// their entry points (abi_dense.cpp) and kernels.  Plain host C++.
#pragma once
#include <cstddef>
#include <cstdint>

namespace moe {

// A launch dimension holds fewer than 2^32 threads: workgroup numbers past
// kGridX continue in y (workgroup = y * kGridX + x), a multiple of 8 that keeps
// a workgroup's XCD its number modulo 8.
constexpr int64_t kGridX = 1 << 20;
inline int64_t grid_x(int64_t workgroups) { return workgroups < kGridX ? workgroups : kGridX; }
inline int64_t grid_y(int64_t workgroups) { return (workgroups + kGridX - 1) / kGridX; }

enum { RES_NONE = 0, RES_BF16 = 1, RES_F32 = 2 };

struct NormArgs {
  const uint16_t* x;
  const void* r;          // residual: bf16 or fp32 rows, or NULL
  const void* w;          // weight: bf16 or fp32 [d]
  void* s;                // stored sum, in the residual's type
  uint16_t* y;            // bf16 output or NULL
  uint8_t* q;             // MXFP8 output or NULL
  uint8_t* qs;
  float* rstd;            // or NULL
  int64_t T, ldx, ldr, lds;
  int d;
  int w_f32;
  float eps;
};

struct NormBwdArgs {
  const uint16_t* dy;
  const void* s;          // bf16 or fp32
  const void* w;
  const float* rstd;
  const void* dres;       // in the type of s, or NULL
  uint16_t* dx;           // bf16
  float* ds;              // fp32 (s in fp32), or NULL
  float* part;            // [parts, d] column sums of each workgroup's rows
  int64_t T, lddy, lds, lddres;
  int d;
  int w_f32;
};

// One launch of the optimiser step: up to kAdamwTensors tensors, passed by
// value (no copy to the device, and a captured call keeps them)
constexpr int kAdamwTensors = 40;
constexpr int kAdamwChunk = 8192;   // elements per workgroup

struct AdamwTensor {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  int64_t n;
};

struct AdamwArgs {
  AdamwTensor t[kAdamwTensors];
  uint32_t start[kAdamwTensors + 1];   // first workgroup of each tensor
  int32_t count;
  int32_t first;                       // the first tensor's index in the whole list
  const int32_t* step;
  const float* gscale;
  double log_b1, log_b2;
  float lr, b1, b2, omb1, omb2, eps, wd;
  uint32_t seed;
};
static_assert(sizeof(AdamwArgs) <= 4000, "kernel arguments");

}  // namespace moe
