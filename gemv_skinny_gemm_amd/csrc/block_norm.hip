// block_norm.hip - a block's output into the residual, and the norm behind it
// (skinny_block_norm), on MI355X (gfx950).

#include <hip/hip_runtime.h>

#include <math.h>

#include "host_util.h"
#include "skinny_gemm.h"

namespace {

using skinny_host::DeviceInfo;
using skinny_host::Range;
using skinny_host::aligned;
using skinny_host::device_info;
using skinny_host::overlap;
using skinny_host::range_of;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any address: rows of an odd width begin anywhere, and the hardware
// takes unaligned vector accesses to global memory.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any4 __attribute__((aligned(4)));

constexpr int kUnit = 8;               // neighbouring values of a thread

struct NormArgs {
  const __bf16* block;
  const float* route_weights;
  const void* post_weight;
  const void* post_bias;
  const void* gate;
  const void* residual;
  void* residual_out;
  const void* weight;
  const void* bias;
  __bf16* out;
  int rows, width, routes;
  int layer;                           // SKINNY_NORM_LAYER
  int residual_f32, weight_f32, gate_rows;
  float residual_scale, block_scale, weight_offset;
  double eps;
};

__device__ __forceinline__ float bf16_lo(unsigned u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) {
  return __builtin_bit_cast(float, u & 0xffff0000u);
}
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, bf16x2{(__bf16)a, (__bf16)b});
}

// Values i .. i + 7 of an array, zeros from `width` on.
__device__ __forceinline__ void load_bf16(const __bf16* p, int i, int width, float (&v)[kUnit]) {
  if (i + kUnit <= width) {
    const u32x4 x = *reinterpret_cast<const u32x4_any*>(p + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bf16_lo(x[e]);
      v[2 * e + 1] = bf16_hi(x[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kUnit; ++e) v[e] = i + e < width ? (float)p[i + e] : 0.0f;
  }
}
__device__ __forceinline__ void load_f32(const float* p, int i, int width, float (&v)[kUnit]) {
  if (i + kUnit <= width) {
    const u32x4 x = *reinterpret_cast<const u32x4_any4*>(p + i);
    const u32x4 y = *reinterpret_cast<const u32x4_any4*>(p + i + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned a = x[e], b = y[e];
      v[e] = __builtin_bit_cast(float, a);
      v[4 + e] = __builtin_bit_cast(float, b);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kUnit; ++e) v[e] = i + e < width ? p[i + e] : 0.0f;
  }
}
__device__ __forceinline__ void load(const void* p, int f32, size_t at, int i, int width,
                                     float (&v)[kUnit]) {
  if (f32) load_f32((const float*)p + at, i, width, v);
  else load_bf16((const __bf16*)p + at, i, width, v);
}

__device__ __forceinline__ void store_bf16(__bf16* p, int i, int width, const float (&v)[kUnit]) {
  if (i + kUnit <= width) {
    u32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    *reinterpret_cast<u32x4_any*>(p + i) = x;
  } else {
#pragma unroll
    for (int e = 0; e < kUnit; ++e)
      if (i + e < width) p[i + e] = (__bf16)v[e];
  }
}
__device__ __forceinline__ void store_f32(float* p, int i, int width, const float (&v)[kUnit]) {
  if (i + kUnit <= width) {
    u32x4 x, y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = __builtin_bit_cast(unsigned, v[e]);
      y[e] = __builtin_bit_cast(unsigned, v[4 + e]);
    }
    *reinterpret_cast<u32x4_any4*>(p + i) = x;
    *reinterpret_cast<u32x4_any4*>(p + i + 4) = y;
  } else {
#pragma unroll
    for (int e = 0; e < kUnit; ++e)
      if (i + e < width) p[i + e] = v[e];
  }
}

// The value of the lane that CTRL names within a row of 16 lanes.
template <int CTRL>
__device__ __forceinline__ double from_lane(double x) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xf, 0xf, true);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (unsigned long long)(unsigned)lo |
                                        (unsigned long long)(unsigned)hi << 32);
}
// The sum over the wave, in every lane: neighbours, pairs, then the mirrored
// halves and rows of 16 lanes (whose lanes agree by then), rows, halves.
__device__ __forceinline__ double wave_sum(double x) {
  x += from_lane<0xb1>(x);             // quad_perm 1 0 3 2
  x += from_lane<0x4e>(x);             // quad_perm 2 3 0 1
  x += from_lane<0x141>(x);            // row_half_mirror
  x += from_lane<0x140>(x);            // row_mirror
#pragma unroll
  for (int off = 16; off < 64; off *= 2) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    const auto lo = off == 16
        ? __builtin_amdgcn_permlane16_swap((unsigned)u, (unsigned)u, false, false)
        : __builtin_amdgcn_permlane32_swap((unsigned)u, (unsigned)u, false, false);
    const auto hi = off == 16
        ? __builtin_amdgcn_permlane16_swap((unsigned)(u >> 32), (unsigned)(u >> 32), false, false)
        : __builtin_amdgcn_permlane32_swap((unsigned)(u >> 32), (unsigned)(u >> 32), false, false);
    const unsigned l0 = lo[0], l1 = lo[1], h0 = hi[0], h1 = hi[1];
    x = __builtin_bit_cast(double, (unsigned long long)l0 | (unsigned long long)h0 << 32) +
        __builtin_bit_cast(double, (unsigned long long)l1 | (unsigned long long)h1 << 32);
  }
  return x;
}

// The sum over a row's threads, in every one of them; `part` is used once only.
template <int TPR>
__device__ __forceinline__ double row_sum(double x, double* part) {
  x = wave_sum(x);
  if constexpr (TPR == 64) return x;
  constexpr int kWaves = TPR / 64;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) x += part[w];
  return x;
}

// norm(v) over the row, in place, times (offset + weight) plus bias.
template <int TPR, int CH>
__device__ __forceinline__ void normalise(const NormArgs& a, float (&v)[CH][kUnit], int lane,
                                          const void* weight, const void* bias, double* part) {
  const double n = (double)a.width;
  double mean = 0.0;
  if (a.layer) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < kUnit; ++e)
        if ((c * TPR + lane) * kUnit + e < a.width) s += (double)v[c][e];
    mean = row_sum<TPR>(s, part) / n;
  }
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < kUnit; ++e) {
      const double d = (double)v[c][e] - mean;
      if ((c * TPR + lane) * kUnit + e < a.width) s = fma(d, d, s);
    }
  const double r = 1.0 / sqrt(row_sum<TPR>(s, part + 16) / n + a.eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * TPR + lane) * kUnit;
    if (i >= a.width) continue;
    float w[kUnit];
    if (weight) {
      load(weight, a.weight_f32, 0, i, a.width, w);
#pragma unroll
      for (int e = 0; e < kUnit; ++e) w[e] += a.weight_offset;
    } else {
#pragma unroll
      for (int e = 0; e < kUnit; ++e) w[e] = 1.0f;
    }
#pragma unroll
    for (int e = 0; e < kUnit; ++e) v[c][e] = (float)(((double)v[c][e] - mean) * r) * w[e];
    if (bias) {
      load(bias, a.weight_f32, 0, i, a.width, w);
#pragma unroll
      for (int e = 0; e < kUnit; ++e) v[c][e] += w[e];
    }
  }
}

// TPR threads hold a row in registers, CH runs of kUnit neighbouring values each.
template <int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void skinny_block_norm_k(const NormArgs a) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;   // of a workgroup
  __shared__ double part[2][32];
  const int lane = threadIdx.x % TPR;
  const int row = blockIdx.x * kRows + threadIdx.x / TPR;
  if (row >= a.rows) return;                         // whole waves, and only without a barrier
  const size_t at = (size_t)row * a.width;

  float h[CH][kUnit], b[CH][kUnit];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * TPR + lane) * kUnit;
#pragma unroll
    for (int e = 0; e < kUnit; ++e) h[c][e] = b[c][e] = 0.0f;
    if (i >= a.width) continue;
    if (a.residual) load(a.residual, a.residual_f32, at, i, a.width, h[c]);
    if (!a.block) continue;
    const __bf16* src = a.block + at * a.routes;
    if (!a.route_weights && a.routes == 1) {
      load_bf16(src, i, a.width, b[c]);
      continue;
    }
    for (int j = 0; j < a.routes; ++j) {
      float x[kUnit];
      load_bf16(src + (size_t)j * a.width, i, a.width, x);
      const float w = a.route_weights ? a.route_weights[(size_t)row * a.routes + j] : 1.0f;
#pragma unroll
      for (int e = 0; e < kUnit; ++e) b[c][e] = fmaf(w, x[e], b[c][e]);
    }
  }
  if (a.block) {
    if (a.post_weight) normalise<TPR, CH>(a, b, lane, a.post_weight, a.post_bias, part[0]);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * TPR + lane) * kUnit;
      if (i >= a.width) continue;
      float g[kUnit];
      if (a.gate) {
        load(a.gate, a.weight_f32, a.gate_rows ? at : 0, i, a.width, g);
#pragma unroll
        for (int e = 0; e < kUnit; ++e) b[c][e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < kUnit; ++e) {
        const float x = a.block_scale * b[c][e];
        h[c][e] = a.residual ? fmaf(a.residual_scale, h[c][e], x) : x;
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < kUnit; ++e) h[c][e] *= a.residual_scale;
  }
  if (a.residual_out) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * TPR + lane) * kUnit;
      if (i >= a.width) continue;
      if (a.residual_f32) store_f32((float*)a.residual_out + at, i, a.width, h[c]);
      else store_bf16((__bf16*)a.residual_out + at, i, a.width, h[c]);
    }
  }
  if (!a.out) return;
  normalise<TPR, CH>(a, h, lane, a.weight, a.bias, part[1]);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * TPR + lane) * kUnit;
    if (i < a.width) store_bf16(a.out + at, i, a.width, h[c]);
  }
}

// ---------------------------------------------------------------------------
// Host side.

bool finite(float x) { return x - x == 0.0f; }

template <int TPR, int CH>
skinny_status launch(const NormArgs& a, hipStream_t stream) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  hipLaunchKernelGGL((skinny_block_norm_k<TPR, CH>), dim3((a.rows + kRows - 1) / kRows),
                     dim3(TPR < 256 ? 256 : TPR), 0, stream, a);
  return hipGetLastError() == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP;
}

}  // namespace

extern "C" {

skinny_status skinny_block_norm(const skinny_norm* norm, void* stream) {
  if (!norm || norm->reserved != 0) return SKINNY_ERR_INVALID_ARG;
  const skinny_norm& n = *norm;
  if ((n.kind != SKINNY_NORM_RMS && n.kind != SKINNY_NORM_LAYER) ||
      (n.residual_dtype != SKINNY_VALUES_BF16 && n.residual_dtype != SKINNY_VALUES_F32) ||
      (n.weight_dtype != SKINNY_VALUES_BF16 && n.weight_dtype != SKINNY_VALUES_F32))
    return SKINNY_ERR_INVALID_ARG;
  if (n.rows < 1 || n.width < 1 || n.routes < 1 || (n.gate_rows != 0 && n.gate_rows != 1))
    return SKINNY_ERR_INVALID_ARG;
  if (!finite(n.eps) || n.eps < 0.0f || !finite(n.residual_scale) || !finite(n.block_scale) ||
      !finite(n.weight_offset))
    return SKINNY_ERR_INVALID_ARG;
  if ((!n.block && !n.residual) || (!n.residual_out && !n.out)) return SKINNY_ERR_INVALID_ARG;
  if (!n.block && (n.post_weight || n.post_bias || n.gate || n.route_weights || n.routes != 1))
    return SKINNY_ERR_INVALID_ARG;
  if ((n.post_bias && !n.post_weight) || (!n.out && (n.weight || n.bias)) ||
      (n.gate_rows && !n.gate))
    return SKINNY_ERR_INVALID_ARG;
  if (n.rows > SKINNY_NORM_MAX_ROWS || n.width > SKINNY_NORM_MAX_WIDTH ||
      n.routes > SKINNY_MAX_TOPK)
    return SKINNY_ERR_UNSUPPORTED;
  const size_t rs = n.residual_dtype == SKINNY_VALUES_F32 ? 4 : 2;
  const size_t ws = n.weight_dtype == SKINNY_VALUES_F32 ? 4 : 2;
  const size_t all = (size_t)n.rows * n.width, one = (size_t)n.width;
  struct Operand {
    const void* p;
    size_t bytes, align;
  };
  const Operand in[] = {
      {n.block, all * n.routes * 2, 2},
      {n.route_weights, (size_t)n.rows * n.routes * 4, 4},
      {n.post_weight, one * ws, ws},
      {n.post_bias, one * ws, ws},
      {n.gate, (n.gate_rows ? all : one) * ws, ws},
      {n.weight, one * ws, ws},
      {n.bias, one * ws, ws},
      {n.residual, all * rs, rs},
  };
  const Range out = range_of(n.out, n.out ? all * 2 : 0);
  const Range res = range_of(n.residual_out, n.residual_out ? all * rs : 0);
  if (!aligned(n.out, 2) || !aligned(n.residual_out, rs)) return SKINNY_ERR_UNSUPPORTED;
  for (const Operand& o : in)
    if (!aligned(o.p, o.align)) return SKINNY_ERR_UNSUPPORTED;
  if (n.out && n.residual_out && overlap(out, res)) return SKINNY_ERR_INVALID_ARG;
  for (const Operand& o : in) {
    if (!o.p) continue;
    const Range r = range_of(o.p, o.bytes);
    if (n.out && overlap(out, r)) return SKINNY_ERR_INVALID_ARG;
    if (n.residual_out && overlap(res, r) && !(o.p == n.residual && o.p == n.residual_out &&
                                                &o == &in[7]))
      return SKINNY_ERR_INVALID_ARG;
  }
  DeviceInfo d;
  const skinny_status st = device_info(&d);
  if (st != SKINNY_OK) return st;
  if (!d.gfx950) return SKINNY_ERR_UNSUPPORTED;

  NormArgs a;
  a.block = (const __bf16*)n.block;
  a.route_weights = n.route_weights;
  a.post_weight = n.post_weight;
  a.post_bias = n.post_bias;
  a.gate = n.gate;
  a.residual = n.residual;
  a.residual_out = n.residual_out;
  a.weight = n.weight;
  a.bias = n.bias;
  a.out = (__bf16*)n.out;
  a.rows = n.rows;
  a.width = n.width;
  a.routes = n.routes;
  a.layer = n.kind == SKINNY_NORM_LAYER;
  a.residual_f32 = n.residual_dtype == SKINNY_VALUES_F32;
  a.weight_f32 = n.weight_dtype == SKINNY_VALUES_F32;
  a.gate_rows = n.gate_rows;
  a.residual_scale = n.residual_scale;
  a.block_scale = n.block_scale;
  a.weight_offset = n.weight_offset;
  a.eps = (double)n.eps;
  const hipStream_t hs = (hipStream_t)stream;
  if (n.width <= 512) return launch<64, 1>(a, hs);
  if (n.width <= 2048) return launch<256, 1>(a, hs);
  if (n.width <= 8192) return launch<1024, 1>(a, hs);
  if (n.width <= 16384) return launch<1024, 2>(a, hs);
  return launch<1024, 4>(a, hs);
}

}  // extern "C"
