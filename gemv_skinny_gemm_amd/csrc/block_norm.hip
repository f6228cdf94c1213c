// block_norm.hip - a block's output into the residual, and the norm behind it
// (skinny_block_norm), on MI355X (gfx950).

#include <hip/hip_runtime.h>

#include <math.h>

#include "host_util.h"
#include "skinny_gemm.h"
#include "wave_util.h"

namespace {

using skinny_host::DeviceInfo;
using skinny_host::Range;
using skinny_host::aligned;
using skinny_host::device_info;
using skinny_host::overlap;
using skinny_host::range_of;
using skinny_wave::lanes_sum;
using skinny_wave::wave_sum;

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
  int gate_rows;
  float residual_scale, block_scale, weight_offset;
  double eps, inv_width;
};

__device__ __forceinline__ float bf16_lo(unsigned u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) {
  return __builtin_bit_cast(float, u & 0xffff0000u);
}
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, bf16x2{(__bf16)a, (__bf16)b});
}

// A unit as it lies in memory, and its values.
template <bool F32>
struct Raw {
  u32x4 x[F32 ? 2 : 1];
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (F32) {
      const unsigned u = x[e / 4][e % 4];
      return __builtin_bit_cast(float, u);
    } else {
      const unsigned u = x[0][e / 2];
      return e % 2 ? bf16_hi(u) : bf16_lo(u);
    }
  }
};
template <bool F32>
__device__ __forceinline__ Raw<F32> load(const void* p, size_t at) {
  Raw<F32> r;
  if constexpr (F32) {
    const float* q = (const float*)p + at;
    r.x[0] = *reinterpret_cast<const u32x4_any4*>(q);
    r.x[1] = *reinterpret_cast<const u32x4_any4*>(q + 4);
  } else {
    r.x[0] = *reinterpret_cast<const u32x4_any*>((const __bf16*)p + at);
  }
  return r;
}
// Rows of fewer values than a unit: lane 0 has them all.
template <bool F32>
__device__ __forceinline__ Raw<F32> load_few(const void* p, size_t at, int width) {
  Raw<F32> r{};
#pragma unroll
  for (int e = 0; e < kUnit; ++e) {
    if (e >= width) continue;
    if constexpr (F32) r.x[e / 4][e % 4] = __builtin_bit_cast(unsigned, ((const float*)p)[at + e]);
    else r.x[0][e / 2] |= (unsigned)((const unsigned short*)p)[at + e] << (16 * (e % 2));
  }
  return r;
}

// Values from `skip` up to `end` of a unit.
template <bool F32>
__device__ __forceinline__ void store(void* p, size_t at, const float (&v)[kUnit], int skip, int end) {
  if (skip == 0 && end == kUnit) {
    if constexpr (F32) {
      u32x4 x, y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = __builtin_bit_cast(unsigned, v[e]);
        y[e] = __builtin_bit_cast(unsigned, v[4 + e]);
      }
      *reinterpret_cast<u32x4_any4*>((float*)p + at) = x;
      *reinterpret_cast<u32x4_any4*>((float*)p + at + 4) = y;
    } else {
      u32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
      *reinterpret_cast<u32x4_any*>((__bf16*)p + at) = x;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < kUnit; ++e) {
    if (e < skip || e >= end) continue;
    if constexpr (F32) ((float*)p)[at + e] = v[e];
    else ((__bf16*)p)[at + e] = (__bf16)v[e];
  }
}

// The sum over a row's threads, in every one of them; `part` is used once only.
__device__ __forceinline__ double row_sum(double x, double* part) {
  x = wave_sum(x);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return x;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  const int w = threadIdx.x & 15;
  return lanes_sum<16>(w < waves ? part[w] : 0.0);
}

// 1 / sqrt(x) within 2^-43: the instruction's number, off by e < 2^-22, after one step of
// Newton's method, which leaves 1.5 e^2; 0 and infinity as it has them.
__device__ __forceinline__ double inverse_root(double x) {
  const double r = __builtin_amdgcn_rsq(x);
  const double y = fma(r * 0.5, fma(-x * r, r, 1.0), r);
  return x > 0.0 && x < __builtin_inf() ? y : r;
}

// Where a thread's units lie.  A row's last unit ends with the row: it begins
// `skip` values early, which belong to the unit before it and take no part here,
// so that every load is one of whole units within the row.
template <int CH>
struct Units {
  int at[CH], skip[CH], end;
  __device__ __forceinline__ Units(int lane, int width) {
    end = min(width, kUnit);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * (int)blockDim.x + lane) * kUnit;
      at[c] = max(min(i, width - kUnit), 0);
      skip[c] = i - at[c];
    }
  }
  __device__ __forceinline__ bool has(int c) const { return skip[c] < kUnit; }
  __device__ __forceinline__ bool has(int c, int e) const { return e >= skip[c] && e < end; }
  template <bool F32>
  __device__ __forceinline__ Raw<F32> get(const void* p, size_t row, int c) const {
    if (__builtin_expect(end < kUnit, 0)) return has(c) ? load_few<F32>(p, row, end) : Raw<F32>{};
    return load<F32>(p, row + at[c]);
  }
};

// norm(v) over the row, in place, times (offset + weight) plus bias.  Values that
// take no part are zeros before, and no matter after.
template <int CH, bool WF>
__device__ __forceinline__ void normalise(const NormArgs& a, float (&v)[CH][kUnit],
                                          const Units<CH>& u, const void* weight,
                                          const void* bias, double* part) {
  double mean = 0.0;
  if (a.layer) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < kUnit; ++e) s += (double)v[c][e];
    mean = row_sum(s, part) / (double)a.width;       // a row of one value has exactly that mean
    // In two parts, so that fp32 differences are rounded relative to themselves.
    const float hi = (float)mean, lo = (float)(mean - (double)hi);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < kUnit; ++e) v[c][e] = u.has(c, e) ? (v[c][e] - hi) - lo : 0.0f;
  }
  double s[2] = {0.0, 0.0};
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < kUnit; ++e) s[e % 2] = fma((double)v[c][e], (double)v[c][e], s[e % 2]);
  const double r = inverse_root(fma(row_sum(s[0] + s[1], part + 16), a.inv_width, a.eps));
  // The product in fp32 wherever r is far from its ends.
  const float rf = (float)r;
  const bool mild = rf > 1e-30f && rf < 1e30f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    Raw<WF> w, b;
    if (weight) w = u.template get<WF>(weight, 0, c);
    if (bias) b = u.template get<WF>(bias, 0, c);
    if (__builtin_expect(mild, 1)) {
#pragma unroll
      for (int e = 0; e < kUnit; ++e) v[c][e] *= rf;
    } else {
#pragma unroll
      for (int e = 0; e < kUnit; ++e) v[c][e] = (float)((double)v[c][e] * r);
    }
    if (weight)
#pragma unroll
      for (int e = 0; e < kUnit; ++e) v[c][e] *= a.weight_offset + w[e];
    if (bias)
#pragma unroll
      for (int e = 0; e < kUnit; ++e) v[c][e] += b[e];
  }
}

// A workgroup holds a row in registers, CH units of 8 neighbouring values per
// thread and as many threads as the row has units for; every value is read and
// written once.
//
// What bounds it: many rows the memory.  Rows of 8192 in bf16, block and residual in,
// residual and x out: 16384 of them 180 us = 5.96 TB/s (a plain copy of 2 GiB
// reaches 4.9 in sum), 1024 13.7; with a norm behind the block, too, 213 us = 5.0.
// Few rows the chain launch - loads - sum over the waves - store: 2.4 us at a width
// of 128, 3.3 at 8192, 6.5 with four sums (two LAYER norms).
//   One unit per thread, against rows of 8192 in 512 threads of two units and 256 of
// four: 180 / 190 / 194 us (16384 rows), 3.2 / 3.5 / 5.0 (one); rows of 4096 in
// 512, 1024 (half of them idle) and 256 threads: 91 / 108 / 93.  Two units from 8193
// values on, four from 16385, whose registers spill whatever the types (17 of bf16, 88 of
// fp32 operands).  2^27 values, bf16 RMS without a norm of the block, in rows of 8192,
// 16384 and 32768: 180 / 191 / 199 us; fp32 residual and weights, two LAYER norms: 355 /
// 418 / 529 (1.6 GB, 3.0 TB/s).
//   A kernel of 64 registers has two workgroups of 16 waves on a CU; 65 had one, and
// 16384 rows of 8192 with two LAYER norms in fp32 took 481 us instead of 422 (two
// registers spill there).
// Loading weights before the sums, to have them at hand behind, costs those
// registers and gained nothing at one row.  Several one-wave rows per workgroup gain
// nothing either (16384 rows of 512: 12.4 us alone, 12.9 by fours), nor do dwords
// around bf16 units of odd rows (16384 x 5001: 201 us, 208 with them).
template <int CH, bool RF, bool WF>
__global__ __launch_bounds__(1024) __attribute__((amdgpu_waves_per_eu(CH == 1 ? 8 : 4)))
void skinny_block_norm_k(const NormArgs a) {
  __shared__ double part[2][32];
  constexpr bool kAhead = CH <= 2;     // registers are left for loads ahead of their use
  const int row = blockIdx.x;
  const size_t at = (size_t)row * a.width;
  const Units<CH> u(threadIdx.x, a.width);

  float v[CH][kUnit];
  Raw<RF> res[CH];
  if (a.residual && (kAhead || !a.block))
#pragma unroll
    for (int c = 0; c < CH; ++c) res[c] = u.template get<RF>(a.residual, at, c);
  if (a.block) {
    const size_t first = at * a.routes;
    Raw<false> x[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) x[c] = u.template get<false>(a.block, first, c);
    if (a.routes == 1 && !a.route_weights) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < kUnit; ++e) v[c][e] = x[c][e];
    } else {
      const float* rw = a.route_weights ? a.route_weights + (size_t)row * a.routes : nullptr;
      for (int j = 0; j < a.routes; ++j) {
        Raw<false> next[CH];
        const int k = min(j + 1, a.routes - 1);
        if constexpr (kAhead)
#pragma unroll
          for (int c = 0; c < CH; ++c)
            next[c] = u.template get<false>(a.block, first + (size_t)k * a.width, c);
        const float w = rw ? rw[j] : 1.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < kUnit; ++e) v[c][e] = j ? fmaf(w, x[c][e], v[c][e]) : w * x[c][e];
#pragma unroll
        for (int c = 0; c < CH; ++c)
          x[c] = kAhead ? next[c] : u.template get<false>(a.block, first + (size_t)k * a.width, c);
      }
    }
    if (a.post_weight) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < kUnit; ++e)
          if (!u.has(c, e)) v[c][e] = 0.0f;
      normalise<CH, WF>(a, v, u, a.post_weight, a.post_bias, part[0]);
    }
    if (a.gate)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const Raw<WF> g = u.template get<WF>(a.gate, a.gate_rows ? at : 0, c);
#pragma unroll
        for (int e = 0; e < kUnit; ++e) v[c][e] *= g[e];
      }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < kUnit; ++e) v[c][e] *= a.block_scale;
    if (a.residual)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if constexpr (!kAhead) res[c] = u.template get<RF>(a.residual, at, c);
#pragma unroll
        for (int e = 0; e < kUnit; ++e) v[c][e] = fmaf(a.residual_scale, res[c][e], v[c][e]);
      }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < kUnit; ++e) v[c][e] = a.residual_scale * res[c][e];
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < kUnit; ++e)
      if (!u.has(c, e)) v[c][e] = 0.0f;
  if (a.residual_out)
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (u.has(c)) store<RF>(a.residual_out, at + u.at[c], v[c], u.skip[c], u.end);
  if (!a.out) return;
  normalise<CH, WF>(a, v, u, a.weight, a.bias, part[1]);
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (u.has(c)) store<false>(a.out, at + u.at[c], v[c], u.skip[c], u.end);
}

// ---------------------------------------------------------------------------
// Host side.

bool finite(float x) { return x - x == 0.0f; }

template <int CH>
skinny_status launch(const NormArgs& a, bool rf, bool wf, hipStream_t stream) {
  const int units = (a.width + CH * kUnit - 1) / (CH * kUnit);
  const dim3 grid(a.rows), threads((units + 63) / 64 * 64);
  if (rf && wf) hipLaunchKernelGGL((skinny_block_norm_k<CH, true, true>), grid, threads, 0, stream, a);
  else if (rf) hipLaunchKernelGGL((skinny_block_norm_k<CH, true, false>), grid, threads, 0, stream, a);
  else if (wf) hipLaunchKernelGGL((skinny_block_norm_k<CH, false, true>), grid, threads, 0, stream, a);
  else hipLaunchKernelGGL((skinny_block_norm_k<CH, false, false>), grid, threads, 0, stream, a);
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
  a.gate_rows = n.gate_rows;
  a.residual_scale = n.residual_scale;
  a.block_scale = n.block_scale;
  a.weight_offset = n.weight_offset;
  a.eps = (double)n.eps;
  a.inv_width = 1.0 / n.width;
  const hipStream_t hs = (hipStream_t)stream;
  const bool rf = n.residual_dtype == SKINNY_VALUES_F32, wf = n.weight_dtype == SKINNY_VALUES_F32;
  if (a.width <= 1024 * kUnit) return launch<1>(a, rf, wf, hs);
  if (a.width <= 2048 * kUnit) return launch<2>(a, rf, wf, hs);
  return launch<4>(a, rf, wf, hs);
}

}  // extern "C"
