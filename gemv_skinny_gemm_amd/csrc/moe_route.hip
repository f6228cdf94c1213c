// moe_route.hip - a router's logits into experts' ids and weights
// (skinny_moe_route), on MI355X (gfx950).

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

typedef unsigned long long u64;

constexpr int kWaves = 4;              // rows of a workgroup, one per wave
constexpr double kNegInf = -__builtin_inf();

struct RouteArgs {
  const void* logits;
  const float* bias;
  int* ids;
  float* weights;
  int rows, experts, topk, groups, each, top_groups;
  int f32, sigmoid, renormalize;
  double scale;
};

// Unsigned numbers that order as x does; every one is above 0, which stands
// for what is not to be chosen.
__device__ __forceinline__ u64 key_of(double x) {
  const u64 u = __builtin_bit_cast(u64, x + 0.0);    // -0 counts as 0
  return u >> 63 ? ~u : u | 1ull << 63;
}

__device__ __forceinline__ u64 wave_max(u64 x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const u64 y = __shfl_xor(x, off);
    x = x > y ? x : y;
  }
  return x;
}
__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = min(x, __shfl_xor(x, off));
  return x;
}
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
  return x;
}

// A wave takes a row; lane holds experts lane, lane + 64, ..
template <int V>
__global__ __launch_bounds__(64 * kWaves) void skinny_moe_route_k(const RouteArgs a) {
  __shared__ double shared[kWaves][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = blockIdx.x * kWaves + wave;
  if (row >= a.rows) return;           // whole waves; the kernel has no barrier
  double l[V], s[V];
  double top = kNegInf;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 64 * v + lane;
    float x = -__builtin_inff();
    if (e < a.experts) {
      const size_t at = (size_t)row * a.experts + e;
      x = a.f32 ? ((const float*)a.logits)[at] : (float)((const __bf16*)a.logits)[at];
      if (x != x) x = -__builtin_inff();
      x = fminf(x, __FLT_MAX__);
    }
    l[v] = x;
    top = fmax(top, l[v]);
  }
  double total = 0.0;
  if (a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const double t = exp(-fabs(l[v]));
      s[v] = (l[v] >= 0.0 ? 1.0 : t) / (1.0 + t);
    }
  } else {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmax(top, __shfl_xor(top, off));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = top == kNegInf ? 0.0 : exp(l[v] - top);
      total += s[v];
    }
    total = wave_sum(total);
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = total > 0.0 ? s[v] / total : 0.0;
  }
  u64 key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 64 * v + lane;
    double c = l[v];
    if (a.bias && e < a.experts) {
      c = s[v] + (double)a.bias[e];
      if (c != c) c = kNegInf;
    }
    l[v] = c;
    key[v] = e < a.experts ? key_of(c) : 0;
  }
  if (a.groups > 1) {
    // Lane g ranks group g from the wave's own part of the shared memory.
    double* c = shared[wave];
#pragma unroll
    for (int v = 0; v < V; ++v) c[64 * v + lane] = l[v];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    u64 worth = 0;
    if (lane < a.groups) {
      double first = kNegInf, second = kNegInf;
      for (int i = 0; i < a.each; ++i) {
        const double x = c[lane * a.each + i];
        second = fmax(second, fmin(first, x));
        first = fmax(first, x);
      }
      double w = first;
      if (a.bias && a.each > 1) {
        w += second;
        if (w != w) w = kNegInf;
      }
      worth = key_of(w);
    }
    u64 kept = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      const u64 best = wave_max(worth);
      const int g = __builtin_ctzll(__ballot(worth == best));
      kept |= 1ull << g;
      if (lane == g) worth = 0;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!(kept >> ((64 * v + lane) / a.each & 63) & 1)) key[v] = 0;
  }
  double mine = 0.0;                   // lane j: the score of choice j
  int id = 0;
  for (int j = 0; j < a.topk; ++j) {
    u64 best = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) best = best > key[v] ? best : key[v];
    best = wave_max(best);
    int e = 64 * V;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
      if (key[v] == best) e = 64 * v + lane;
    e = wave_min(e);
    double got = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e == 64 * v + lane) {
        got = s[v];
        key[v] = 0;
      }
    got = __shfl(got, e & 63);
    if (lane == j) {
      mine = got;
      id = e;
    }
  }
  if (a.renormalize) {
    total = wave_sum(mine);
    mine = total > 0.0 ? mine / total : 0.0;
  }
  if (lane < a.topk) {
    const size_t at = (size_t)row * a.topk + lane;
    a.ids[at] = id;
    a.weights[at] = (float)(mine * a.scale);
  }
}

template <int V>
skinny_status launch(const RouteArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((skinny_moe_route_k<V>), dim3((a.rows + kWaves - 1) / kWaves),
                     dim3(64 * kWaves), 0, stream, a);
  return hipGetLastError() == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP;
}

}  // namespace

extern "C" {

skinny_status skinny_moe_route(const skinny_route* route, void* stream) {
  if (!route || route->reserved != 0) return SKINNY_ERR_INVALID_ARG;
  const skinny_route& r = *route;
  if ((r.dtype != SKINNY_VALUES_BF16 && r.dtype != SKINNY_VALUES_F32) ||
      (r.scoring != SKINNY_ROUTE_SOFTMAX && r.scoring != SKINNY_ROUTE_SIGMOID) ||
      (r.renormalize != 0 && r.renormalize != 1))
    return SKINNY_ERR_INVALID_ARG;
  if (r.rows < 1 || r.experts < 1 || r.topk < 1 || r.groups < 1 || r.top_groups < 1 ||
      r.top_groups > r.groups || r.experts % r.groups != 0 ||
      (long long)r.top_groups * (r.experts / r.groups) < r.topk || !(r.scale - r.scale == 0.0f))
    return SKINNY_ERR_INVALID_ARG;
  if (!r.logits || !r.ids || !r.weights) return SKINNY_ERR_INVALID_ARG;
  if (r.rows > SKINNY_ROUTE_MAX_ROWS || r.experts > SKINNY_ROUTE_MAX_EXPERTS ||
      r.topk > SKINNY_MAX_TOPK || r.groups > SKINNY_ROUTE_MAX_GROUPS)
    return SKINNY_ERR_UNSUPPORTED;
  const size_t es = r.dtype == SKINNY_VALUES_F32 ? 4 : 2;
  if (!aligned(r.logits, es) || !aligned(r.bias, 4) || !aligned(r.ids, 4) || !aligned(r.weights, 4))
    return SKINNY_ERR_UNSUPPORTED;
  const Range lr = range_of(r.logits, (size_t)r.rows * r.experts * es);
  const Range br = range_of(r.bias, r.bias ? (size_t)r.experts * 4 : 0);
  const Range ir = range_of(r.ids, (size_t)r.rows * r.topk * 4);
  const Range wr = range_of(r.weights, (size_t)r.rows * r.topk * 4);
  if (overlap(ir, wr) || overlap(ir, lr) || overlap(wr, lr) ||
      (r.bias && (overlap(ir, br) || overlap(wr, br))))
    return SKINNY_ERR_INVALID_ARG;
  DeviceInfo d;
  const skinny_status st = device_info(&d);
  if (st != SKINNY_OK) return st;
  if (!d.gfx950) return SKINNY_ERR_UNSUPPORTED;

  RouteArgs a;
  a.logits = r.logits;
  a.bias = r.bias;
  a.ids = r.ids;
  a.weights = r.weights;
  a.rows = r.rows;
  a.experts = r.experts;
  a.topk = r.topk;
  a.groups = r.groups;
  a.each = r.experts / r.groups;
  a.top_groups = r.top_groups;
  a.f32 = r.dtype == SKINNY_VALUES_F32;
  a.sigmoid = r.scoring == SKINNY_ROUTE_SIGMOID;
  a.renormalize = r.renormalize;
  a.scale = (double)r.scale;
  const hipStream_t hs = (hipStream_t)stream;
  if (r.experts <= 64) return launch<1>(a, hs);
  if (r.experts <= 128) return launch<2>(a, hs);
  if (r.experts <= 256) return launch<4>(a, hs);
  if (r.experts <= 512) return launch<8>(a, hs);
  return launch<16>(a, hs);
}

}  // extern "C"
