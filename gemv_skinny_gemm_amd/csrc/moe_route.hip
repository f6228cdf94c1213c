// moe_route.hip - a router's logits into experts' ids and weights
// (skinny_moe_route), on MI355X (gfx950).

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
using skinny_wave::u64;
using skinny_wave::wave_max;
using skinny_wave::wave_sum;

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

// Unsigned numbers that order as x does; every one is above 0, which stands for
// what is not to be chosen.
__device__ __forceinline__ u64 key_of(double x) {
  const u64 u = __builtin_bit_cast(u64, x + 0.0);    // -0 counts as 0
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x + 0.0f);
  return u >> 31 ? ~u : u | 1u << 31;
}

__device__ __forceinline__ double sigmoid(double l) {
  const double t = exp(-fabs(l));
  return (l >= 0.0 ? 1.0 : t) / (1.0 + t);
}

__device__ __forceinline__ float of_lane(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
__device__ __forceinline__ double of_lane(double x, int lane) {
  const u64 u = __builtin_bit_cast(u64, x);
  const unsigned lo = __builtin_amdgcn_readlane((unsigned)u, lane);
  const unsigned hi = __builtin_amdgcn_readlane((unsigned)(u >> 32), lane);
  return __builtin_bit_cast(double, (u64)lo | (u64)hi << 32);
}

// The lanes that hold the wave's largest key.
__device__ __forceinline__ u64 lanes_of_max(unsigned key) { return __ballot(key == wave_max(key)); }
__device__ __forceinline__ u64 lanes_of_max(u64 key) {
  // By their upper halves, and by the lower ones where those do not tell.
  const unsigned hi = (unsigned)(key >> 32), top = wave_max(hi);
  const u64 equal = __ballot(hi == top);
  if ((equal & (equal - 1)) == 0) return equal;
  const unsigned lo = hi == top ? (unsigned)key : 0, most = wave_max(lo);
  return __ballot(hi == top && lo == most);
}

// What the wave wrote to its own shared memory, for its other lanes.
__device__ __forceinline__ void in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wave takes a row; lane l holds experts l, l + 64, ..  Without a bias (Key
// unsigned) the choice goes by the logits, in 32 bits, and only chosen ones are
// exponentiated, unless the weights are shares of all; with one (Key u64) all scores
// are needed, in 64 bits.  A bf16 logit leaves 16 bits of its key for the expert's
// number (PACKED), lower ones the larger, so that no two keys are equal and the
// largest says which it is.
//
// What bounds it: the wave's instructions, of few rows their chain (1 row of 8 experts
// 2.1 us, which is a launch; 16 rows of 256 biased experts in groups 7.5: 12 times the
// largest of the wave's 64-bit keys), of many their number: 16384 rows of bf16, 6 of
// 161 experts each, in 8.5 us, 16 of 1024 in 32, 8 of 256 biased ones in 32, where
// reading the logits would take 1.2, 7 and 1.9.  With the number apart from the key, as
// fp32 logits need it (11.2 and 54 us), the first two took 11.1 and 60.
// There each lane's own largest key is found again in every turn: ballots over every
// place instead, to find the first of equals, took 84 us for the 60.
template <int V, typename Key, bool PACKED>
__global__ __launch_bounds__(64 * kWaves) void skinny_moe_route_k(const RouteArgs a) {
  constexpr bool kBiased = sizeof(Key) == 8;
  // Groups' members side by side, one place between groups to spread them over the banks.
  __shared__ double members[kBiased ? kWaves : 1][kBiased ? 64 * V + SKINNY_ROUTE_MAX_GROUPS : 1];
  __shared__ unsigned best_of[kWaves][SKINNY_ROUTE_MAX_GROUPS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = blockIdx.x * kWaves + wave;
  if (row >= a.rows) return;           // whole waves; the kernel has no barrier
  float l[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = min(64 * v + lane, a.experts - 1);
    const size_t at = (size_t)row * a.experts + e;
    l[v] = !PACKED && a.f32 ? ((const float*)a.logits)[at] : (float)((const __bf16*)a.logits)[at];
  }
  Key key[V];
  double s[kBiased ? V : 1];
  double total = 0.0;                  // of the exponentials, over all experts
  float top = -__builtin_inff();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (l[v] != l[v] || 64 * v + lane >= a.experts) l[v] = -__builtin_inff();
    if constexpr (PACKED) {            // before the cut: bf16's largest is not infinity
      const int e = 64 * v + lane;
      key[v] = e < a.experts ? (key_of(l[v]) & 0xffff0000u) | (unsigned)(0xffff - e) : 0;
    }
    l[v] = fminf(l[v], __FLT_MAX__);
    top = fmaxf(top, l[v]);
  }
  if (!a.sigmoid && (kBiased || !a.renormalize)) {
    const unsigned k = wave_max(key_of(top));
    top = __builtin_bit_cast(float, k >> 31 ? k & 0x7fffffffu : ~k);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const double x = top == -__builtin_inff() ? 0.0 : exp((double)l[v] - (double)top);
      if constexpr (kBiased) s[v] = x;
      total += x;
    }
    total = wave_sum(total);
  }
  if constexpr (kBiased) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 64 * v + lane;
      s[v] = a.sigmoid ? sigmoid((double)l[v]) : total > 0.0 ? s[v] / total : 0.0;
      double c = s[v] + (double)a.bias[min(e, a.experts - 1)];
      if (c != c) c = kNegInf;
      key[v] = e < a.experts ? key_of(c) : 0;
      if (a.groups > 1 && e < a.experts) members[wave][e + e / a.each] = c;
    }
  } else if constexpr (!PACKED) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = 64 * v + lane < a.experts ? key_of(l[v]) : 0;
  }
  if (a.groups > 1) {
    Key worth = 0;                     // of group `lane`
    if constexpr (kBiased) {
      in_order();
      if (lane < a.groups) {
        const double* c = members[wave] + lane * (a.each + 1);
        double first = kNegInf, second = kNegInf;
#pragma unroll 8
        for (int i = 0; i < a.each; ++i) {
          const double x = c[i];
          second = fmax(second, fmin(first, x));
          first = fmax(first, x);
        }
        double w = a.each > 1 ? first + second : first;
        if (w != w) w = kNegInf;
        worth = key_of(w);
      }
    } else {
      if (lane < a.groups) best_of[wave][lane] = 0;
      in_order();
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[v]) atomicMax(&best_of[wave][(64 * v + lane) / a.each], key[v]);
      in_order();
      if (lane < a.groups) worth = best_of[wave][lane];
    }
    u64 kept = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      const int g = __builtin_ctzll(lanes_of_max(worth));
      kept |= 1ull << g;
      if (lane == g) worth = 0;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!(kept >> ((64 * v + lane) / a.each & 63) & 1)) key[v] = 0;
  }
  // Lane j gets choice j: its number, and its logit or score.
  int id = 0;
  double mine = kBiased ? 0.0 : kNegInf;
  if constexpr (PACKED) {
    unsigned choice = 0;
    for (int j = 0; j < a.topk; ++j) {
      unsigned best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = max(best, key[v]);
      best = wave_max(best);
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = key[v] == best ? 0 : key[v];
      choice = lane == j ? best : choice;
    }
    id = 0xffff - (int)(choice & 0xffffu);
    const unsigned u = (choice >> 31 ? choice & 0x7fffffffu : ~choice) & 0xffff0000u;
    if (lane < a.topk) mine = (double)fminf(__builtin_bit_cast(float, u), __FLT_MAX__);
  } else {
    for (int j = 0; j < a.topk; ++j) {
      Key best = key[0];               // the lane's own largest, and the first place of it
      int at = 0;
#pragma unroll
      for (int v = 1; v < V; ++v) {
        const bool more = key[v] > best;
        best = more ? key[v] : best;
        at = more ? v : at;
      }
      u64 equal = lanes_of_max(best);
      int lane0 = __builtin_ctzll(equal), v0 = __builtin_amdgcn_readlane(at, lane0);
      while (equal &= equal - 1) {     // the first of equals
        const int other = __builtin_ctzll(equal), v1 = __builtin_amdgcn_readlane(at, other);
        if (v1 < v0) {
          v0 = v1;
          lane0 = other;
        }
      }
      double got = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (v0 == v) {
          if constexpr (kBiased) got = of_lane(s[v], lane0);
          else got = (double)of_lane(l[v], lane0);
        }
        key[v] = lane == lane0 && v0 == v ? 0 : key[v];
      }
      if (lane == j) {
        mine = got;
        id = 64 * v0 + lane0;
      }
    }
  }
  if constexpr (!kBiased) {
    if (a.sigmoid) {
      mine = lane < a.topk ? sigmoid(mine) : 0.0;
    } else {
      // Without a bias the first choice has the largest logit of all.
      const float first = __builtin_bit_cast(
          float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, (float)mine)));
      mine = lane >= a.topk || first == -__builtin_inff() ? 0.0 : exp(mine - (double)first);
      if (!a.renormalize) mine = total > 0.0 ? mine / total : 0.0;
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
  const dim3 grid((a.rows + kWaves - 1) / kWaves), threads(64 * kWaves);
  if (a.bias) hipLaunchKernelGGL((skinny_moe_route_k<V, u64, false>), grid, threads, 0, stream, a);
  else if (a.f32) hipLaunchKernelGGL((skinny_moe_route_k<V, unsigned, false>), grid, threads, 0, stream, a);
  else hipLaunchKernelGGL((skinny_moe_route_k<V, unsigned, true>), grid, threads, 0, stream, a);
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
  // The experts of a lane.  16384 rows of 96 experts in the instance for 256 take 10.4 us for
  // 8.7 (bf16), 13.7 for 11.2 (fp32) and 28.8 for 20.7 (biased), 192 experts 10.4 for 9.4,
  // 14.2 for 13.0 and 30.9 for 26.9.  Six and twelve per lane would take 12.2 for 14.1 (384,
  // bf16) and 18.0 for 21.5 (768), and have no instances.
  if (r.experts <= 64) return launch<1>(a, hs);
  if (r.experts <= 128) return launch<2>(a, hs);
  if (r.experts <= 192) return launch<3>(a, hs);
  if (r.experts <= 256) return launch<4>(a, hs);
  if (r.experts <= 512) return launch<8>(a, hs);
  return launch<16>(a, hs);
}

}  // extern "C"
