// verify_draft.hip - gfx950 kernels and C ABI of skinny_verify_draft: which of
// a step's drafted tokens the target model keeps, and the token that follows
// them, from the logits of the vocabulary projection and given random numbers.
//
// A verify step passes a handful of drafted tokens through the model at once
// ("9% faster GLM-5.3-Flash prefill with GPU-to-GPU IPC (and why TileLang
// didn't help)", section "TileLang: twice as fast, and no faster"); this is
// its end, beside the greedy token of skinny_lm_head_argmax, and like it stays
// on the device.
//
// The result is whole numbers, decided by comparisons of probabilities, so it
// must not depend on how a sum was rounded: a boundary of the cumulative
// distribution that moves by 2^-24 of the total gives another token once in a
// few hundred calls at 150 thousand entries.  Exponentials and sums are
// therefore fp64 throughout (one wave instruction of fp64 FMA costs what an fp32
// one does on this GPU), which puts the boundaries within about 2^-50.
//
// Two launches:
//   skinny_verify_stats   workgroup (slice, row, target or draft): the largest
//     logit of kSlice, the first place of it, and the sum of exp((l - max) / t);
//   skinny_verify_pick    workgroup (slice, sequence): from the rows' slices,
//     the normalisers and with them the first row that stops (each workgroup
//     the same, in the same order), then its slice's sum of the weights to
//     sample from, max(0, p - q).  The sequence's last workgroup to arrive
//     (a counter that the first launch cleared) finds the slice, then the
//     entry, where the running sum passes u times the total.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "host_util.h"
#include "skinny_gemm.h"

namespace {

using skinny_host::DeviceInfo;
using skinny_host::Range;
using skinny_host::aligned;
using skinny_host::device_info;
using skinny_host::overlap;
using skinny_host::range_of;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kSlice = 4096;                       // logits per workgroup
constexpr int kPer = kSlice / kThreads;            // per thread
constexpr int kRowLanes = 16;                      // lanes that read one row's slices
constexpr int kRowsAtOnce = kThreads / kRowLanes;
constexpr float kNegInf = -__builtin_inff();

struct Stat {
  double sum;            // sum over the slice of exp((l - max) / t)
  float max;             // -inf: no entry above -inf
  int first;             // lowest index of max
};

struct VerifyArgs {
  const int* q_start;
  const void* logits;    // [T][V]
  const void* draft;     // [T][V] or NULL
  const int* tokens;     // [T]
  const float* temperature;
  const float* accept_u; // [T]
  const float* sample_u; // [S]
  int* out_tokens;       // [T]
  int* accepted;         // [S]
  Stat* stats;           // [2][T][slices]
  double* weight;        // [S][slices]
  int* arrived;          // [S]
  int T, S, V, slices;
};

struct Rows {
  int q0, n;
};

__device__ __forceinline__ Rows rows_of(const VerifyArgs& a, int s) {
  Rows r;
  r.q0 = min(max(a.q_start[s], 0), a.T);
  r.n = min(max(a.q_start[s + 1], r.q0), a.T) - r.q0;
  return r;
}

__device__ __forceinline__ float temperature_of(const VerifyArgs& a, int s) {
  return a.temperature ? a.temperature[s] : 1.0f;
}

// exp(x) for x <= 0 in fp64: x = n ln 2 + r, |r| <= ln 2 / 2, and the Taylor
// series of exp(r) to r^12 (the next term is below 2^-52).  Below -700, and
// for NaN, 0.
__device__ __forceinline__ double exp_below(double x) {
  constexpr double kLog2e = 1.4426950408889634074, kLn2Hi = 0x1.62e42fefa39efp-1,
                   kLn2Lo = 0x1.abc9e3b39803fp-56;
  const double n = rint(x * kLog2e);
  const double r = fma(-n, kLn2Lo, fma(-n, kLn2Hi, x));
  double p = 1.0 / 479001600.0;
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  const double y = __builtin_ldexp(p, (int)fmax(n, -1100.0));
  return x >= -700.0 ? y : 0.0;
}

// exp((l - max) / t) with inv = 1 / t: 1 at the maximum (an infinite one too),
// 0 for NaN and -inf.
__device__ __forceinline__ double weight_of(float l, float top, double inv) {
  if (l == top) return top > kNegInf ? 1.0 : 0.0;
  return exp_below(((double)l - (double)top) * inv);
}

template <typename L>
__device__ __forceinline__ float logit(const void* p, size_t i) {
  return (float)static_cast<const L*>(p)[i];
}

// Logits at + 0 .. 7 (bf16) or 0 .. 3 (fp32) in one load.
template <typename L>
constexpr int kVec = 16 / (int)sizeof(L);
template <typename L>
__device__ __forceinline__ void load_vec(const void* p, size_t at, float* out) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const L*>(p) + at);
  if constexpr (sizeof(L) == 2) {
    const bf16x8 e = __builtin_bit_cast(bf16x8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = (float)e[i];
  } else {
    const f32x4 e = __builtin_bit_cast(f32x4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = e[i];
  }
}

// A thread's kPer logits of a slice that begins at n0, as runs of kVec
// neighbours (VEC) or single ones, NaN past the end; index of the j-th.
template <typename L, bool VEC>
__device__ __forceinline__ int index_of(int j) {
  constexpr int W = VEC ? kVec<L> : 1;
  return (j / W * kThreads + (int)threadIdx.x) * W + j % W;
}
template <typename L, bool VEC>
__device__ __forceinline__ void load_slice(const void* row, int n0, int V, float (&l)[kPer]) {
  if constexpr (VEC) {
    constexpr int W = kVec<L>;
#pragma unroll
    for (int j = 0; j < kPer; j += W) {
      const int n = n0 + index_of<L, true>(j);
      load_vec<L>(row, min(n, V - W), l + j);
      if (n >= V) {
#pragma unroll
        for (int e = 0; e < W; ++e) l[j + e] = __builtin_nanf("");
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int n = n0 + index_of<L, false>(j);
      l[j] = n < V ? logit<L>(row, n) : __builtin_nanf("");
    }
  }
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
  return x;
}

__device__ __forceinline__ void take_first(float v, int i, float& bv, int& bi) {
  if (v > bv || (v == bv && i < bi)) {
    bv = v;
    bi = i;
  }
}

// Sequence of row t, or -1.
__device__ __forceinline__ int find_row(const VerifyArgs& a, int t) {
  const int lane = threadIdx.x & 63;
  for (int s0 = 0; s0 < a.S; s0 += 64) {
    const int s = s0 + lane;
    const bool hit = s < a.S && a.q_start[s] <= t && t < a.q_start[s + 1];
    const unsigned long long b = __ballot(hit);
    if (b) return s0 + __builtin_ctzll(b);
  }
  return -1;
}

template <typename L, bool VEC>
__global__ __launch_bounds__(kThreads) void skinny_verify_stats(const VerifyArgs a) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slice = blockIdx.x, row = blockIdx.y, which = blockIdx.z;
  if (slice == 0 && row == 0 && which == 0)
    for (int i = tid; i < a.S; i += kThreads) a.arrived[i] = 0;
  const int s = find_row(a, row);
  if (s < 0) return;
  const Rows r = rows_of(a, s);
  const float t = temperature_of(a, s);
  const bool greedy = !(t > 0.0f);
  // The draft's last row drafted nothing, and a greedy sequence asks only the target.
  if (which == 1 && (greedy || row + 1 == r.q0 + r.n)) return;
  const void* src = static_cast<const L*>(which ? a.draft : a.logits) + (size_t)row * a.V;
  const int n0 = slice * kSlice;
  float l[kPer];
  load_slice<L, VEC>(src, n0, a.V, l);
  float top = kNegInf;
  int first = a.V;
#pragma unroll
  for (int j = 0; j < kPer; ++j) take_first(l[j], n0 + index_of<L, VEC>(j), top, first);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const float ov = __shfl_xor(top, off);
    const int oi = __shfl_xor(first, off);
    take_first(ov, oi, top, first);
  }
  __shared__ float sv[kThreads / 64];
  __shared__ int si[kThreads / 64];
  __shared__ double ss[kThreads / 64];
  if (lane == 0) {
    sv[wave] = top;
    si[wave] = first;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) take_first(sv[w], si[w], top, first);
  double sum = 0.0;
  if (!greedy) {
    const double inv = 1.0 / (double)t;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum += weight_of(l[j], top, inv);
    sum = wave_sum(sum);
    if (lane == 0) ss[wave] = sum;
    __syncthreads();
    sum = (ss[0] + ss[1]) + (ss[2] + ss[3]);
  }
  if (tid == 0)
    a.stats[((size_t)which * a.T + row) * a.slices + slice] = Stat{sum, top, first};
}

// A row's maximum, where it first is, and the sum of weights, from its slices:
// the same in all kRowLanes lanes.
struct RowStat {
  float top;
  int first;
  double sum;
};
__device__ __forceinline__ RowStat row_stat(const Stat* st, int slices, double inv) {
  const int l = threadIdx.x & (kRowLanes - 1);
  RowStat r{kNegInf, 0x7fffffff, 0.0};
  for (int i = l; i < slices; i += kRowLanes) take_first(st[i].max, st[i].first, r.top, r.first);
#pragma unroll
  for (int off = kRowLanes / 2; off > 0; off >>= 1) {
    const float ov = __shfl_xor(r.top, off);
    const int oi = __shfl_xor(r.first, off);
    take_first(ov, oi, r.top, r.first);
  }
  if (inv > 0.0) {
    for (int i = l; i < slices; i += kRowLanes) r.sum += st[i].sum * weight_of(st[i].max, r.top, inv);
#pragma unroll
    for (int off = kRowLanes / 2; off > 0; off >>= 1) r.sum += __shfl_xor(r.sum, off);
  }
  return r;
}

// Of the row that stops a sequence: what its weights are made of.
struct Stop {
  int row;               // within the sequence
  int greedy_token;
  float p_top, q_top;
  double p_inv, q_inv;   // 1 / sum (0: nothing)
  int drafted;           // without a draft distribution: the rejected token, else -1
};

// max(0, p - q) of one entry; `plain`: p itself.  Both products are rounded
// before the difference (no fused multiply-add), so equal rows leave exactly 0.
template <typename L>
__device__ __forceinline__ double residual(const Stop& st, double inv, float lp, float lq, int n,
                                           bool plain) {
#pragma clang fp contract(off)
  const double p = weight_of(lp, st.p_top, inv) * st.p_inv;
  if (plain) return p;
  if (n == st.drafted) return 0.0;
  return fmax(p - weight_of(lq, st.q_top, inv) * st.q_inv, 0.0);
}

template <typename L, bool VEC>
__global__ __launch_bounds__(kThreads) void skinny_verify_pick(const VerifyArgs a) {
  __shared__ Stop stop;
  __shared__ int first_stop;
  __shared__ int is_last;
  __shared__ double swave[kThreads / 64];
  __shared__ int found;
  __shared__ int last_positive;
  __shared__ double goal_s, before_s;
  __shared__ int slice_s, plain_s;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slice = blockIdx.x, s = blockIdx.y;
  const Rows r = rows_of(a, s);
  if (r.n == 0) {
    if (slice == 0 && tid == 0) a.accepted[s] = 0;
    return;
  }
  const float t = temperature_of(a, s);
  const bool greedy = !(t > 0.0f);
  if (greedy && slice != 0) return;
  const double inv = greedy ? 0.0 : 1.0 / (double)t;

  // The first row that stops: a rejection, or the last row.  kRowLanes lanes per row.
  for (int i0 = 0;; i0 += kRowsAtOnce) {
    if (tid == 0) first_stop = r.n;
    __syncthreads();
    const int i = i0 + tid / kRowLanes;
    Stop mine{};
    bool stops = false;
    if (i < r.n) {
      const int row = r.q0 + i;
      const bool final = i == r.n - 1;
      const RowStat p = row_stat(a.stats + (size_t)row * a.slices, a.slices, inv);
      const int d = final ? -1 : a.tokens[row + 1];
      const bool in = d >= 0 && d < a.V;
      mine.row = i;
      mine.greedy_token = p.top > kNegInf ? p.first : 0;
      mine.p_top = p.top;
      mine.p_inv = p.sum > 0.0 ? 1.0 / p.sum : 0.0;
      mine.drafted = -1;
      const double u = a.accept_u[row];
      if (greedy) {
        stops = !(in && p.top > kNegInf && d == p.first && u < 1.0);
      } else {
        double q = 1.0;
        if (!final && a.draft) {
          const RowStat qs = row_stat(a.stats + ((size_t)a.T + row) * a.slices, a.slices, inv);
          mine.q_top = qs.top;
          mine.q_inv = qs.sum > 0.0 ? 1.0 / qs.sum : 0.0;
          if (in) q = weight_of(logit<L>(a.draft, (size_t)row * a.V + d), qs.top, inv) * mine.q_inv;
        } else if (!final) {
          mine.drafted = d;
        }
        const double pd =
            in ? weight_of(logit<L>(a.logits, (size_t)row * a.V + d), p.top, inv) * mine.p_inv : 0.0;
        stops = final || !(u * q < pd);
      }
    }
    if (stops && tid % kRowLanes == 0) atomicMin(&first_stop, i);
    __syncthreads();
    const int at = first_stop;
    if (at < r.n) {
      if (i == at && tid % kRowLanes == 0) stop = mine;
      __syncthreads();
      break;
    }
    __syncthreads();
  }
  const Stop st = stop;
  const int row = r.q0 + st.row;
  const bool final = st.row == r.n - 1;

  int token = 0;
  if (greedy) {
    token = st.greedy_token;
  } else {
    // This slice's share of the weights.
    const void* lp_row = static_cast<const L*>(a.logits) + (size_t)row * a.V;
    const bool with_q = a.draft && !final;
    const void* lq_row = with_q ? static_cast<const L*>(a.draft) + (size_t)row * a.V : lp_row;
    float lp[kPer], lq[kPer];
    const int n0 = slice * kSlice;
    load_slice<L, VEC>(lp_row, n0, a.V, lp);
    if (with_q) load_slice<L, VEC>(lq_row, n0, a.V, lq);
    double w = 0.0;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      w += residual<L>(st, inv, lp[j], with_q ? lq[j] : kNegInf, n0 + index_of<L, VEC>(j), final);
    w = wave_sum(w);
    if (lane == 0) swave[wave] = w;
    __syncthreads();
    if (tid == 0) {
      a.weight[(size_t)s * a.slices + slice] = (swave[0] + swave[1]) + (swave[2] + swave[3]);
      __threadfence();
      is_last = __hip_atomic_fetch_add(&a.arrived[s], 1, __ATOMIC_ACQ_REL,
                                       __HIP_MEMORY_SCOPE_AGENT) == a.slices - 1;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();

    // The slice where the running sum passes u times the total; without any
    // weight (p nowhere above q), the same over p itself.
    if (wave == 0) {
      const double* ws = a.weight + (size_t)s * a.slices;
      const Stat* ps = a.stats + (size_t)row * a.slices;
      double total = 0.0;
      for (int i = lane; i < a.slices; i += 64) total += ws[i];
      total = wave_sum(total);
      const bool plain = !(total > 0.0);
      if (plain) {
        total = 0.0;
        for (int i = lane; i < a.slices; i += 64)
          total += ps[i].sum * weight_of(ps[i].max, st.p_top, inv) * st.p_inv;
        total = wave_sum(total);
      }
      const double u = a.sample_u[s];
      const double goal = (u > 0.0 ? u : 0.0) * total;
      double before = 0.0;
      int at = -1, last = 0;
      double at_before = 0.0, last_before = 0.0;
      for (int i0 = 0; i0 < a.slices && at < 0; i0 += 64) {
        const int i = i0 + lane;
        double x = 0.0;
        if (i < a.slices)
          x = plain ? ps[i].sum * weight_of(ps[i].max, st.p_top, inv) * st.p_inv : ws[i];
        double incl = x;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const double o = __shfl_up(incl, off);
          if (lane >= off) incl += o;
        }
        const unsigned long long over = __ballot(x > 0.0 && before + incl > goal);
        const unsigned long long some = __ballot(x > 0.0);
        if (some) {
          const int b = 63 - __builtin_clzll(some);
          last = i0 + b;
          last_before = before + __shfl(incl, b) - __shfl(x, b);
        }
        if (over) {
          const int b = __builtin_ctzll(over);
          at = i0 + b;
          const double prev = __shfl(incl, b ? b - 1 : 0);
          at_before = b ? before + prev : before;
        }
        before += __shfl(incl, 63);
      }
      if (lane == 0) {
        slice_s = at < 0 ? last : at;
        before_s = at < 0 ? last_before : at_before;
        goal_s = goal;
        plain_s = plain || final;
        found = a.V;
        last_positive = 0;
      }
    }
    __syncthreads();
    // The entry in it: kPer neighbours per thread, in order.
    const int m0 = slice_s * kSlice + tid * kPer;
    const bool plain = plain_s;
    double x[kPer];
    double sum = 0.0;
    int positive = -1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int n = m0 + j;
      const float vp = n < a.V ? logit<L>(lp_row, n) : __builtin_nanf("");
      const float vq = with_q && n < a.V ? logit<L>(lq_row, n) : kNegInf;
      const double y = residual<L>(st, inv, vp, vq, n, plain);
      if (y > 0.0) positive = n;
      sum += y;
      x[j] = sum;
    }
    double incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double o = __shfl_up(incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 63) swave[wave] = incl;
    __syncthreads();
    double base = before_s;
    for (int w2 = 0; w2 < wave; ++w2) base += swave[w2];
    base += incl - sum;
    int hit = a.V;
#pragma unroll
    for (int j = kPer - 1; j >= 0; --j)
      if (base + x[j] > goal_s && x[j] > (j ? x[j - 1] : 0.0)) hit = m0 + j;
    if (hit < a.V) atomicMin(&found, hit);
    if (positive >= 0) atomicMax(&last_positive, positive);
    __syncthreads();
    token = found < a.V ? found : last_positive;
  }

  for (int i = tid; i < r.n; i += kThreads)
    a.out_tokens[r.q0 + i] = i < st.row ? a.tokens[r.q0 + i + 1] : i == st.row ? token : -1;
  if (tid == 0) a.accepted[s] = st.row;
}

// ---------------------------------------------------------------------------
// Host side.

int slices_of(int vocab) { return (vocab + kSlice - 1) / kSlice; }

size_t up(size_t b) { return (b + 255) / 256 * 256; }

struct Layout {
  size_t stats, weight, arrived, total;
};

Layout layout(int rows, int seqs, int vocab) {
  const size_t sl = slices_of(vocab);
  Layout w;
  w.stats = 0;
  w.weight = up((size_t)2 * rows * sl * sizeof(Stat));
  w.arrived = w.weight + up((size_t)seqs * sl * sizeof(double));
  w.total = w.arrived + up((size_t)seqs * sizeof(int));
  return w;
}

skinny_status check_sizes(int rows, int seqs, int vocab) {
  if (rows < 1 || seqs < 1 || vocab < 1) return SKINNY_ERR_INVALID_ARG;
  if (rows > SKINNY_VERIFY_MAX_ROWS || seqs > SKINNY_VERIFY_MAX_ROWS ||
      vocab > SKINNY_VERIFY_MAX_VOCAB)
    return SKINNY_ERR_UNSUPPORTED;
  return SKINNY_OK;
}

template <typename L, bool VEC>
skinny_status launch(const VerifyArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((skinny_verify_stats<L, VEC>), dim3(a.slices, a.T, a.draft ? 2 : 1),
                     dim3(kThreads), 0, stream, a);
  if (hipGetLastError() != hipSuccess) return SKINNY_ERR_HIP;
  hipLaunchKernelGGL((skinny_verify_pick<L, VEC>), dim3(a.slices, a.S), dim3(kThreads), 0, stream,
                     a);
  return hipGetLastError() == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP;
}

template <typename L>
skinny_status launch_as(const VerifyArgs& a, hipStream_t stream) {
  if (a.V % kVec<L> == 0 && aligned(a.logits, 16) && (!a.draft || aligned(a.draft, 16)))
    return launch<L, true>(a, stream);
  return launch<L, false>(a, stream);
}

}  // namespace

extern "C" {

size_t skinny_verify_workspace_bytes(int rows, int seqs, int vocab) {
  if (check_sizes(rows, seqs, vocab) != SKINNY_OK) return 0;
  return layout(rows, seqs, vocab).total;
}

skinny_status skinny_verify_draft(const skinny_verify* verify, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!verify) return SKINNY_ERR_INVALID_ARG;
  const skinny_verify& v = *verify;
  if (v.dtype != SKINNY_LOGITS_BF16 && v.dtype != SKINNY_LOGITS_F32) return SKINNY_ERR_INVALID_ARG;
  skinny_status st = check_sizes(v.rows, v.seqs, v.vocab);
  if (st != SKINNY_OK) return st;
  if (!v.q_start || !v.logits || !v.tokens || !v.accept_u || !v.sample_u || !v.out_tokens ||
      !v.accepted)
    return SKINNY_ERR_INVALID_ARG;
  const size_t e = v.dtype == SKINNY_LOGITS_BF16 ? 2 : 4;
  if (!aligned(v.logits, e) || !aligned(v.draft_logits, e)) return SKINNY_ERR_UNSUPPORTED;
  const void* four[] = {v.q_start,  v.tokens,     v.temperature, v.accept_u,
                        v.sample_u, v.out_tokens, v.accepted};
  for (const void* p : four)
    if (!aligned(p, 4)) return SKINNY_ERR_UNSUPPORTED;
  const Layout w = layout(v.rows, v.seqs, v.vocab);
  if (!workspace || workspace_bytes < w.total) return SKINNY_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SKINNY_ERR_UNSUPPORTED;
  const size_t lb = (size_t)v.rows * v.vocab * e;
  const Range written[] = {range_of(v.out_tokens, (size_t)v.rows * 4),
                           range_of(v.accepted, (size_t)v.seqs * 4),
                           range_of(workspace, workspace_bytes)};
  const Range read[] = {range_of(v.q_start, (size_t)(v.seqs + 1) * 4),
                        range_of(v.logits, lb),
                        range_of(v.draft_logits, v.draft_logits ? lb : 0),
                        range_of(v.tokens, (size_t)v.rows * 4),
                        range_of(v.temperature, v.temperature ? (size_t)v.seqs * 4 : 0),
                        range_of(v.accept_u, (size_t)v.rows * 4),
                        range_of(v.sample_u, (size_t)v.seqs * 4)};
  for (int i = 0; i < 3; ++i) {
    for (int j = i + 1; j < 3; ++j)
      if (overlap(written[i], written[j])) return SKINNY_ERR_INVALID_ARG;
    for (const Range& x : read)
      if (x.lo != x.hi && overlap(written[i], x)) return SKINNY_ERR_INVALID_ARG;
  }
  DeviceInfo d;
  st = device_info(&d);
  if (st != SKINNY_OK) return st;
  if (!d.gfx950) return SKINNY_ERR_UNSUPPORTED;

  VerifyArgs a;
  a.q_start = v.q_start;
  a.logits = v.logits;
  a.draft = v.draft_logits;
  a.tokens = v.tokens;
  a.temperature = v.temperature;
  a.accept_u = v.accept_u;
  a.sample_u = v.sample_u;
  a.out_tokens = v.out_tokens;
  a.accepted = v.accepted;
  unsigned char* ws = (unsigned char*)workspace;
  a.stats = (Stat*)(ws + w.stats);
  a.weight = (double*)(ws + w.weight);
  a.arrived = (int*)(ws + w.arrived);
  a.T = v.rows;
  a.S = v.seqs;
  a.V = v.vocab;
  a.slices = slices_of(v.vocab);
  return v.dtype == SKINNY_LOGITS_BF16 ? launch_as<__bf16>(a, (hipStream_t)stream)
                                       : launch_as<float>(a, (hipStream_t)stream);
}

}  // extern "C"
