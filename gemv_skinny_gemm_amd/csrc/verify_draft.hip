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
// one does on this GPU).  2^y is within 2^-47 of itself by its series and |y| 2^-52
// by y's own rounding; entries far below the largest add little to a sum, so
// boundaries are within about 2^-46 of the total (1.4e-14).
//
// Two launches:
//   skinny_verify_stats   workgroup (slice, row, target or draft): the largest
//     logit of a slice, the first place of it, and the sum of exp((l - max) / t);
//   skinny_verify_pick    workgroup (slice, sequence): from the rows' slices,
//     the normalisers and with them the first row that stops (each workgroup
//     the same, in the same order), then its waves' sums of the weights to
//     sample from, max(0, p - q), over a quarter slice each.  The sequence's last
//     workgroup to arrive (a counter that the first launch cleared) finds the
//     quarter, then the entry, where the running sum passes u times the
//     total; sums are added in index order, so it does not matter who came last.
// The sums pass between workgroups as relaxed device-scope words that the first
// launch set to a mark: a word read before it arrived is read again, up to a limit
// of polls, behind which the sequence gets -1 in the place of its results.  Fences in
// their place cost about 8 us a call here (they write back and invalidate an
// XCD's whole L2).
//
// What bounds it, measured on 37 rows of 152064 bf16 logits with as many of the
// draft's: 26.0 us (15.0 + 11.4), where reading them would take 3.  The first launch
// issues 30 vector instructions per logit (11 FMA of the exponential, the rest around
// them), 18.4 thousand cycles per SIMD or 7.7 us at 2.4 GHz, and without the
// exponentials takes 9.4: what is not issue is the launch and the chains of some
// eleven workgroups per CU (row's sequence - logits - maximum - sum - join).  The
// second one is the latency of its chain.  A few rows are the two launches' latency:
// 11.0 us for 2 rows of 32003, 14.2 for
// 6 of 152064.  Slices are 4096 entries, or 2048 where that makes at most 64 of a
// row (what one trip of the second launch reads) and 1024 of all rows: 32003
// entries 11.8 against 13.2 us at 4 rows, 13.5 against 14.2 at 32; beyond the
// one bound (152064) 15.3 against 13.9 at 4 rows, beyond the other (64 rows of
// 64000) 23.5 against 21.1.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "host_util.h"
#include "skinny_gemm.h"

namespace {

using skinny_host::DeviceInfo;
using skinny_host::Range;
using skinny_host::aligned;
using skinny_host::device_info;
using skinny_host::overlap;
using skinny_host::range_of;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
// Logits of a slice, one workgroup's: PER per lane.
template <int PER>
constexpr int kSlice = kThreads * PER;
template <int PER>
constexpr int kSub = 64 * PER;                     // per wave
constexpr int kPerLong = 16, kPerShort = 8;
constexpr int kRowLanes = 16;                      // lanes that read one row's slices
constexpr int kRowsAtOnce = kThreads / kRowLanes;
constexpr int kBatch = 4;                          // exponentials at a time
constexpr float kNegInf = -__builtin_inff();
constexpr unsigned long long kNotYet = ~0ull;      // a NaN that no sum is
std::atomic<long long> g_polls{1 << 16};

struct Stat {
  double sum;            // sum over the slice of exp((l - max) / t)
  float max;             // -inf: no entry above -inf
  int first;             // lowest index of max (a greedy sequence's rows)
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
  unsigned long long* weight;   // [S][slices][kWaves] fp64
  float* drafted;        // [2][T] logit of the token drafted at each row (NaN: none)
  int* arrived;          // [S]
  int T, S, V, slices;
  long long polls;       // of a word that has not arrived, before giving up; < 0: at once
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

// 2^y for -1000 <= y <= 0 in fp64: y = n + f, |f| <= 1/2, n from the low bits of
// y + 1.5 * 2^52, and the Taylor series of exp(f ln 2) to the 11th power (the
// next term is below 2^-47 of it); n is added to the exponent's bits.  Below
// that, and for NaN, 0, or without EXACT 2^-1000, which adds nothing to a sum
// that has a 1 in it.
struct Taylor {
  double c[12];
  constexpr Taylor() : c{} {
    c[0] = 1.0;
    for (int k = 1; k < 12; ++k) c[k] = c[k - 1] * 0.69314718055994530942 / k;
  }
};
// N at a time, step by step: a chain of dependent fp64 instructions alone leaves
// the ALUs waiting.
template <bool EXACT, int N>
__device__ __forceinline__ void exp2_below(double (&y)[N]) {
  constexpr Taylor t;
  double last = t.c[11];
  asm("" : "+v"(last));                            // a register, not two moves at each use
  constexpr double kShift = 6755399441055744.0;    // 1.5 * 2^52
  double s[N], f[N], p[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (!EXACT) y[i] = __builtin_fmax(y[i], -1000.0);
    s[i] = y[i] + kShift;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f[i] = y[i] - (s[i] - kShift);
    p[i] = last;
  }
#pragma unroll
  for (int k = 10; k >= 0; --k)
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = fma(p[i], f[i], t.c[k]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const u32x2 n = __builtin_bit_cast(u32x2, s[i]);
    u32x2 r = __builtin_bit_cast(u32x2, p[i]);
    r[1] += n[0] << 20;
    const double x = __builtin_bit_cast(double, r);
    y[i] = !EXACT || y[i] >= -1000.0 ? x : 0.0;
  }
}

// exp((l - top) / t) with c = log2 e / t, top below +inf: 1 at the maximum, 0
// for NaN and -inf (and for top -inf).
template <bool EXACT, int N>
__device__ __forceinline__ void finite_weights(const float* l, double top, double c,
                                               double (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = ((double)l[i] - top) * c;
  exp2_below<EXACT>(w);
}
// The same for any top; where it is +inf, 1 at the infinite entries and 0 elsewhere.
template <int N>
__device__ __forceinline__ void weights_of(const float* l, float top, double c, double (&w)[N]) {
  finite_weights<true>(l, (double)top, c, w);
  if (top == -kNegInf) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = l[i] == top ? 1.0 : 0.0;
  }
}
__device__ __forceinline__ double weight_of(float l, float top, double c) {
  double w[1];
  weights_of(&l, top, c, w);
  return w[0];
}

// Lane exchanges on the vector ALUs: rotation within 16 lanes, and with the
// lanes 16 and 32 away.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, true);
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, dpp<CTRL, ROWS>(__builtin_bit_cast(int, x)));
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double dpp(double x) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
  const unsigned lo = (unsigned)dpp<CTRL, ROWS>((int)(unsigned)u);
  const unsigned hi = (unsigned)dpp<CTRL, ROWS>((int)(unsigned)(u >> 32));
  return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
constexpr int kRor = 0x120, kShr = 0x110, kBcast15 = 0x142, kBcast31 = 0x143;

template <typename T, typename F>
__device__ __forceinline__ T reduce16(T x, F f) {
  x = f(x, dpp<kRor + 1>(x));
  x = f(x, dpp<kRor + 2>(x));
  x = f(x, dpp<kRor + 4>(x));
  return f(x, dpp<kRor + 8>(x));
}
struct Halves {
  unsigned a, b;
};
__device__ __forceinline__ Halves across16(unsigned u) {
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned a = s[0], b = s[1];
  return Halves{a, b};
}
__device__ __forceinline__ Halves across32(unsigned u) {
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned a = s[0], b = s[1];
  return Halves{a, b};
}
// f of a value and that of the lane 16 (32) away, in the same order for both.
#define SKINNY_JOIN(across)                                                           \
  if constexpr (sizeof(T) == 4) {                                                      \
    const Halves h = across(__builtin_bit_cast(unsigned, x));                          \
    return f(__builtin_bit_cast(T, h.a), __builtin_bit_cast(T, h.b));                  \
  } else {                                                                             \
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);            \
    const Halves lo = across((unsigned)u), hi = across((unsigned)(u >> 32));           \
    const unsigned long long a = (unsigned long long)hi.a << 32 | lo.a;                \
    const unsigned long long b = (unsigned long long)hi.b << 32 | lo.b;                \
    return f(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));                      \
  }
template <typename T, typename F>
__device__ __forceinline__ T join16(T x, F f) {
  SKINNY_JOIN(across16)
}
template <typename T, typename F>
__device__ __forceinline__ T join32(T x, F f) {
  SKINNY_JOIN(across32)
}
#undef SKINNY_JOIN
template <typename T, typename F>
__device__ __forceinline__ T reduce64(T x, F f) {
  return join32(join16(reduce16(x, f), f), f);
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ int lower(int a, int b) { return min(a, b); }
__device__ __forceinline__ double plus(double a, double b) { return a + b; }

// Sum over the lanes up to and with this one.
__device__ __forceinline__ double scan64(double x) {
  x += dpp<kShr + 1>(x);
  x += dpp<kShr + 2>(x);
  x += dpp<kShr + 4>(x);
  x += dpp<kShr + 8>(x);
  x += dpp<kBcast15, 0xa>(x);
  return x + dpp<kBcast31, 0xc>(x);
}
__device__ __forceinline__ double lane_of(double x, int lane) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
  const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)u, lane);
  const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(u >> 32), lane);
  return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
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

// A lane's PER of the wave's logits from n0 on, as runs of kVec neighbours (VEC)
// or single ones, NaN past the end; place of the j-th.
template <typename L, bool VEC>
__device__ __forceinline__ int index_of(int j) {
  constexpr int W = VEC ? kVec<L> : 1;
  return (j / W * 64 + (int)(threadIdx.x & 63)) * W + j % W;
}
template <typename L, bool VEC, int PER>
__device__ __forceinline__ void load_sub(const void* row, int n0, int V, float (&l)[PER]) {
  if constexpr (VEC) {
    constexpr int W = kVec<L>;
#pragma unroll
    for (int j = 0; j < PER; j += W) {
      const int n = n0 + index_of<L, true>(j);
      load_vec<L>(row, min(n, V - W), l + j);
      if (n >= V) {
#pragma unroll
        for (int e = 0; e < W; ++e) l[j + e] = __builtin_nanf("");
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int n = n0 + index_of<L, false>(j);
      const float x = logit<L>(row, min(n, V - 1));
      l[j] = n < V ? x : __builtin_nanf("");
    }
  }
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

template <typename L, bool VEC, int PER>
__global__ __launch_bounds__(kThreads) void skinny_verify_stats(const VerifyArgs a) {
  __shared__ float sv[kWaves];
  __shared__ int si[kWaves];
  __shared__ double ss[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slice = blockIdx.x, row = blockIdx.y, which = blockIdx.z;
  const void* src = static_cast<const L*>(which ? a.draft : a.logits) + (size_t)row * a.V;
  const int n0 = slice * kSlice<PER> + wave * kSub<PER>;
  float l[PER];
  const auto load = [&] {
    load_sub<L, VEC, PER>(src, n0, a.V, l);
    if (slice == 0 && tid == 0) {
      const int d = row + 1 < a.T ? a.tokens[row + 1] : -1;
      a.drafted[(size_t)which * a.T + row] =
          d >= 0 && d < a.V ? logit<L>(src, d) : __builtin_nanf("");
    }
  };
  // The target's are on their way while the row's sequence is found.  The draft's
  // wait until it is known that they are asked: those of other rows need not be there.
  if (which == 0) load();
  if (row == 0 && which == 0) {
    for (int i = tid; i < a.S * kWaves; i += kThreads)
      a.weight[((size_t)(i / kWaves) * a.slices + slice) * kWaves + i % kWaves] = kNotYet;
    if (slice == 0)
      for (int i = tid; i < a.S; i += kThreads) a.arrived[i] = 0;
  }
  const int s = find_row(a, row);
  if (s < 0) return;
  const Rows r = rows_of(a, s);
  const float t = temperature_of(a, s);
  const bool greedy = !(t > 0.0f);
  // The draft's last row drafted nothing, and a greedy sequence asks only the target.
  if (which == 1) {
    if (greedy || row + 1 == r.q0 + r.n) return;
    load();
  }
  // Each wave's maximum and sum, then the four joined.
  float top = kNegInf;
#pragma unroll
  for (int j = 0; j < PER; ++j) top = fmaxf(top, l[j]);
  const float wtop = reduce64(top, larger);
  int first = a.V;
  double sum = 0.0;
  const double c = 1.4426950408889634074 / (double)t;
  if (greedy) {
#pragma unroll
    for (int j = PER - 1; j >= 0; --j) first = l[j] == wtop ? n0 + index_of<L, VEC>(j) : first;
    first = reduce64(first, lower);
  } else {
    if (wtop < -kNegInf) {
      const double dtop = wtop;
#pragma unroll
      for (int j = 0; j < PER; j += kBatch) {
        double w[kBatch];
        finite_weights<false>(l + j, dtop, c, w);
#pragma unroll
        for (int e = 0; e < kBatch; ++e) sum += w[e];
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) sum += l[j] == wtop ? 1.0 : 0.0;
    }
    sum = reduce64(sum, plus);
  }
  if (lane == 0) {
    sv[wave] = wtop;
    si[wave] = first;
    ss[wave] = sum;
  }
  __syncthreads();
  if (wave != 0) return;
  const int w = lane & (kWaves - 1);
  top = sv[w];
  first = si[w];
  float all = top;
  int at = first;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) take_first(sv[k], si[k], all, at);
  sum = greedy ? 0.0 : ss[w] * weight_of(top, all, c);
  sum += dpp<kRor + 1>(sum);
  sum += dpp<kRor + 2>(sum);
  if (lane == 0) a.stats[((size_t)which * a.T + row) * a.slices + slice] = Stat{sum, all, at};
}

// A row's maximum, where it first is, and the sum of weights, from its slices:
// kRowLanes lanes take every kRowLanes-th, kAhead at a time, and end with the same.
struct RowStat {
  float top;
  int first;
  double sum;
};
constexpr int kAhead = 4;
__device__ __forceinline__ void load_stats(const Stat* st, int i0, int slices, Stat (&x)[kAhead]) {
#pragma unroll
  for (int e = 0; e < kAhead; ++e) {
    const int i = i0 + e * kRowLanes;
    x[e] = st[min(i, slices - 1)];
    if (i >= slices) x[e] = Stat{0.0, kNegInf, 0x7fffffff};
  }
}
__device__ __forceinline__ void add_stats(const Stat (&x)[kAhead], double c, RowStat& r) {
  const float had = r.top;
#pragma unroll
  for (int e = 0; e < kAhead; ++e) take_first(x[e].max, x[e].first, r.top, r.first);
  float top[kAhead + 1];
  double w[kAhead + 1];
#pragma unroll
  for (int e = 0; e < kAhead; ++e) top[e] = x[e].max;
  top[kAhead] = had;
  weights_of(top, r.top, c, w);
  r.sum *= w[kAhead];
#pragma unroll
  for (int e = 0; e < kAhead; ++e) r.sum += x[e].sum * w[e];
}
__device__ __forceinline__ void row_end(double c, RowStat& r) {
  const float had = r.top;
  r.top = reduce16(r.top, larger);
  r.first = reduce16(had == r.top ? r.first : 0x7fffffff, lower);
  r.sum = reduce16(r.sum * weight_of(had, r.top, c), plus);
}

// Of the row that stops a sequence: what its weights are made of.
struct Stop {
  int row;               // within the sequence
  int greedy_token;
  float p_top, q_top;
  double p_inv, q_inv;   // 1 / sum (0: nothing)
  int drafted;           // without a draft distribution: the rejected token, else -1
};

// max(0, p - q) of N entries from logits lp and lq (without with_q, q is 1 at the
// rejected token, or nothing); n: their places; `plain`: p itself.  Both products
// are rounded before the difference (no fused multiply-add), so equal rows leave
// exactly 0.
template <int N>
__device__ __forceinline__ void residuals(const Stop& st, double c, const float* lp,
                                          const float* lq, bool with_q, const int (&n)[N],
                                          bool plain, double (&w)[N]) {
#pragma clang fp contract(off)
  weights_of(lp, st.p_top, c, w);
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] *= st.p_inv;
  if (plain) return;
  if (with_q) {
    double q[N];
    weights_of(lq, st.q_top, c, q);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = fmax(w[i] - q[i] * st.q_inv, 0.0);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = n[i] == st.drafted ? 0.0 : w[i];
  }
}

template <typename L, bool VEC, int PER>
__global__ __launch_bounds__(kThreads) void skinny_verify_pick(const VerifyArgs a) {
  constexpr int kFind = kSub<PER> / kThreads;        // entries of a thread in the last search
  __shared__ Stop stops[kWaves];
  __shared__ int is_last, found, positive;
  __shared__ double wsum[kWaves];
  __shared__ double goal_s, before_s;
  __shared__ int sub_s, plain_s, gave_up;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slice = blockIdx.x, s = blockIdx.y;
  const Rows r = rows_of(a, s);
  const float t = temperature_of(a, s);
  const double u = a.sample_u[s];
  if (r.n == 0) {
    if (slice == 0 && tid == 0) a.accepted[s] = 0;
    return;
  }
  const bool greedy = !(t > 0.0f);
  if (greedy && slice != 0) return;
  // What a row gives out if its draft is kept; on its way while it is decided.
  const int kept = tid + 1 < r.n ? a.tokens[r.q0 + tid + 1] : -1;
  const double c = greedy ? 0.0 : 1.4426950408889634074 / (double)t;

  // The first row that stops: a rejection, or the last row.  kRowLanes lanes per row.
  Stop st{};
  for (int i0 = 0;; i0 += kRowsAtOnce) {
    const int i = i0 + tid / kRowLanes, l = tid & (kRowLanes - 1);
    Stop mine{};
    bool stop = false;
    if (i < r.n) {
      const int row = r.q0 + i;
      const bool final = i == r.n - 1;
      const bool asks = !final && !greedy && a.draft;
      const int d = final ? -1 : a.tokens[row + 1];
      const double au = a.accept_u[row];
      const bool in = d >= 0 && d < a.V;
      RowStat p{kNegInf, 0x7fffffff, 0.0}, q{kNegInf, 0x7fffffff, 0.0};
      const Stat* ps = a.stats + (size_t)row * a.slices;
      const Stat* qs = a.stats + ((size_t)(asks ? a.T : 0) + row) * a.slices;
      const float pl = a.drafted[row], ql = a.drafted[(asks ? a.T : 0) + row];
      for (int k = l; k - l < a.slices; k += kRowLanes * kAhead) {
        Stat x[kAhead], y[kAhead];
        load_stats(ps, k, a.slices, x);
        if (asks) load_stats(qs, k, a.slices, y);
        add_stats(x, c, p);
        if (asks) add_stats(y, c, q);
      }
      row_end(c, p);
      mine.row = i;
      // (Rows that two sequences claim may have been the other's, who sampled.)
      mine.greedy_token = p.top > kNegInf && p.first < a.V ? p.first : 0;
      mine.p_top = p.top;
      mine.p_inv = p.sum > 0.0 ? 1.0 / p.sum : 0.0;
      mine.drafted = -1;
      if (greedy) {
        stop = !(in && p.top > kNegInf && d == p.first && au < 1.0);
      } else {
        double qd = 1.0;
        if (asks) {
          row_end(c, q);
          mine.q_top = q.top;
          mine.q_inv = q.sum > 0.0 ? 1.0 / q.sum : 0.0;
          qd = weight_of(ql, q.top, c) * mine.q_inv;
        } else if (!final) {
          mine.drafted = d;
        }
        const double pd = in ? weight_of(pl, p.top, c) * mine.p_inv : 0.0;
        stop = final || !(au * qd < pd);
      }
    }
    const unsigned long long b = __ballot(stop);
    if (lane == 0) stops[wave].row = r.n;
    if (b && lane == __builtin_ctzll(b)) stops[wave] = mine;
    __syncthreads();
    st.row = r.n;
#pragma unroll
    for (int w = kWaves - 1; w >= 0; --w)
      if (stops[w].row < r.n) st = stops[w];
    if (st.row < r.n) break;
    __syncthreads();
  }
  const int row = r.q0 + st.row;
  const bool final = st.row == r.n - 1;

  int token = 0;
  bool failed = false;
  if (greedy) {
    token = st.greedy_token;
  } else {
    // This wave's share of the weights.
    const void* lp_row = static_cast<const L*>(a.logits) + (size_t)row * a.V;
    const bool with_q = a.draft && !final;
    const void* lq_row = with_q ? static_cast<const L*>(a.draft) + (size_t)row * a.V : lp_row;
    const int subs = a.slices * kWaves;
    unsigned long long* words = a.weight + (size_t)s * subs;
    {
      float lp[PER], lq[PER];
      const int n0 = (slice * kWaves + wave) * kSub<PER>;
      load_sub<L, VEC, PER>(lp_row, n0, a.V, lp);
      load_sub<L, VEC, PER>(lq_row, n0, a.V, lq);         // without q, lp again
      double w = 0.0;
#pragma unroll
      for (int j = 0; j < PER; j += kBatch) {
        int n[kBatch];
        double x[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) n[e] = n0 + index_of<L, VEC>(j + e);
        residuals(st, c, lp + j, lq + j, with_q, n, final, x);
#pragma unroll
        for (int e = 0; e < kBatch; ++e) w += x[e];
      }
      w = reduce64(w, plus);
      if (lane == 0)
        __hip_atomic_store(words + slice * kWaves + wave, __builtin_bit_cast(unsigned long long, w),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (tid == 0)
      is_last = __hip_atomic_fetch_add(&a.arrived[s], 1, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT) == a.slices - 1;
    __syncthreads();
    if (!is_last) return;

    // The wave's share where the running sum passes u times the total; without
    // any weight (p nowhere above q), the same over p itself, slice by slice.
    if (wave == 0) {
      const Stat* ps = a.stats + (size_t)row * a.slices;
      constexpr int kRun = 4;                        // words of a lane, neighbours
      double w[kRun], total = 0.0;
      // The lane's run of words from i0 on.  With `plain` a slice's sum counts
      // at its first word, and the slice is searched as a whole.
      static_assert(kRun == kWaves, "a lane's run is a slice");
      bool missing = a.polls < 0;
      const auto fetch = [&](int i0, bool plain) {
        const int i = i0 + lane * kRun;
        double x = 0.0;
        if (plain) {
          const Stat y = ps[min(i / kWaves, a.slices - 1)];
          w[0] = i < subs ? y.sum * weight_of(y.max, st.p_top, c) * st.p_inv : 0.0;
          w[1] = w[2] = w[3] = 0.0;
          x = w[0];
        } else {
          unsigned long long y[kRun];
          bool all = false;
          for (long long k = 0; !all && k <= a.polls; ++k) {
            all = true;
#pragma unroll
            for (int e = 0; e < kRun; ++e)
              y[e] = __hip_atomic_load(words + min(i, subs - kRun) + e, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int e = 0; e < kRun; ++e) all = all && y[e] != kNotYet;
          }
          missing = missing || !all;
#pragma unroll
          for (int e = 0; e < kRun; ++e) {
            w[e] = all && i < subs ? __builtin_bit_cast(double, y[e]) : 0.0;
            x += w[e];
          }
        }
        return x;
      };
      bool plain = false;
      for (int pass = 0; pass < 2 && !(total > 0.0); ++pass) {
        plain = pass;
        for (int i0 = 0; i0 < subs; i0 += 64 * kRun) total += lane_of(scan64(fetch(i0, plain)), 63);
      }
      const double goal = (u > 0.0 ? u : 0.0) * total;
      double before = 0.0, at_before = 0.0;
      int at = -1;                                   // else the last word with any weight
      bool hit = false;
      for (int i0 = 0; i0 < subs && !hit; i0 += 64 * kRun) {
        if (subs > 64 * kRun) fetch(i0, plain);      // else they are still there
        const double incl = scan64((w[0] + w[1]) + (w[2] + w[3]));
        const double prev = dpp<0x138>(incl);        // the lane before (wave_shr:1), 0 for the first
        double run = before + prev, b_over = 0.0, b_some = 0.0;
        int over = -1, some = -1;
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
          if (w[e] > 0.0) {
            some = e;
            b_some = run;
            if (over < 0 && run + w[e] > goal) {
              over = e;
              b_over = run;
            }
          }
          run += w[e];
        }
        const unsigned long long bo = __ballot(over >= 0), bs = __ballot(some >= 0);
        if (bo) {
          const int b = __builtin_ctzll(bo);
          at = i0 + b * kRun + __builtin_amdgcn_readlane(over, b);
          at_before = lane_of(b_over, b);
          hit = true;
        } else if (bs) {
          const int b = 63 - __builtin_clzll(bs);
          at = i0 + b * kRun + __builtin_amdgcn_readlane(some, b);
          at_before = lane_of(b_some, b);
        }
        before += lane_of(incl, 63);
      }
      const bool any_missing = __any(missing);
      if (lane == 0) {
        gave_up = any_missing;
        sub_s = max(at, 0);
        before_s = at_before;
        goal_s = goal;
        plain_s = plain;
        found = a.V;
        positive = 0;
      }
    }
    __syncthreads();
    // The entry among them: kFind neighbours per thread, in order.
    const bool plain = plain_s;
    double before = before_s;
    for (int k = 0; k < (plain ? kWaves : 1); ++k) {
      const int m0 = (sub_s + k) * kSub<PER> + tid * kFind;
      double x[kFind], sum = 0.0;
      float lp[kFind], lq[kFind];
      int n[kFind], some = -1;
#pragma unroll
      for (int j = 0; j < kFind; ++j) {
        n[j] = m0 + j;
        const int at = min(n[j], a.V - 1);
        lp[j] = logit<L>(lp_row, at);
        lq[j] = with_q ? logit<L>(lq_row, at) : kNegInf;
        if (n[j] >= a.V) lp[j] = __builtin_nanf("");
      }
      residuals(st, c, lp, lq, with_q, n, plain || final, x);
#pragma unroll
      for (int j = 0; j < kFind; ++j) {
        if (x[j] > 0.0) some = n[j];
        sum += x[j];
      }
      const double incl = scan64(sum);
      if (lane == 63) wsum[wave] = incl;
      __syncthreads();
      double run = before + dpp<0x138>(incl);
      for (int w = 0; w < wave; ++w) run += wsum[w];
      int hit = a.V;
#pragma unroll
      for (int j = 0; j < kFind; ++j) {
        run += x[j];
        if (hit == a.V && x[j] > 0.0 && run > goal_s) hit = m0 + j;
      }
      // One lane per wave: the lanes' places ascend, and 64 atomics on one word
      // are 64 in a row.
      const unsigned long long bh = __ballot(hit < a.V), bs = __ballot(some >= 0);
      if (bh && lane == __builtin_ctzll(bh)) atomicMin(&found, hit);
      if (bs && lane == 63 - __builtin_clzll(bs)) atomicMax(&positive, some);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) before += wsum[w];
      __syncthreads();
      if (found < a.V) break;
    }
    token = found < a.V ? found : positive;
    failed = gave_up;
  }

  for (int i = tid; i < r.n; i += kThreads) {
    const int next = i == tid ? kept : i + 1 < r.n ? a.tokens[r.q0 + i + 1] : -1;
    a.out_tokens[r.q0 + i] = failed ? -1 : i < st.row ? next : i == st.row ? token : -1;
  }
  if (tid == 0) a.accepted[s] = failed ? -1 : st.row;
}

// ---------------------------------------------------------------------------
// Host side.

constexpr int kShortSlices = 64, kShortGroups = 1024;   // of a row, of all rows

int slices_of(int vocab, int per) {
  const int slice = kThreads * per;
  return (vocab + slice - 1) / slice;
}
// Logits per lane of a step, by the rule above.
int per_of(int rows, int vocab) {
  const int slices = slices_of(vocab, kPerShort);
  return slices <= kShortSlices && rows <= kShortGroups / slices ? kPerShort : kPerLong;
}

size_t up(size_t b) { return (b + 255) / 256 * 256; }

struct Layout {
  size_t stats, weight, drafted, arrived, total;
};

// Room for either length of slices, so that more rows, sequences or entries
// never need less than fewer.
Layout layout(int rows, int seqs, int vocab) {
  const size_t sl = slices_of(vocab, kPerLong);
  const size_t few = std::min(slices_of(vocab, kPerShort), kShortSlices);
  const size_t stats = std::max(rows * sl, std::min(rows * few, (size_t)kShortGroups));
  Layout w;
  w.stats = 0;
  w.weight = up(2 * stats * sizeof(Stat));
  w.drafted = w.weight + up((size_t)seqs * std::max(sl, few) * kWaves * sizeof(double));
  w.arrived = w.drafted + up((size_t)2 * rows * sizeof(float));
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

template <typename L, bool VEC, int PER>
skinny_status launch(const VerifyArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((skinny_verify_stats<L, VEC, PER>), dim3(a.slices, a.T, a.draft ? 2 : 1),
                     dim3(kThreads), 0, stream, a);
  if (hipGetLastError() != hipSuccess) return SKINNY_ERR_HIP;
  hipLaunchKernelGGL((skinny_verify_pick<L, VEC, PER>), dim3(a.slices, a.S), dim3(kThreads), 0,
                     stream, a);
  return hipGetLastError() == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP;
}

template <typename L>
skinny_status launch_as(const VerifyArgs& a, hipStream_t stream) {
  const bool vec = a.V % kVec<L> == 0 && aligned(a.logits, 16) && (!a.draft || aligned(a.draft, 16));
  if (per_of(a.T, a.V) == kPerShort)
    return vec ? launch<L, true, kPerShort>(a, stream) : launch<L, false, kPerShort>(a, stream);
  return vec ? launch<L, true, kPerLong>(a, stream) : launch<L, false, kPerLong>(a, stream);
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
  a.weight = (unsigned long long*)(ws + w.weight);
  a.drafted = (float*)(ws + w.drafted);
  a.arrived = (int*)(ws + w.arrived);
  a.T = v.rows;
  a.S = v.seqs;
  a.V = v.vocab;
  a.slices = slices_of(v.vocab, per_of(v.rows, v.vocab));
  a.polls = g_polls.load();
  return v.dtype == SKINNY_LOGITS_BF16 ? launch_as<__bf16>(a, (hipStream_t)stream)
                                       : launch_as<float>(a, (hipStream_t)stream);
}

void skinny_verify_set_spin_limit(long long polls) { g_polls.store(polls); }

}  // extern "C"
