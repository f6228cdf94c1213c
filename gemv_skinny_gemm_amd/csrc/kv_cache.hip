// kv_cache.hip - gfx950 kernels and C ABI for the paged key/value cache of a
// decode or verify step: skinny_kv_append (position rotation, then the cache
// write in bf16 or in e4m3 with one scale per page and head) and
// skinny_kv_attention (each token's attention over its sequence's cache).
//
// Both stand between two of the step's linears: the QKV linear's y is
// kv_append's input, kv_attention's output is the O linear's x.  A decode
// step's attention reads every cached byte once per step, so like the linears
// it is bound by HBM bandwidth; grouped query heads share each byte ("Developing
// a custom Qwen2.5 72B inference engine from scratch - what is the real
// bottleneck?", section 6.3).
//
// Device arrays that describe the batch are never trusted: row ranges are
// clamped to [0, T], lengths to the page table, and a page number outside the
// pool is a page that no key of it is seen in and no row is written to.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

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
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBF16 = SKINNY_KV_BF16;
constexpr int kFP8 = SKINNY_KV_FP8;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxPosition = 1 << 30;
constexpr float kE4m3Max = 448.0f;
constexpr int kMinScaleExp = -64;

// The batch and the cache, as both operators' kernels take them.
struct KvArgs {
  unsigned char* k;        // [pages][kv_heads][P][D]
  unsigned char* v;
  float* k_scale;          // [pages][kv_heads] (FP8)
  float* v_scale;
  const int* q_start;      // [S + 1]
  const int* kv_len;       // [S]
  const int* table;        // [S][max_pages]
  int S;
  int T;
  int max_pages;
  int pages;
  int kv_heads;
  int group;               // query heads per KV head
  int group_shift;         // its log2, or -1: a division is some 200 cycles of a short call
  int log2p;               // log2 of the page's tokens
};

// A value that all lanes hold, or one lane's, as a scalar: addresses and
// branches that depend on it stay out of the vector registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int lane_of(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ float lane_of(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

__device__ __forceinline__ int by_group(const KvArgs& a, int x) {
  return a.group_shift >= 0 ? x >> a.group_shift : x / a.group;
}

// One sequence: rows q0 .. q0 + n of the batch; row i at position base + i,
// of which the first `cap` positions have a place in the page table.
struct Seq {
  int q0, n, base, cap;
};

__device__ __forceinline__ Seq load_seq(const KvArgs& a, int s) {
  Seq q;
  q.q0 = min(max(a.q_start[s], 0), a.T);
  q.n = min(max(a.q_start[s + 1], q.q0), a.T) - q.q0;
  const int len = min(max(a.kv_len[s], 0), kMaxPosition);
  q.base = len - q.n;
  q.cap = min(len, a.max_pages << a.log2p);
  return q;
}
__device__ __forceinline__ Seq uniform(const Seq& q) {
  return Seq{uniform(q.q0), uniform(q.n), uniform(q.base), uniform(q.cap)};
}

// Sum of two counts that stops at the largest int, so that row ranges which
// overlap (q_start not ascending) cannot wrap a count around.
constexpr int kMaxCount = 0x7fffffff;
__device__ __forceinline__ int add_count(int a, int b) {
  return (int)min((unsigned)a + (unsigned)b, (unsigned)kMaxCount);
}

// Inclusive sum over the wave's lanes of counts: shifts by 1, 2, 4, 8 within
// each 16 lanes, then the last lane of a row into the next row and of the lower
// half into the upper.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_from(int v) {
  return add_count(v, __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, true));
}
__device__ __forceinline__ int wave_scan(int v) {
  v = add_from<0x111, 0xf>(v);                       // row_shr
  v = add_from<0x112, 0xf>(v);
  v = add_from<0x114, 0xf>(v);
  v = add_from<0x118, 0xf>(v);
  v = add_from<0x142, 0xa>(v);                       // row_bcast15
  return add_from<0x143, 0xc>(v);                    // row_bcast31
}

// In a list of counts (one per sequence, `incl` their running sums over the
// wave's lanes, `before` the sum ahead of lane 0), the lane whose share holds
// `index`, or -1; `at` becomes the index within that share.
__device__ __forceinline__ int scan_find(int incl, int before, int index, int& at) {
  const unsigned long long b = __ballot(incl > index);
  if (!b) return -1;
  const int lane = __builtin_ctzll(b);
  at = index - (lane ? lane_of(incl, max(lane - 1, 0)) : before);
  return lane;
}

// ---------------------------------------------------------------------------
// Appending.

struct AppendArgs {
  KvArgs kv;
  const __bf16* qkv;       // [T][(q_heads + 2 kv_heads) D]
  __bf16* q_out;           // [T][q_heads D]
  const float* inv_freq;   // [rot / 2], or NULL
  int q_heads;
  int head_dim;
  int rot;                 // rotated values of a head, a multiple of 16
  int interleaved;         // pairs (2i, 2i + 1) rather than (i, i + rot / 2)
  int kv_blocks;           // workgroups of (touched page, head, k or v), the first of a launch
};

// A step of few rows takes skinny_kv_append_few, whose threads hold four values
// each; more rows take skinny_kv_append_many, whose threads hold 16 and share the
// angles.  Few rows cost a launch and one chain of reads (4 us in a graph); many
// are bound by bytes and the rotation in fp64 side by side: 4099 rows of 64
// + 2 x 8 heads of 128 into e4m3 pages take 44 us (160 MB: 3.6 TB/s, where
// a copy would take 33), 101 on the kernel of few rows.
constexpr int kQHeadsPerBlock = 16;  // few rows: query heads of one row's workgroup
constexpr int kUnit = 16;            // values of a unit: two runs of 8, at pa and pb

// cos and sin of pos * f.  The angle of a far position needs more than fp32
// (an error of 2^-24 of 10^6 rad is 0.06 rad), so it is taken in fp64 and
// reduced to half turns by 1 / pi in two doubles.
__device__ __forceinline__ void rotation(int pos, float f, double& c, double& s) {
  constexpr double kInvPiHi = 0x1.45f306dc9c883p-2, kInvPiLo = -0x1.6b01ec5417056p-56;
  const double x = (double)pos * (double)f;
  const double p = x * kInvPiHi;
  const double e = fma(x, kInvPiHi, -p) + x * kInvPiLo;
  sincospi((p - 2.0 * rint(0.5 * p)) + e, &s, &c);
}

// fp64 -> fp32 rounded to odd: an inexact value gets an odd last bit, so a
// later rounding to bf16 or e4m3 is that of the fp64 value itself (one
// rounding, not two).
__device__ __forceinline__ float to_odd(double x) {
  const float f = (float)x;
  const double back = (double)f;
  const unsigned u = __builtin_bit_cast(unsigned, f);
  // The nearest fp32 is one of the two neighbours; of an even one, take the other.
  const bool finite = (u & 0x7f800000u) != 0x7f800000u;
  const bool move = back != x && finite && !(u & 1);
  unsigned r = fabs(back) < fabs(x) ? u + 1 : u - 1;
  if (f == 0.0f) r = 1u | (x < 0.0 ? 0x80000000u : 0u);
  return __builtin_bit_cast(float, move ? r : u);
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  bf16x2 r;
  r[0] = (__bf16)a;
  r[1] = (__bf16)b;
  return __builtin_bit_cast(unsigned, r);
}

__device__ __forceinline__ float bf16_lo(unsigned u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) {
  return __builtin_bit_cast(float, u & 0xffff0000u);
}

// Two fp32 -> two e4m3 bytes, to nearest even; beyond 448 (infinities too)
// the largest number, NaN stays NaN.
__device__ __forceinline__ unsigned pack_e4m3(float a, float b) {
  const float ca = fminf(fmaxf(a, -kE4m3Max), kE4m3Max);
  const float cb = fminf(fmaxf(b, -kE4m3Max), kE4m3Max);
  unsigned r = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(ca, cb, 0, false) & 0xffffu;
  if (a != a) r = (r & 0xff00u) | 0x7fu;
  if (b != b) r = (r & 0x00ffu) | 0x7f00u;
  return r;
}

// The smallest power of two that brings a page's largest value to 448 = 1.75 *
// 2^8 or below.
__device__ __forceinline__ float page_scale(float top) {
  const unsigned bits = __builtin_bit_cast(unsigned, top);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return __builtin_bit_cast(float, (unsigned)(max(e, kMinScaleExp) + 127) << 23);
}

// Whether a page's scale, the same for all lanes, is a power of two: then products
// with it or its inverse are exact in fp32 (but for results that underflow, whose
// code is 0 all the same).
__device__ __forceinline__ bool power_of_two(float x) {
  return (uniform(__builtin_bit_cast(int, x)) & 0x7fffff) == 0;
}

// Other scales, the user's: x / scale rounded to odd, so that the code is the only
// rounding: a tie stays one, and nothing becomes one.  The product with the inverse
// is put right by what it leaves of x, to the last bit where the quotient is short.
__device__ __forceinline__ float quotient(float x, double scale, double inv) {
  const double q = x * inv;
  return to_odd(fma(fma(-q, scale, (double)x), inv, q));
}

// A page's older codes, four to a dword, from scale `had` to 1 / inv, a power of
// two: exact if `had` is one, but for codes that become subnormal; else rounded
// once, a code times both being exact in fp64.
__device__ __forceinline__ void rescale(unsigned* codes, int n, float had, double inv, int tid) {
  const double ratio = (double)had * inv;
  const auto every = [&](auto times) {
    for (int i = tid; i < n; i += kThreads) {
      const unsigned c = codes[i];
      const f32x2 x = __builtin_amdgcn_cvt_pk_f32_fp8(c, false);
      const f32x2 y = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
      codes[i] = pack_e4m3(times(x[0]), times(x[1])) | pack_e4m3(times(y[0]), times(y[1])) << 16;
    }
  };
  if (__builtin_expect(power_of_two(had), 1)) every([r = (float)ratio](float x) { return x * r; });
  else every([&](float x) { return to_odd(x * ratio); });
}

// A quad is four values of a head: two neighbours at pa and two at pb that
// rotate together (half-split: partners lie rot / 2 apart), or, unrotated or
// interleaved, four in a row.
struct Quad {
  int pa, pb;
  bool turned;
};

__device__ __forceinline__ Quad quad_of(int j, int rot, int interleaved) {
  Quad u;
  u.turned = 4 * j < rot;
  const bool split = u.turned && !interleaved;
  u.pa = split ? 2 * j : 4 * j;
  u.pb = split ? rot / 2 + 2 * j : 4 * j + 2;
  return u;
}

// Rotates a quad's values by the frequencies (c0, s0), (c1, s1) in fp64.
__device__ __forceinline__ f32x4 turn(unsigned a, unsigned b, int interleaved, double c0, double s0,
                                      double c1, double s1) {
  const double a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
  f32x4 r;
  if (interleaved) {
    r[0] = to_odd(a0 * c0 - a1 * s0);
    r[1] = to_odd(a0 * s0 + a1 * c0);
    r[2] = to_odd(b0 * c1 - b1 * s1);
    r[3] = to_odd(b0 * s1 + b1 * c1);
  } else {
    r[0] = to_odd(a0 * c0 - b0 * s0);
    r[1] = to_odd(a1 * c1 - b1 * s1);
    r[2] = to_odd(a0 * s0 + b0 * c0);
    r[3] = to_odd(a1 * s1 + b1 * c1);
  }
  return r;
}

// Unit j of a head: half-split, its runs lie rot / 2 apart and rotate with each
// other; interleaved, or not rotated, they are neighbours.
struct Unit {
  int pa, pb;
  bool turned;
};

__device__ __forceinline__ Unit unit_of(int j, int rot, int interleaved) {
  Unit u;
  u.turned = kUnit * j < rot;
  const bool split = u.turned && !interleaved;
  u.pa = split ? 8 * j : kUnit * j;
  u.pb = split ? rot / 2 + 8 * j : kUnit * j + 8;
  return u;
}

// cos and sin of one row's angles in LDS: unit j rotates by frequencies 8j .. 8j
// + 7, and entry e of all units lies together, so that the units' lanes read
// neighbours.
__device__ __forceinline__ int turn_at(int freq, int rot) {
  return freq % 8 * (rot / kUnit) + freq / 8;
}
typedef double f64x2 __attribute__((ext_vector_type(2)));

// A unit's values in fp64, rotated.
struct Values {
  double a[8], b[8];
};
__device__ __forceinline__ Values unpack(u32x4 x, u32x4 y) {
  Values v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.a[2 * i] = bf16_lo(x[i]);
    v.a[2 * i + 1] = bf16_hi(x[i]);
    v.b[2 * i] = bf16_lo(y[i]);
    v.b[2 * i + 1] = bf16_hi(y[i]);
  }
  return v;
}
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(Values& v, const f64x2* cs, int j, int rot) {
  const int step = rot / kUnit;
  const auto pair = [&](double& a, double& b, int e) {
    const f64x2 t = cs[e * step + j];
    const double x = a * t[0] - b * t[1];
    b = a * t[1] + b * t[0];
    a = x;
  };
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pair(v.a[2 * i], v.a[2 * i + 1], i);
      pair(v.b[2 * i], v.b[2 * i + 1], 4 + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) pair(v.a[i], v.b[i], i);
  }
}

// Eight fp64 -> bf16, each rounded once, to nearest even.  fp64 -> fp32 -> bf16
// rounds wrongly only where the fp32 value lies half way between two bf16 ones
// (its low 16 bits are 0x8000), once in 2^16; then it goes over rounding to odd.
__device__ __forceinline__ u32x4 round_bf16(const double (&v)[8]) {
  float f[8];
  bool half = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = (float)v[i];
    half = half || (__builtin_bit_cast(unsigned, f[i]) & 0xffffu) == 0x8000u;
  }
  if (half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_odd(v[i]);
  }
  return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
               pack_bf16(f[6], f[7])};
}

// Sequence of batch row t, or -1 for a row behind the last one.
__device__ __forceinline__ int find_row(const KvArgs& a, int t) {
  const int lane = threadIdx.x & 63;
  for (int s0 = 0; s0 < a.S; s0 += 64) {
    const int s = s0 + lane;
    const bool hit = s < a.S && a.q_start[s] <= t && t < a.q_start[s + 1];
    const unsigned long long b = __ballot(hit);
    if (b) return s0 + __builtin_ctzll(b);
  }
  return -1;
}

// First page and number of pages that a sequence's new rows fall into.
__device__ __forceinline__ int touched(const Seq& q, int log2p, int& first) {
  const int lo = max(q.base, 0), hi = min(q.base + q.n, q.cap);
  first = lo >> log2p;
  return lo < hi ? ((hi - 1) >> log2p) - first + 1 : 0;
}

// The unit-th page that receives rows, sequences in order.
struct NewRows {
  int page;       // -1: there is none, or not in the pool
  int lo;         // position of the first
  int count;      // 1 .. page_tokens
  int older;      // rows of the sequence before them in the page
  size_t row;     // the first one's, in the batch
};
__device__ __forceinline__ NewRows find_page(const KvArgs& kv, int unit) {
  const int lane = threadIdx.x & 63;
  int s = -1, page_no = 0, before = 0;
  for (int s0 = 0; s0 < kv.S && s < 0; s0 += 64) {
    int first = 0, c = 0;
    if (s0 + lane < kv.S) c = touched(load_seq(kv, s0 + lane), kv.log2p, first);
    const int incl = add_count(wave_scan(c), before);
    int idx;
    const int at = scan_find(incl, before, unit, idx);
    if (at >= 0) {
      s = s0 + at;
      page_no = lane_of(first, at) + idx;
    }
    before = lane_of(incl, 63);
  }
  if (s < 0) return NewRows{-1, 0, 0, 0, 0};
  const Seq q = uniform(load_seq(kv, s));
  const int lo = max(max(q.base, 0), page_no << kv.log2p);
  const int hi = min(min(q.base + q.n, q.cap), (page_no + 1) << kv.log2p);
  const int page = kv.table[(size_t)s * kv.max_pages + page_no];
  return NewRows{page < kv.pages ? page : -1, lo, hi - lo, lo & ((1 << kv.log2p) - 1),
                 (size_t)(q.q0 + (lo - q.base))};
}

// One workgroup per (page that receives rows, KV head, k or v), which alone
// reads and writes that page's block and scale, then one per token and
// kQHeadsPerBlock query heads.  The rotated rows wait in LDS (as fp32 rounded
// to odd) between the maximum and the rounding.
template <int DT>
__global__ __launch_bounds__(kThreads) void skinny_kv_append_few(const AppendArgs a) {
  extern __shared__ f32x4 rows[];                    // [new rows][D / 4]
  __shared__ float smax[kWaves];
  const KvArgs& kv = a.kv;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int D = a.head_dim;
  const int upr = D / 4;                             // units per row
  const size_t row_elems = (size_t)(a.q_heads + 2 * kv.kv_heads) * D;

  if ((int)blockIdx.x >= a.kv_blocks) {              // query heads
    const int chunks = (a.q_heads + kQHeadsPerBlock - 1) / kQHeadsPerBlock;
    const int b = blockIdx.x - a.kv_blocks;
    const int t = b / chunks;
    const int h0 = b % chunks * kQHeadsPerBlock;
    const int h1 = min(h0 + kQHeadsPerBlock, a.q_heads);
    const int s = find_row(kv, t);
    if (s < 0) return;
    const Seq q = uniform(load_seq(kv, s));
    const int pos = q.base + (t - q.q0);
    double* cs = reinterpret_cast<double*>(rows);    // [rot / 2] (cos, sin)
    for (int i = tid; i < a.rot / 2; i += kThreads) rotation(pos, a.inv_freq[i], cs[2 * i], cs[2 * i + 1]);
    __syncthreads();
    const unsigned* src = reinterpret_cast<const unsigned*>(a.qkv + t * row_elems);
    unsigned* dst = reinterpret_cast<unsigned*>(a.q_out + (size_t)t * a.q_heads * D);
    for (int i = h0 * upr + tid; i < h1 * upr; i += kThreads) {
      const int h = i / upr, j = i % upr;
      const Quad u = quad_of(j, a.rot, a.interleaved);
      unsigned x = src[(h * D + u.pa) / 2], y = src[(h * D + u.pb) / 2];
      if (u.turned) {
        const f32x4 r = turn(x, y, a.interleaved, cs[4 * j], cs[4 * j + 1], cs[4 * j + 2],
                             cs[4 * j + 3]);
        x = pack_bf16(r[0], r[1]);
        y = pack_bf16(r[2], r[3]);
      }
      dst[(h * D + u.pa) / 2] = x;
      dst[(h * D + u.pb) / 2] = y;
    }
    return;
  }

  const bool is_v = blockIdx.x & 1;
  const int h = (blockIdx.x >> 1) % kv.kv_heads;
  const NewRows fresh = find_page(kv, (blockIdx.x >> 1) / kv.kv_heads);
  if (fresh.page < 0) return;
  const int P = 1 << kv.log2p, lo = fresh.lo, count = fresh.count, older = fresh.older,
            page = fresh.page;
  constexpr int kEsize = DT == kBF16 ? 2 : 1;
  unsigned char* block = (is_v ? kv.v : kv.k) + ((size_t)page * kv.kv_heads + h) * P * D * kEsize;
  const int rot = is_v ? 0 : a.rot;
  const unsigned* src = reinterpret_cast<const unsigned*>(
      a.qkv + fresh.row * row_elems +
      (size_t)(a.q_heads + (is_v ? kv.kv_heads : 0) + h) * D);

  float top = 0.0f;
  for (int i = tid; i < count * upr; i += kThreads) {
    const int r = i / upr, j = i % upr;
    const Quad u = quad_of(j, rot, a.interleaved);
    const unsigned x = src[(r * row_elems + u.pa) / 2], y = src[(r * row_elems + u.pb) / 2];
    f32x4 w{bf16_lo(x), bf16_hi(x), bf16_lo(y), bf16_hi(y)};
    if (u.turned) {
      double c0, s0, c1, s1;
      rotation(lo + r, a.inv_freq[2 * j], c0, s0);
      rotation(lo + r, a.inv_freq[2 * j + 1], c1, s1);
      w = turn(x, y, a.interleaved, c0, s0, c1, s1);
    }
    if constexpr (DT == kBF16) {
      unsigned* dst = reinterpret_cast<unsigned*>(block) + (size_t)(older + r) * D / 2;
      dst[u.pa / 2] = pack_bf16(w[0], w[1]);
      dst[u.pb / 2] = pack_bf16(w[2], w[3]);
    } else {
      rows[i] = w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float m = fabsf(w[e]);
        if (m < __builtin_inff()) top = fmaxf(top, m);
      }
    }
  }
  if constexpr (DT == kFP8) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    if (lane == 0) smax[tid >> 6] = top;
    float* scale = (is_v ? kv.v_scale : kv.k_scale) + (size_t)page * kv.kv_heads + h;
    const float had = older ? *scale : 0.0f;
    __syncthreads();
    top = fmaxf(fmaxf(smax[0], smax[1]), fmaxf(smax[2], smax[3]));
    const float need = page_scale(top);
    const float now = had >= need ? had : need;
    const double inv = 1.0 / (double)now;
    const bool exact = power_of_two(now);
    if (older && now != had) rescale(reinterpret_cast<unsigned*>(block), older * upr, had, inv, tid);
    const auto every = [&](auto scaled) {
      for (int i = tid; i < count * upr; i += kThreads) {
        const int r = i / upr, j = i % upr;
        const Quad u = quad_of(j, rot, a.interleaved);
        const f32x4 w = rows[i];
        unsigned short* dst = reinterpret_cast<unsigned short*>(block + (size_t)(older + r) * D);
        dst[u.pa / 2] = (unsigned short)pack_e4m3(scaled(w[0]), scaled(w[1]));
        dst[u.pb / 2] = (unsigned short)pack_e4m3(scaled(w[2]), scaled(w[3]));
      }
    };
    if (__builtin_expect(exact, 1)) every([f = (float)inv](float x) { return x * f; });
    else every([&](float x) { return quotient(x, now, inv); });
    if (tid == 0) *scale = now;
  }
}

// Query heads of many rows: a workgroup takes kQRows rows, one per wave, whose
// angles (cs: [kQRows][rot / 2]) its threads compute together.
constexpr int kQRows = kWaves;
constexpr int kQAhead = 2;           // units of a lane in flight
template <bool INTERLEAVED>
__device__ __forceinline__ void append_queries(const AppendArgs& a, int block, f64x2* cs,
                                               int (&places)[kQRows]) {
  const KvArgs& kv = a.kv;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int D = a.head_dim;
  const int upr = D / kUnit;                         // units of a head
  const int units = a.q_heads * upr;
  const size_t row_elems = (size_t)(a.q_heads + 2 * kv.kv_heads) * D;
  const int t = block * kQRows + wave;
  const __bf16* src = a.qkv + t * row_elems;
  __bf16* dst = a.q_out + (size_t)t * a.q_heads * D;
  u32x4 x[kQAhead], y[kQAhead];
  const auto load = [&](int i0) {
#pragma unroll
    for (int e = 0; e < kQAhead; ++e) {
      const int i = min(i0 + 64 * e + lane, units - 1);
      const Unit u = unit_of(i % upr, a.rot, INTERLEAVED);
      x[e] = *reinterpret_cast<const u32x4*>(src + (size_t)(i / upr) * D + u.pa);
      y[e] = *reinterpret_cast<const u32x4*>(src + (size_t)(i / upr) * D + u.pb);
    }
  };
  int s = -1;
  if (t < kv.T) {
    load(0);                                         // on their way while the row is looked up
    s = find_row(kv, t);
    if (s >= 0) {
      const Seq q = load_seq(kv, s);
      if (lane == 0) places[wave] = q.base + (t - q.q0);
    }
  }
  if (s < 0 && lane == 0) places[wave] = 0;
  __syncthreads();
  for (int i = tid; i < kQRows * (a.rot / 2); i += kThreads) {
    const int r = i / (a.rot / 2), f = i % (a.rot / 2);
    double c, sn;
    rotation(places[r], a.inv_freq[f], c, sn);
    cs[r * (a.rot / 2) + turn_at(f, a.rot)] = f64x2{c, sn};
  }
  __syncthreads();
  if (s < 0) return;
  const f64x2* mine = cs + wave * (a.rot / 2);
  for (int i0 = 0; i0 < units; i0 += 64 * kQAhead) {
    u32x4 nx[kQAhead], ny[kQAhead];
#pragma unroll
    for (int e = 0; e < kQAhead; ++e) {
      nx[e] = x[e];
      ny[e] = y[e];
    }
    if (i0 + 64 * kQAhead < units) load(i0 + 64 * kQAhead);
#pragma unroll
    for (int e = 0; e < kQAhead; ++e) {
      const int i = i0 + 64 * e + lane;
      if (i >= units) continue;
      const Unit u = unit_of(i % upr, a.rot, INTERLEAVED);
      if (u.turned) {
        Values v = unpack(nx[e], ny[e]);
        turn<INTERLEAVED>(v, mine, i % upr, a.rot);
        nx[e] = round_bf16(v.a);
        ny[e] = round_bf16(v.b);
      }
      *reinterpret_cast<u32x4*>(dst + (size_t)(i / upr) * D + u.pa) = nx[e];
      *reinterpret_cast<u32x4*>(dst + (size_t)(i / upr) * D + u.pb) = ny[e];
    }
  }
}

// A step of many rows: one workgroup per (page, KV head, k or v), then those of
// the query heads, which fill the chip beside the pages' arithmetic.  A pass takes a
// unit per thread, kThreads * kUnit / D rows, whose angles lie in LDS; an e4m3
// page's values wait in registers between the maximum and the rounding (PASSES of
// 16 fp32, rounded to odd).
template <int DT, bool INTERLEAVED, int PASSES>
__global__ __launch_bounds__(kThreads) void skinny_kv_append_many(const AppendArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ float smax[kWaves];
  __shared__ int places[kQRows];
  const KvArgs& kv = a.kv;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int D = a.head_dim;
  const int upr = D / kUnit;                         // units of a head
  const size_t row_elems = (size_t)(a.q_heads + 2 * kv.kv_heads) * D;
  f64x2* cs = reinterpret_cast<f64x2*>(lds);         // [rows of a pass][rot / 2]
  if ((int)blockIdx.x >= a.kv_blocks) {
    append_queries<INTERLEAVED>(a, blockIdx.x - a.kv_blocks, cs, places);
    return;
  }

  const bool is_v = blockIdx.x & 1;
  const int h = (blockIdx.x >> 1) % kv.kv_heads;
  const NewRows fresh = find_page(kv, (blockIdx.x >> 1) / kv.kv_heads);
  if (fresh.page < 0) return;
  const int P = 1 << kv.log2p, lo = fresh.lo, count = fresh.count, older = fresh.older,
            page = fresh.page;
  constexpr int kEsize = DT == kBF16 ? 2 : 1;
  unsigned char* block = (is_v ? kv.v : kv.k) + ((size_t)page * kv.kv_heads + h) * P * D * kEsize;
  const int rot = is_v ? 0 : a.rot;
  const __bf16* src = a.qkv + fresh.row * row_elems +
                      (size_t)(a.q_heads + (is_v ? kv.kv_heads : 0) + h) * D;
  float* scale = nullptr;
  float had = 0.0f;
  if constexpr (DT == kFP8) {
    scale = (is_v ? kv.v_scale : kv.k_scale) + (size_t)page * kv.kv_heads + h;
    if (older) had = *scale;
  }
  const int step = kThreads / upr;                   // rows of a pass
  const int j = tid % upr;
  const Unit u = unit_of(j, rot, INTERLEAVED);
  u32x4 x[PASSES], y[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const __bf16* row = src + (size_t)min(p * step + tid / upr, count - 1) * row_elems;
    x[p] = *reinterpret_cast<const u32x4*>(row + u.pa);
    y[p] = *reinterpret_cast<const u32x4*>(row + u.pb);
  }

  float top = 0.0f;
  float w[DT == kFP8 ? PASSES : 1][kUnit];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r0 = p * step, n = min(step, count - r0), r = r0 + tid / upr;
    if (n <= 0) break;
    if (rot) {
      if (p) __syncthreads();
      // A thread takes a frequency over a run of rows: the first row's angle, then
      // a complex product by the frequency's own per row (fp64: a few 2^-53).
      const int half = rot / 2, runs = max(1, kThreads / half), run = (n + runs - 1) / runs;
      for (int i = tid; i < half * runs; i += kThreads) {
        const int f = i % half, r1 = i / half * run;
        if (r1 >= n) continue;
        double c, sn, cf, sf;
        rotation(lo + r0 + r1, a.inv_freq[f], c, sn);
        rotation(1, a.inv_freq[f], cf, sf);
        for (int k = r1; k < min(r1 + run, n); ++k) {
          cs[k * half + turn_at(f, rot)] = f64x2{c, sn};
          const double next = c * cf - sn * sf;
          sn = c * sf + sn * cf;
          c = next;
        }
      }
      __syncthreads();
    }
    const bool live = r < count;
    Values v;
    if (live && u.turned) {
      v = unpack(x[p], y[p]);
      turn<INTERLEAVED>(v, cs + (r - r0) * (rot / 2), j, rot);
    }
    if constexpr (DT == kBF16) {
      if (live) {
        if (u.turned) {
          x[p] = round_bf16(v.a);
          y[p] = round_bf16(v.b);
        }
        __bf16* dst = reinterpret_cast<__bf16*>(block) + (size_t)(older + r) * D;
        *reinterpret_cast<u32x4*>(dst + u.pa) = x[p];
        *reinterpret_cast<u32x4*>(dst + u.pb) = y[p];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[p][2 * e] = bf16_lo(x[p][e]);
        w[p][2 * e + 1] = bf16_hi(x[p][e]);
        w[p][8 + 2 * e] = bf16_lo(y[p][e]);
        w[p][8 + 2 * e + 1] = bf16_hi(y[p][e]);
      }
      if (live && u.turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[p][e] = to_odd(v.a[e]);
          w[p][8 + e] = to_odd(v.b[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < kUnit; ++e) {
        const float m = fabsf(w[p][e]);
        if (live && m < __builtin_inff()) top = fmaxf(top, m);
      }
    }
  }
  if constexpr (DT == kFP8) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    if (lane == 0) smax[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(smax[0], smax[1]), fmaxf(smax[2], smax[3]));
    const float need = page_scale(top);
    const float now = had >= need ? had : need;
    const double inv = 1.0 / (double)now;
    const bool exact = power_of_two(now);
    if (older && now != had) rescale(reinterpret_cast<unsigned*>(block), older * D / 4, had, inv, tid);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * step + tid / upr;
      if (r >= count) break;
      if (__builtin_expect(exact, 1)) {
#pragma unroll
        for (int e = 0; e < kUnit; ++e) w[p][e] *= (float)inv;
      } else {
#pragma unroll
        for (int e = 0; e < kUnit; ++e) w[p][e] = quotient(w[p][e], now, inv);
      }
      unsigned c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[e] = pack_e4m3(w[p][4 * e], w[p][4 * e + 1]) |
               pack_e4m3(w[p][4 * e + 2], w[p][4 * e + 3]) << 16;
      unsigned char* dst = block + (size_t)(older + r) * D;
      *reinterpret_cast<u32x2*>(dst + u.pa) = u32x2{c[0], c[1]};
      *reinterpret_cast<u32x2*>(dst + u.pb) = u32x2{c[2], c[3]};
    }
    if (tid == 0) *scale = now;
  }
}

// ---------------------------------------------------------------------------
// Attention.
//
// out = softmax(scale q k^T + mask) v over a sequence's cache, one pass with
// the running maximum m and sum l of exp2 (scores carry log2 e): a larger
// maximum scales the sums by 2^(m - m').
//
// A work item is (sequence, KV head, row group): up to ROWS rows, row r =
// i * group + g being token i under query head g of the KV head, so each cached
// byte serves every head that shares it.  A workgroup's waves are RW by KW: RW
// waves take 16 RT rows each of the same keys (the second to read a key finds
// it in the caches), KW waves take different keys.  A wave takes 32 keys at a
// time and keeps everything in registers:
//   S^T = K Q^T    v_mfma_f32_16x16x32_bf16, A = 16 keys, B = 16 rows.  Lane
//                  (c = lane % 16, g = lane / 16) ends with row c's scores of
//                  keys 4g .. 4g + 3, so a row's statistics need two lane
//                  exchanges (lanes +16, +32) and nothing else;
//   O^T += V^T P^T the products' k index may run over the keys in any order
//                  that A and B share: lane (c, g) takes as its eight keys the
//                  ones whose scores it holds (4g + 0..3 of both 16-key
//                  halves), so P goes from the scores straight into the B
//                  operand, as two bf16 numbers per probability (below).  For A the
//                  lane loads D / 16 neighbouring values of those eight keys and
//                  turns the 8 x D / 16 block around with byte permutes: output tile
//                  j holds values c D/16 + j.
// Keys and values therefore go from HBM to registers with no LDS and no
// barrier in the loop; e4m3 codes become bf16 exactly, and a page's scale is
// folded into the scores (k) and the probabilities (v).
//
// Short items stay whole, each in one workgroup (stays_whole).  Else the blocks
// of 32 KW keys of all items, in order, are cut into equal shares, one per
// workgroup (every workgroup computes the cut from the batch's device arrays);
// each wave takes an equal run of a segment's keys.  A segment that is
// not a whole item leaves its m, l and O in the workspace, and a second launch
// joins an item's segments in order: no atomics, so a result depends on the
// lengths and the grid only.  (Joining in the first launch, by the last segment
// to arrive, was measured at 1.5 to 3 times the whole call: the fences between
// workgroups of different XCDs write back and invalidate the L2 caches that the
// other waves stream through.)
//
// What bounds it, measured: long contexts the reads (bf16, 16 sequences, 64
// query and 8 KV heads of 128: 538 MB of pages in 99.0 us = 5.4 TB/s, 2167 MB in
// 346 = 6.3; e4m3, one sequence of 131072 keys: 51.8 us = 5.2 TB/s, where 4 us
// are the second launch and about 5 the start and the waves' join); a short call
// the chain start - page numbers - keys - join - second launch (4000 keys under
// one KV head: 10.0 us, of which 3.2 the second launch).  Rows of several tokens
// share the keys' bytes but not the work on them: 131072 keys under 8, 16, 32, 48,
// 64 and 96 rows per KV head take 52, 53, 57, 78, 78 and 126 us (32 keys by 32 rows
// are some 2000 cycles of a wave's instructions), two sequences of 12 verified
// tokens between them read 77 MB in 38.6 us, prompts of 4099 rows in three sequences
// of up to 9001 keys take 1364 us (504 TFLOP/s; bf16 3376, 204).  Tried on the two
// sequences when a probability was one bf16 number, against 35.6 us then, and no
// faster: three row tiles per wave with q in LDS (36.6 us), four row waves (45.9),
// a second tile of keys and values in flight in registers (82; it spills), two
// workgroups per CU (45.0; 59.6 against 51.7 on the long sequence).

constexpr int kMaxGroups = 256;          // workgroups of the grid, one per CU, at most
constexpr size_t kSplitBytes = kMaxGroups * 32;
constexpr float kNegInf = -__builtin_inff();
// The maximum of a row that sees keys, but with scores of -inf (or NaN) only: lower
// than another share's, and at the end 0 / 0, where -inf, no key seen, is zeros.
constexpr float kAllNegInf = -__FLT_MAX__;
// m need not be the maximum itself, only near it: sums are scaled again when a
// score passes it by more than this (probabilities then reach 2^8, far from
// fp32's and bf16's ends).  A wave's first tiles would otherwise do so nearly
// every time, one of its 16 rows finding a new maximum (1 to 2% of a verify step's
// time, nothing elsewhere).
constexpr float kSlack = 8.0f;

// What a share leaves for the second launch: the item that begins in it and
// goes on in the next ones, if there is one.
struct Split {
  int n;          // segments, one per share from this one on (0: no such item)
  int rows;       // rows of the item
  int row0;       // the first one's number: token * group + query head of its KV head
  int q0;         // the sequence's first row in the batch
  int h;          // KV head
};
static_assert(kMaxGroups * sizeof(Split) <= kSplitBytes, "room for every share's");

struct AttnArgs {
  KvArgs kv;
  const __bf16* q;         // [T][q_heads D]
  __bf16* out;             // [T][q_heads D]
  Split* splits;           // [grid]
  float* part;             // [2 grid] segments: [ROWS][D] sums, [ROWS] m, [ROWS] l
  float scale;             // softmax scale * log2 e
  int groups;              // workgroups
  int whole;               // each item is one block of one workgroup: nothing to join
};

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool HIGH>
__device__ __forceinline__ unsigned e4m3x2_to_bf16(unsigned v) {
  return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, HIGH));
}

// Blocks of one (row group, KV head) of a sequence, and its row groups.
// An item without keys has one block, for its rows' zeros.
struct Cut {
  int rows;       // of a row group
  int keys;       // of a block
  int whole;      // each item is one block
};
__device__ __forceinline__ int seq_blocks(const Seq& q, Cut cut) {
  return cut.whole ? 1 : max(1, (q.cap + cut.keys - 1) / cut.keys);
}
__device__ __forceinline__ int seq_row_groups(const Seq& q, int group, Cut cut) {
  return (q.n * group + cut.rows - 1) / cut.rows;
}
__device__ __forceinline__ int seq_work(const KvArgs& a, const Seq& q, Cut cut) {
  const long long w = (long long)seq_row_groups(q, a.group, cut) * a.kv_heads * seq_blocks(q, cut);
  return (int)(w < kMaxCount ? w : kMaxCount);
}

// Where a block number falls.
struct Place {
  int s;          // sequence
  int item;       // h * row groups + row group
  int blk;        // block within the item
  int nb;         // blocks of the item
  int rgs;        // row groups of the sequence
  Seq q;
};

// The sequences' work, in running sums over the wave's lanes, 64 at a time;
// the first 64 sequences' stay in the lanes.
struct Work {
  Seq q;          // of sequence `lane`
  int incl;       // blocks up to and with it
  int total;      // blocks of all sequences
};

__device__ __forceinline__ Work all_work(const KvArgs& a, Cut cut) {
  const int lane = threadIdx.x & 63;
  Work w{};
  int own = 0;
  if (lane < a.S) {
    w.q = load_seq(a, lane);
    own = seq_work(a, w.q, cut);
  }
  w.incl = wave_scan(own);
  w.total = lane_of(w.incl, 63);
  for (int s0 = 64; s0 < a.S; s0 += 64) {
    const int more = s0 + lane < a.S ? seq_work(a, load_seq(a, s0 + lane), cut) : 0;
    w.total = add_count(w.total, lane_of(wave_scan(more), 63));
  }
  return w;
}

__device__ __forceinline__ Place place_of(const KvArgs& a, Cut cut, const Work& work, int pos) {
  const int lane = threadIdx.x & 63;
  Place p{};
  int idx = 0;
  int at = scan_find(work.incl, 0, pos, idx);
  if (at >= 0) {
    p.s = at;
    p.q = Seq{lane_of(work.q.q0, at), lane_of(work.q.n, at), lane_of(work.q.base, at),
              lane_of(work.q.cap, at)};
  } else {
    int before = lane_of(work.incl, 63);
    for (int s0 = 64; s0 < a.S && at < 0; s0 += 64) {
      const int more = s0 + lane < a.S ? seq_work(a, load_seq(a, s0 + lane), cut) : 0;
      const int incl = add_count(wave_scan(more), before);
      at = scan_find(incl, before, pos, idx);
      p.s = s0 + at;
      before = lane_of(incl, 63);
    }
    p.q = uniform(load_seq(a, p.s));
  }
  p.nb = seq_blocks(p.q, cut);
  p.rgs = seq_row_groups(p.q, a.group, cut);
  p.item = idx / p.nb;
  p.blk = idx - p.item * p.nb;
  return p;
}

// The cut of `total` blocks into equal shares, the first `rest` of them one
// block longer.
struct Shares {
  int base, rest;
  __device__ __forceinline__ Shares(int total, int groups)
      : base(total / groups), rest(total - base * groups) {}
  __device__ __forceinline__ int begin(int b) const { return b * base + min(b, rest); }
  __device__ __forceinline__ int of(int pos) const {      // the share of a block
    const int longer = rest * (base + 1);
    return pos < longer ? pos / (base + 1) : rest + (pos - longer) / base;
  }
};

// Floats of one segment in the workspace.
template <int D>
__host__ __device__ constexpr int part_floats(int rows) {
  return rows * (D + 2);
}

// A lane's value and that of the lane 32 (or 16) away, in either order.
struct Pair {
  float a, b;
};
__device__ __forceinline__ Pair across32(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned lo = s[0], hi = s[1];
  return Pair{__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}
__device__ __forceinline__ Pair across16(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned lo = s[0], hi = s[1];
  return Pair{__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}

// Largest value, and sum, over the four lanes of a row (lane, +16, +32, +48).
__device__ __forceinline__ float row_max(float x) {
  const Pair p = across32(x);
  const Pair q = across16(fmaxf(p.a, p.b));
  return fmaxf(q.a, q.b);
}
__device__ __forceinline__ float row_sum(float x) {
  const Pair p = across32(x);
  const Pair q = across16(p.a + p.b);
  return q.a + q.b;
}

// Bytes (FP8) or halves (bf16) of x that are no finite number, as full masks.
template <int DT>
__device__ __forceinline__ unsigned not_finite(unsigned x) {
  if constexpr (DT == kFP8) {
    const unsigned f = ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // 0x7f: NaN
    return f | (f - (f >> 7));
  } else {
    const unsigned f = ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;   // exponent all ones
    return f | (f - (f >> 15));
  }
}

// A use of a loaded value that costs no instruction: the wait for it stands
// here, and later ones in a loop need not allow for it.
template <typename T>
__device__ __forceinline__ void arrived(T& x) {
  asm volatile("" : "+v"(x));
}
template <typename T, int N>
__device__ __forceinline__ void arrived(T (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) arrived(x[i]);
}

// Results of matrix instructions, before vector instructions read them.  The
// hardware does not hold a vector read back until the matrix instruction has
// written (12 slots are enough for these); the compiler fills the slots between
// instructions of one basic block, but where a branch came in between it was
// seen to leave them out, and the scores then lacked their last product.  The
// slots stand here: behind every value's matrix instructions, and what depends
// on the values behind the slots (volatile asm keeps its order).
template <typename... T>
__device__ __forceinline__ void settle(T&... x) {
  (arrived(x), ...);
  asm volatile("s_nop 7\n\ts_nop 3");
  (arrived(x), ...);
}

// Loads of the cache; NT with the nontemporal hint, for bytes that one wave of
// the call reads, in whole cache lines.
template <bool NT, typename T>
__device__ __forceinline__ T load_as(const unsigned char* p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
  else return *reinterpret_cast<const T*>(p);
}
template <bool NT, int W>
__device__ __forceinline__ void load_words(const unsigned char* p, unsigned (&out)[W]) {
  if constexpr (W == 1) {
    out[0] = load_as<NT, unsigned>(p);
  } else if constexpr (W == 2) {
    const u32x2 x = load_as<NT, u32x2>(p);
    out[0] = x[0];
    out[1] = x[1];
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const u32x4 x = load_as<NT, u32x4>(p + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) out[i + e] = x[e];
    }
  }
}

template <int DT, int D>
struct Shape {
  static constexpr int kRowBytes = D * (DT == kBF16 ? 2 : 1);
  static constexpr int kLoads = kRowBytes / 64;      // 16-byte K loads per lane and 16 keys
  static constexpr int kSteps = D / 32;              // products over D per 16 keys
  static constexpr int kPart = DT == kBF16 ? 1 : 2;  // of them from one K load
  static constexpr int kTiles = D / 16;              // output tiles
  static constexpr int kWords = kRowBytes / 64;      // dwords of a lane's part of a V row
};

// A operand of the e-th product with a K load.
template <int DT>
__device__ __forceinline__ u32x4 k_part(u32x4 raw, int e) {
  if constexpr (DT == kBF16) return raw;
  const unsigned x = raw[2 * e], y = raw[2 * e + 1];
  return u32x4{e4m3x2_to_bf16<false>(x), e4m3x2_to_bf16<true>(x), e4m3x2_to_bf16<false>(y),
               e4m3x2_to_bf16<true>(y)};
}

// Value j of a lane's part of two keys' V rows, side by side: in the dword's
// low (j even) or high half's bytes for e4m3 codes, in its halves for bf16.
template <int DT, int D>
__device__ __forceinline__ unsigned v_pair(const unsigned (&raw)[8][Shape<DT, D>::kWords], int p,
                                           int j) {
  if constexpr (DT == kFP8)
    return __builtin_amdgcn_perm(raw[2 * p + 1][j / 4], raw[2 * p][j / 4],
                                 j % 4 < 2 ? 0x05010400u : 0x07030602u);
  else
    return __builtin_amdgcn_perm(raw[2 * p + 1][j / 2], raw[2 * p][j / 2],
                                 j % 2 ? 0x07060302u : 0x05040100u);
}
template <int DT>
__device__ __forceinline__ unsigned v_bf16(unsigned m, int j) {
  if constexpr (DT == kFP8) return j % 2 ? e4m3x2_to_bf16<true>(m) : e4m3x2_to_bf16<false>(m);
  return m;
}

// A operand of output tile j: V^T of the lane's eight keys.
template <int DT, int D>
__device__ __forceinline__ u32x4 v_tile(const unsigned (&raw)[8][Shape<DT, D>::kWords], int j) {
  u32x4 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) r[p] = v_bf16<DT>(v_pair<DT, D>(raw, p, j), j);
  return r;
}

// The same with 1 in the place of +inf and NaN (sign 0), or of -inf and NaN
// (sign 1), and 0 elsewhere; e4m3 has NaN only.
template <int DT, int D>
__device__ __forceinline__ u32x4 v_marks(const unsigned (&raw)[8][Shape<DT, D>::kWords], int j,
                                         int sign) {
  u32x4 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const unsigned x = v_pair<DT, D>(raw, p, j);
    unsigned bad = not_finite<DT>(x);
    if constexpr (DT == kFP8) {
      bad &= 0x38383838u;
    } else {
      const unsigned nan = ((x & 0x7fu) ? 0xffffu : 0u) | ((x & 0x7f0000u) ? 0xffff0000u : 0u);
      const unsigned s = x & 0x80008000u;
      const unsigned neg = s | (s - (s >> 15));
      bad &= (nan | (sign ? neg : ~neg)) & 0x3f803f80u;
    }
    r[p] = v_bf16<DT>(bad, j);
  }
  return r;
}

// 1 / the sum of a row's weights.
__device__ __forceinline__ float inverse(float top, float sum) {
  if (top == kAllNegInf) return __builtin_nanf("");
  return top == kNegInf ? 0.0f : 1.0f / sum;
}

template <int DT, int D, int RT, int RW, int NW>
__global__ __launch_bounds__(64 * NW) void skinny_kv_attention_k(const AttnArgs a) {
  using Sh = Shape<DT, D>;
  constexpr int KW = NW / RW;
  constexpr int kWaveRows = 16 * RT;
  constexpr int ROWS = kWaveRows * RW;
  constexpr int kAll = 64 * NW;                      // threads
  constexpr int kStride = D + 4;                     // LDS row of the waves' sums, padded
  constexpr int kKeys = 32 * KW;                     // keys of a block
  const Cut cut{ROWS, kKeys, a.whole};
  // Keys that one wave reads come in whole 128-byte lines: lane (c, g) loads
  // 16-byte part g + 4 (c % 2) of a line of key c & ~1, then of c | 1.  Products
  // with both halves of q leave each score in two neighbouring rows, in one lane.
  // Whole lines and the nontemporal hint: 51.7 us against 53.0 with the hint on
  // half lines and 56.2 without it (131072 keys, e4m3), 99.6, 102.5 and 106.1 us
  // (16 sequences, bf16).
  constexpr bool kOnce = RW == 1 && Sh::kRowBytes >= 128;
  constexpr bool kLines = kOnce;
  __shared__ __attribute__((aligned(16))) float sums[NW][16][kStride];
  __shared__ float sm[NW][16], sl[NW][16];
  const KvArgs& kv = a.kv;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int rw = wave % RW, kw = wave / RW;
  const int c = lane & 15, g = lane >> 4;
  const int P = 1 << kv.log2p;
  const int q_heads = kv.kv_heads * kv.group;

  const Work work = all_work(kv, cut);
  const Shares shares(work.total, a.groups);
  int pos = shares.begin(blockIdx.x);
  const int end = shares.begin(blockIdx.x + 1);
  Split split{};

  while (pos < end) {
    const Place pl = place_of(kv, cut, work, pos);
    const int h = pl.rgs == 1 ? pl.item : pl.item / pl.rgs, rg = pl.item - h * pl.rgs;
    const Seq q = pl.q;
    const int steps = min(pl.nb - pl.blk, end - pos);
    const bool whole = steps == pl.nb;
    // 32-key tiles of each wave.
    const int blocks = a.whole ? (q.cap + kKeys - 1) / kKeys : steps;
    const int row_count = min(q.n * kv.group - rg * ROWS, ROWS);
    // This wave's rows, and the keys seen by the first and the last of them.
    const int row0 = rg * ROWS + rw * kWaveRows;
    const int wave_rows = min(row_count - rw * kWaveRows, kWaveRows);
    const int lim_lo = min(max(q.base + by_group(kv, row0) + 1, 0), q.cap);
    const int lim_hi = wave_rows <= 0 ? 0
        : min(max(q.base + by_group(kv, row0 + wave_rows - 1) + 1, 0), q.cap);

    // Row rt * 16 + c of the wave's rows in this lane's column.
    u32x4 qf[RT][Sh::kSteps];
    int lim[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = row0 + rt * 16 + c;
      const int tok = by_group(kv, r), head = r - tok * kv.group;
      const bool live = rt * 16 + c < wave_rows;
      lim[rt] = live ? min(max(q.base + tok + 1, 0), q.cap) : lim_hi;
      const __bf16* src = a.q + ((size_t)(q.q0 + tok) * q_heads + h * kv.group + head) * D;
#pragma unroll
      for (int st = 0; st < Sh::kSteps; ++st) {
        // The 8 values of the product's k index that this lane's K load holds.
        const int d = DT == kBF16 ? 32 * st + 8 * g : 64 * (st / 2) + 16 * g + 8 * (st % 2);
        qf[rt][st] = live ? *reinterpret_cast<const u32x4*>(src + d) : u32x4{0, 0, 0, 0};
      }
    }

    f32x4 o[RT][Sh::kTiles];
    float m[RT], l[RT];

    // This wave's keys: as many tiles of 32 as the segment has blocks.
    const int key0 = (pl.blk * KW + kw * blocks) * 32;
    const int tiles = min(max((lim_hi - key0 + 31) / 32, 0), blocks);
    const int* table = kv.table + (size_t)pl.s * kv.max_pages;
    const int last_page = max(q.cap - 1, 0) >> kv.log2p;
    int window = -1;                                 // first page whose number the lanes hold
    int w_page = -1;
    float w_ks = 0.0f, w_vs = 0.0f;
    const size_t page_bytes = (size_t)kv.kv_heads * P * Sh::kRowBytes;

    // Page number and scales of the page that holds `key`, from the lanes.
    const auto look = [&](int key) {
      if (window < 0 || (key >> kv.log2p) < window || ((key + 16) >> kv.log2p) >= window + 64) {
        window = key >> kv.log2p;
        w_page = table[min(window + lane, last_page)];
        const bool good = w_page >= 0 && w_page < kv.pages;
        w_page = good ? w_page : -1;
        if constexpr (DT == kFP8) {
          const size_t at = (size_t)max(w_page, 0) * kv.kv_heads + h;
          w_ks = good ? kv.k_scale[at] : 0.0f;
          w_vs = good ? kv.v_scale[at] : 0.0f;
        }
      }
    };
    // A tile's two halves of 16 keys: where they lie, and the lane that has
    // their page's scales.
    struct Half {
      size_t off;
      int at;
      bool there;
    };
    const auto half_of = [&](int key) {
      Half x;
      x.at = (key >> kv.log2p) - window;
      const int page = lane_of(w_page, x.at);
      x.there = page >= 0;
      x.off = (size_t)max(page, 0) * page_bytes + (size_t)(h * P + (key & (P - 1))) * Sh::kRowBytes;
      return x;
    };
    u32x4 kf[2][Sh::kLoads];
    unsigned vf[8][Sh::kWords];
    const auto load_k = [&](const Half (&at)[2]) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (kLines) {
          const unsigned char* kp =
              kv.k + at[u].off + (c & ~1) * Sh::kRowBytes + (g + 4 * (c & 1)) * 16;
#pragma unroll
          for (int i = 0; i < Sh::kLoads; ++i)
            kf[u][i] = load_as<kOnce, u32x4>(kp + Sh::kRowBytes * (i % 2) + 128 * (i / 2));
        } else {
          const unsigned char* kp = kv.k + at[u].off + c * Sh::kRowBytes + g * 16;
#pragma unroll
          for (int i = 0; i < Sh::kLoads; ++i) kf[u][i] = load_as<kOnce, u32x4>(kp + 64 * i);
        }
      }
    };
    const auto load_v = [&](const Half (&at)[2]) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const unsigned char* vp = kv.v + at[u].off + 4 * g * Sh::kRowBytes + c * (4 * Sh::kWords);
#pragma unroll
        for (int r = 0; r < 4; ++r) load_words<kOnce, Sh::kWords>(vp + r * Sh::kRowBytes, vf[4 * u + r]);
      }
    };

    // The next tile's keys load behind this tile's scores, its values behind
    // this tile's output; the last tile loads itself once more.
    //   Values that are no finite numbers leave the products, and come back behind
    // the loop for the rows that see their keys: in tiles with a mask, where 0 * inf
    // and 0 * NaN would reach rows that do not, and, once sums have turned out not
    // to be finite, in a second run over all tiles, where a probability that
    // vanishes in fp32 would make a NaN of an infinity.
    Half now[2];
    bool dirty = false;                              // such values were found
    const auto run = [&](auto clean) {               // whether this is the second run
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        m[rt] = kNegInf;
        l[rt] = 0.0f;
#pragma unroll
        for (int j = 0; j < Sh::kTiles; ++j) o[rt][j] = f32x4{0, 0, 0, 0};
      }
      if (tiles <= 0) return;
      look(key0);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int st = 0; st < Sh::kSteps; ++st) arrived(qf[rt][st]);
      now[0] = half_of(key0);
      now[1] = half_of(key0 + 16);
      load_k(now);
      load_v(now);
      int t = 0;
      do {
        const int key = key0 + 32 * t;
        const bool there[2] = {now[0].there, now[1].there};
        const bool good = there[0] && there[1];
        const bool masked = !good || key + 32 > lim_lo;   // some row does not see some key

        u32x4 pf[RT], pr[RT];                        // p in bf16, and what that leaves of it
        f32x4 sc[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if constexpr (kLines) {
              f32x4 lo[2]{}, hi[2]{};                // even and odd keys
#pragma unroll
              for (int i = 0; i < Sh::kLoads; ++i)
#pragma unroll
                for (int e = 0; e < Sh::kPart; ++e) {
                  const u32x4 kk = k_part<DT>(kf[u][i], e);
                  const int st = 2 * Sh::kPart * (i / 2) + e;
                  lo[i % 2] = mfma_bf16(kk, qf[rt][st], lo[i % 2]);
                  hi[i % 2] = mfma_bf16(kk, qf[rt][st + Sh::kPart], hi[i % 2]);
                }
              settle(lo, hi);
              sc[rt][u] = f32x4{lo[0][0] + hi[0][1], lo[1][0] + hi[1][1], lo[0][2] + hi[0][3],
                                lo[1][2] + hi[1][3]};
            } else {
              f32x4 s{0, 0, 0, 0};
#pragma unroll
              for (int st = 0; st < Sh::kSteps; ++st)
                s = mfma_bf16(k_part<DT>(kf[u][st / Sh::kPart], st % Sh::kPart), qf[rt][st], s);
              sc[rt][u] = s;
            }
          }
        settle(sc);
        float ks[2], vs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          ks[u] = DT == kFP8 ? a.scale * lane_of(w_ks, now[u].at) : a.scale;
          vs[u] = DT == kFP8 ? lane_of(w_vs, now[u].at) : 1.0f;
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            sc[rt][u] *= ks[u];
            if (masked) {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (!there[u] || key + 16 * u + 4 * g + r >= lim[rt]) sc[rt][u][r] = kNegInf;
            }
          }
        const int next = key0 + 32 * min(t + 1, tiles - 1);
        look(next);
        now[0] = half_of(next);
        now[1] = half_of(next + 16);
        load_k(now);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          float top = m[rt];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, sc[rt][u][r]);
          top = row_max(top);
          if (__any(top > m[rt] + kSlack)) {
            const float f = top > m[rt] ? __builtin_amdgcn_exp2f(m[rt] - top) : 1.0f;
            l[rt] *= f;
#pragma unroll
            for (int j = 0; j < Sh::kTiles; ++j) o[rt][j] *= f;
            m[rt] = fmaxf(m[rt], top);
          }
          const float ref = m[rt] == kNegInf ? 0.0f : m[rt];
          float p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(sc[rt][i / 4][i % 4] - ref);
            l[rt] += p[i];
            if constexpr (DT == kFP8) p[i] *= vs[i / 4];
          }
          if (masked) {
            // A key that the row does not see takes no part, whatever its page's scale holds.
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (!there[i / 4] || key + 16 * (i / 4) + 4 * g + i % 4 >= lim[rt]) p[i] = 0.0f;
          }
          // A probability is the sum of two bf16 numbers, within 2^-16 of itself; one
          // alone, within 2^-8, is the largest error of the whole operator (up to
          // 31 times what the other sums leave).  The second products cost where rows
          // bound a call: 35.4 to 38.7 us on two sequences of 12 verified tokens
          // between them, 7.8 to 8.2 on short ones of 64; nothing where keys do.
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            pf[rt][i] = pack_bf16(p[2 * i], p[2 * i + 1]);
            float lo = p[2 * i] - bf16_lo(pf[rt][i]), hi = p[2 * i + 1] - bf16_hi(pf[rt][i]);
            if constexpr (clean.value) {             // (a page's scale that is no finite number)
              lo = lo - lo == 0.0f ? lo : 0.0f;
              hi = hi - hi == 0.0f ? hi : 0.0f;
            }
            pr[rt][i] = pack_bf16(lo, hi);
          }
        }
        if (clean.value || masked) {
          unsigned any = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int w = 0; w < Sh::kWords; ++w) any |= not_finite<DT>(vf[i][w]);
          if (__any(any != 0)) {
            dirty = true;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int w = 0; w < Sh::kWords; ++w) vf[i][w] &= ~not_finite<DT>(vf[i][w]);
          }
        }
#pragma unroll
        for (int j = 0; j < Sh::kTiles; ++j) {
          const u32x4 vt = v_tile<DT, D>(vf, j);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) o[rt][j] = mfma_bf16(vt, pf[rt], o[rt][j]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) o[rt][j] = mfma_bf16(vt, pr[rt], o[rt][j]);
        }
        load_v(now);
      } while (++t < tiles);
      settle(o);
    };
    run(std::false_type{});
    // 0 as long as every sum is finite; one chain per register of a tile.
    f32x4 zero{0, 0, 0, 0};
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < Sh::kTiles; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) zero[r] = fmaf(o[rt][j][r], 0.0f, zero[r]);
    const bool clean = __any((zero[0] + zero[1]) + (zero[2] + zero[3]) != 0.0f);
    if (__builtin_expect(clean, 0)) run(std::true_type{});

    for (int t = dirty ? 0 : tiles; t < tiles; ++t) {
      const int key = key0 + 32 * t;
      look(key);
      now[0] = half_of(key);
      now[1] = half_of(key + 16);
      if (!clean && now[0].there && now[1].there && key + 32 <= lim_lo) continue;
      load_v(now);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        u32x4 seen{0, 0, 0, 0};                      // 1 where the row sees the key
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (now[x / 4].there && key + 16 * (x / 4) + 4 * g + x % 4 < lim[rt])
            seen[x / 2] |= 0x3f80u << (16 * (x % 2));
#pragma unroll
        for (int sign = 0; sign < (DT == kBF16 ? 2 : 1); ++sign)
#pragma unroll
          for (int j = 0; j < Sh::kTiles; ++j) {
            f32x4 hits = mfma_bf16(v_marks<DT, D>(vf, j, sign), seen, f32x4{0, 0, 0, 0});
            settle(hits);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (hits[r] > 0.0f)
                o[rt][j][r] += DT == kFP8 ? __builtin_nanf("") : (sign ? kNegInf : -kNegInf);
          }
      }
    }

    bool none = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) none = none || (m[rt] == kNegInf && key0 < lim[rt]);
    for (int t = __any(none) ? 0 : tiles; t < tiles; ++t) {
      const int key = key0 + 32 * t;
      look(key);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool there = half_of(key + 16 * u).there;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          if (there && key + 16 * u < lim[rt] && m[rt] == kNegInf) m[rt] = kAllNegInf;
      }
    }

    // The waves' sums, 16 rows of each row wave at a time.
    float* part = a.part + (size_t)(2 * blockIdx.x + (pl.blk == 0 ? 1 : 0)) * part_floats<D>(ROWS);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float lw = row_sum(l[rt]);
      if (g == 0) {
        sm[wave][c] = m[rt];
        sl[wave][c] = lw;
      }
      // Lane (c, g), tile j, register r holds value (4g + r) D/16 + j of row c.
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < Sh::kTiles; ++j)
          sums[wave][c][(4 * g + r) * Sh::kTiles + j] = o[rt][j][r];
      __syncthreads();
      for (int i = tid; i < 16 * RW * (D / 4); i += kAll) {
        const int d = i % (D / 4) * 4, rr = i / (D / 4) % 16, w0 = i / (D / 4) / 16;
        const int row = w0 * kWaveRows + rt * 16 + rr;
        if (row < row_count) {
          float top = kNegInf;
#pragma unroll
          for (int w = 0; w < KW; ++w) top = fmaxf(top, sm[w * RW + w0][rr]);
          float sum = 0.0f;
          f32x4 x{0, 0, 0, 0};
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            const float mw = sm[w * RW + w0][rr], lw2 = sl[w * RW + w0][rr];
            const float f = mw == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mw - top);
            sum += f * lw2;
            x += f * *reinterpret_cast<const f32x4*>(&sums[w * RW + w0][rr][d]);
          }
          if (whole) {
            const float inv = inverse(top, sum);
            const int r = rg * ROWS + row, tok = by_group(kv, r), head = r - tok * kv.group;
            *reinterpret_cast<u32x2*>(a.out +
                ((size_t)(q.q0 + tok) * q_heads + h * kv.group + head) * D + d) =
                u32x2{pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv)};
          } else {
            *reinterpret_cast<f32x4*>(part + row * D + d) = x;
            if (d == 0) {
              part[ROWS * D + row] = top;
              part[ROWS * D + ROWS + row] = sum;
            }
          }
        }
      }
      __syncthreads();
    }
    if (pl.blk == 0 && !whole)
      split = Split{shares.of(pos + pl.nb - 1) - (int)blockIdx.x + 1, row_count, rg * ROWS, q.q0, h};
    pos += steps;
  }
  if (tid == 0) a.splits[blockIdx.x] = split;
}

// Joins the segments of the item that goes on from share blockIdx.x, kJoinRows<D>
// of its rows from blockIdx.y on: per row D / 4 lanes (4 values each) in kJoinSets
// sets that take every kJoinSets-th segment, kJoinAhead of them in flight, with
// the running maximum and sum of a softmax; the sets' results are then added in
// order.
constexpr int kJoinThreads = 512;
constexpr int kJoinSets = 4;
constexpr int kJoinAhead = 8;
template <int D>
constexpr int kJoinRows = kJoinThreads / (kJoinSets * (D / 4));
template <int D>
__global__ __launch_bounds__(kJoinThreads) void skinny_kv_attention_join(const AttnArgs a, int rows) {
  constexpr int kLanes = D / 4;
  __shared__ f32x4 sx[kJoinSets][kJoinRows<D>][kLanes];
  __shared__ float st[kJoinSets][kJoinRows<D>], sl[kJoinSets][kJoinRows<D>];
  const Split sp = a.splits[blockIdx.x];
  if (sp.n == 0 || blockIdx.y * kJoinRows<D> >= sp.rows) return;
  const int n = sp.n;
  const int d = threadIdx.x % kLanes, set = threadIdx.x / kLanes % kJoinSets;
  const int slot = threadIdx.x / (kLanes * kJoinSets);
  const int row = blockIdx.y * kJoinRows<D> + slot;
  const int from = min(row, sp.rows - 1);
  // Segment k is share blockIdx.x + k's; the item's first one stands second in
  // its share's pair.
  const size_t stride = part_floats<D>(rows);
  const float* part = a.part + (size_t)(2 * blockIdx.x) * stride;
  float top = kNegInf, sum = 0.0f;
  f32x4 x{0, 0, 0, 0};
  for (int k0 = set; k0 < n; k0 += kJoinSets * kJoinAhead) {
    float mk[kJoinAhead], lk[kJoinAhead];
    f32x4 y[kJoinAhead];
#pragma unroll
    for (int e = 0; e < kJoinAhead; ++e) {
      const int k = min(k0 + e * kJoinSets, n - 1);
      const float* s = part + (size_t)(2 * k + (k == 0 ? 1 : 0)) * stride;
      mk[e] = s[rows * D + from];
      lk[e] = s[rows * D + rows + from];
      y[e] = *reinterpret_cast<const f32x4*>(s + from * D + 4 * d);
    }
    float next = top;
#pragma unroll
    for (int e = 0; e < kJoinAhead; ++e) next = fmaxf(next, mk[e]);
    const float f0 = top == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(top - next);
    sum *= f0;
    x *= f0;
    top = next;
#pragma unroll
    for (int e = 0; e < kJoinAhead; ++e)
      if (k0 + e * kJoinSets < n) {
        const float f = mk[e] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mk[e] - top);
        sum += f * lk[e];
        x += f * y[e];
      }
  }
  sx[set][slot][d] = x;
  if (d == 0) {
    st[set][slot] = top;
    sl[set][slot] = sum;
  }
  __syncthreads();
  if (set != 0 || row >= sp.rows) return;
#pragma unroll
  for (int k = 1; k < kJoinSets; ++k) top = fmaxf(top, st[k][slot]);
  sum = 0.0f;
  x = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < kJoinSets; ++k) {
    const float tk = st[k][slot], lk = sl[k][slot];
    const float f = tk == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(tk - top);
    sum += f * lk;
    x += f * sx[k][slot][d];
  }
  const float inv = inverse(top, sum);
  const int group = a.kv.group, r = sp.row0 + row;
  *reinterpret_cast<u32x2*>(a.out + ((size_t)(sp.q0 + r / group) * a.kv.kv_heads * group +
                                     sp.h * group + r % group) * D + 4 * d) =
      u32x2{pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv)};
}

// ---------------------------------------------------------------------------
// Host side.

using Kernel = void (*)(AppendArgs);
template <int DT, bool INTERLEAVED>
Kernel append_many_as(int passes) {
  return passes <= 1   ? skinny_kv_append_many<DT, INTERLEAVED, 1>
         : passes <= 2 ? skinny_kv_append_many<DT, INTERLEAVED, 2>
         : passes <= 4 ? skinny_kv_append_many<DT, INTERLEAVED, 4>
                       : skinny_kv_append_many<DT, INTERLEAVED, 8>;
}
template <int DT>
Kernel append_many(int passes, bool interleaved) {
  return interleaved ? append_many_as<DT, true>(passes) : append_many_as<DT, false>(passes);
}

// Steps that skinny_kv_append_few takes: as many rows, their e4m3 pages' values
// within that much LDS.  Measured on MI355X with 64 + 2 x 8 heads of 128, few
// against many: 4.3 / 7.8 us at 1 row, 7.1 / 8.7 at 32, 8.9 / 9.2 at 64, 10.9 /
// 9.9 at 128, 21.9 / 15.7 at 1024.
constexpr int kFewRows = 64;
constexpr size_t kFewLds = 32 * 1024;

size_t pool_elems(const skinny_kv_cache& c) {
  return (size_t)c.pages * c.kv_heads * c.page_tokens * c.head_dim;
}

skinny_status check_cache(const skinny_kv_cache* c) {
  if (!c || c->reserved != 0) return SKINNY_ERR_INVALID_ARG;
  if (c->dtype != SKINNY_KV_BF16 && c->dtype != SKINNY_KV_FP8) return SKINNY_ERR_INVALID_ARG;
  if (c->pages < 1 || c->kv_heads < 1 || c->page_tokens < 1 || c->head_dim < 1)
    return SKINNY_ERR_INVALID_ARG;
  if (!c->k || !c->v) return SKINNY_ERR_INVALID_ARG;
  const bool fp8 = c->dtype == SKINNY_KV_FP8;
  if (fp8 != (c->k_scale != nullptr) || fp8 != (c->v_scale != nullptr))
    return SKINNY_ERR_INVALID_ARG;
  if (c->page_tokens < SKINNY_KV_MIN_PAGE || c->page_tokens > SKINNY_KV_MAX_PAGE ||
      (c->page_tokens & (c->page_tokens - 1)))
    return SKINNY_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return SKINNY_ERR_UNSUPPORTED;
  if (c->kv_heads > SKINNY_KV_MAX_HEADS) return SKINNY_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SKINNY_ERR_UNSUPPORTED;
  if (fp8 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))) return SKINNY_ERR_UNSUPPORTED;
  return SKINNY_OK;
}

skinny_status check_batch(const skinny_kv_cache& c, const skinny_kv_batch* b) {
  if (!b || b->reserved != 0) return SKINNY_ERR_INVALID_ARG;
  if (b->seqs < 1 || b->tokens < 1 || b->max_pages < 1) return SKINNY_ERR_INVALID_ARG;
  if (!b->q_start || !b->kv_len || !b->page_table) return SKINNY_ERR_INVALID_ARG;
  if (b->seqs > SKINNY_KV_MAX_SEQS || b->tokens > SKINNY_KV_MAX_TOKENS)
    return SKINNY_ERR_UNSUPPORTED;
  if ((long long)b->max_pages * c.page_tokens > kMaxPosition) return SKINNY_ERR_UNSUPPORTED;
  if (!aligned(b->q_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->page_table, 4))
    return SKINNY_ERR_UNSUPPORTED;
  return SKINNY_OK;
}

// A written buffer against everything else of the call.
constexpr int kSharedRanges = 7;
void shared_ranges(const skinny_kv_cache& c, const skinny_kv_batch& b, Range (&r)[kSharedRanges]) {
  const size_t bytes = pool_elems(c) * (c.dtype == SKINNY_KV_BF16 ? 2 : 1);
  const size_t sb = c.k_scale ? (size_t)c.pages * c.kv_heads * 4 : 0;
  r[0] = range_of(c.k, bytes);
  r[1] = range_of(c.v, bytes);
  r[2] = range_of(c.k_scale, sb);
  r[3] = range_of(c.v_scale, sb);
  r[4] = range_of(b.q_start, (size_t)(b.seqs + 1) * 4);
  r[5] = range_of(b.kv_len, (size_t)b.seqs * 4);
  r[6] = range_of(b.page_table, (size_t)b.seqs * b.max_pages * 4);
}

bool meets(Range w, const Range* r, int n) {
  for (int i = 0; i < n; ++i)
    if (r[i].lo != r[i].hi && overlap(w, r[i])) return true;
  return false;
}

int log2_of(int p) {
  int l = 0;
  while ((1 << l) < p) ++l;
  return l;
}

KvArgs kv_args(const skinny_kv_cache& c, const skinny_kv_batch& b, int group) {
  KvArgs a;
  a.k = (unsigned char*)c.k;
  a.v = (unsigned char*)c.v;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.q_start = b.q_start;
  a.kv_len = b.kv_len;
  a.table = b.page_table;
  a.S = b.seqs;
  a.T = b.tokens;
  a.max_pages = b.max_pages;
  a.pages = c.pages;
  a.kv_heads = c.kv_heads;
  a.group = group;
  a.group_shift = group & (group - 1) ? -1 : log2_of(group);
  a.log2p = log2_of(c.page_tokens);
  return a;
}

skinny_status check_heads(const skinny_kv_cache& c, int q_heads) {
  if (q_heads < 1 || q_heads % c.kv_heads != 0) return SKINNY_ERR_INVALID_ARG;
  if (q_heads > SKINNY_KV_MAX_HEADS) return SKINNY_ERR_UNSUPPORTED;
  return SKINNY_OK;
}

// How a launch cuts an item's rows: RT tiles of 16 rows per wave, RW row waves
// of the workgroup's NW.  RT is what fits beside a tile of keys and values in
// the registers of two waves per SIMD (one at head_dim 256, whose workgroups
// have four waves); RW grows with the rows of an average sequence under one KV
// head.
struct RowCut {
  int rt, rw;
};
constexpr int most_row_tiles(int dtype, int head_dim) {
  return head_dim == 64 || (head_dim == 128 && dtype == SKINNY_KV_FP8) ? 2 : 1;
}
constexpr int waves_of(int head_dim) { return head_dim == 256 ? 4 : 8; }
RowCut row_cut(const skinny_kv_cache& c, const skinny_kv_batch& b, int q_heads) {
  const long long tokens = (b.tokens + b.seqs - 1) / b.seqs;
  const long long rows = tokens * (q_heads / c.kv_heads);
  RowCut r{1, 1};
  if (rows <= 16) return r;
  r.rt = most_row_tiles(c.dtype, c.head_dim);
  const int most = 8 / r.rt < waves_of(c.head_dim) ? 8 / r.rt : waves_of(c.head_dim);
  while (r.rw < most && 16 * r.rt * r.rw < rows) r.rw *= 2;
  return r;
}

// Items (row groups under each KV head) of all sequences at most.
long long max_items(const skinny_kv_cache& c, const skinny_kv_batch& b, int q_heads, RowCut r) {
  const long long rows = (long long)b.tokens * (q_heads / c.kv_heads);
  const long long g = rows / (16 * r.rt * r.rw) + (b.seqs < b.tokens ? b.seqs : b.tokens);
  return (g < rows ? g : rows) * c.kv_heads;
}

// Blocks of all items at most: every sequence at the page table's length.
long long max_work(const skinny_kv_cache& c, const skinny_kv_batch& b, int q_heads, RowCut r) {
  const long long keys = (long long)b.max_pages * c.page_tokens;
  const long long block = 32 * (waves_of(c.head_dim) / r.rw);
  return max_items(c, b, q_heads, r) * ((keys + block - 1) / block);
}

size_t attention_workspace(const skinny_kv_cache& c, const skinny_kv_batch& b, int q_heads) {
  const RowCut r = row_cut(c, b, q_heads);
  const long long w = max_work(c, b, q_heads, r);
  if (w >= kMaxCount) return 0;                      // more blocks than the kernels count
  const long long groups = w < kMaxGroups ? w : kMaxGroups;
  return kSplitBytes + (size_t)(2 * groups) * (16 * r.rt * r.rw) * (c.head_dim + 2) * sizeof(float);
}

// Whether a call's items stay whole, one workgroup each and no second launch: at
// most four tiles and 32 KB of keys and values per wave by the page table's
// width, and no more items than workgroups (or one tile, which has no parts).
// Whole against split, us: e4m3, 5 sequences, 32 heads on 8 of 64: 6.2 / 7.7 at
// 256 keys, 8.4 / 9.5 at 777, 10.3 / 9.8 at 1500 (6 tiles: split), 12.1 / 9.7 at
// 2048; bf16, 16 sequences, 64 on 8 of 128: 8.7 / 10.4 at 256, 11.4 / 12.4 at 512,
// 13.6 / 12.7 at 777 (split); 48 such sequences, 384 items: 15.1 / 16.7 at 256 (one
// tile), 19.8 / 17.9 at 512 (split).
constexpr int kWholeTiles = 4;
constexpr int kWholeBytes = 32 * 1024;
bool stays_whole(const skinny_kv_cache& c, const skinny_kv_batch& b, RowCut r, long long items,
                 long long groups) {
  const long long keys = (long long)b.max_pages * c.page_tokens;
  const int block = 32 * (waves_of(c.head_dim) / r.rw);
  const long long tiles = (keys + block - 1) / block;
  const int bytes = 32 * 2 * c.head_dim * (c.dtype == SKINNY_KV_BF16 ? 2 : 1);
  return tiles <= kWholeTiles && tiles * bytes <= kWholeBytes && (tiles == 1 || items <= groups);
}

template <int DT, int D, int RT, int RW>
skinny_status launch_attention(const AttnArgs& a, int rows, hipStream_t stream) {
  constexpr int NW = waves_of(D);
  constexpr int ROWS = 16 * RT * RW;
  hipLaunchKernelGGL((skinny_kv_attention_k<DT, D, RT, RW, NW>), dim3(a.groups), dim3(64 * NW), 0,
                     stream, a);
  if (hipGetLastError() != hipSuccess) return SKINNY_ERR_HIP;
  if (a.groups == 1 || a.whole) return SKINNY_OK;    // nothing is split
  if (rows > ROWS) rows = ROWS;
  hipLaunchKernelGGL((skinny_kv_attention_join<D>),
                     dim3(a.groups - 1, (rows + kJoinRows<D> - 1) / kJoinRows<D>),
                     dim3(kJoinThreads), 0, stream, a, ROWS);
  return hipGetLastError() == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP;
}

template <int DT, int D>
skinny_status launch_rows(const AttnArgs& a, RowCut r, int rows, hipStream_t stream) {
  constexpr int RT = most_row_tiles(DT, D);
  if (r.rt == 1 && r.rw == 1) return launch_attention<DT, D, 1, 1>(a, rows, stream);
  if (r.rw == 2) return launch_attention<DT, D, RT, 2>(a, rows, stream);
  if (r.rw == 4) return launch_attention<DT, D, RT, 4>(a, rows, stream);
  if constexpr (RT == 2) return launch_attention<DT, D, 2, 1>(a, rows, stream);
  if constexpr (RT == 1 && waves_of(D) == 8) return launch_attention<DT, D, 1, 8>(a, rows, stream);
  return SKINNY_ERR_UNSUPPORTED;
}

template <int DT>
skinny_status launch_dim(const AttnArgs& a, int d, RowCut r, int rows, hipStream_t stream) {
  if (d == 64) return launch_rows<DT, 64>(a, r, rows, stream);
  if (d == 128) return launch_rows<DT, 128>(a, r, rows, stream);
  return launch_rows<DT, 256>(a, r, rows, stream);
}

}  // namespace

extern "C" {

skinny_status skinny_kv_append(const skinny_kv_cache* cache, const skinny_kv_batch* batch,
                               const void* qkv, int q_heads, const float* inv_freq,
                               int rotary_dim, int interleaved, void* q_out, void* stream) {
  skinny_status st = check_cache(cache);
  if (st == SKINNY_OK) st = check_batch(*cache, batch);
  if (st == SKINNY_OK) st = check_heads(*cache, q_heads);
  if (st != SKINNY_OK) return st;
  const skinny_kv_cache& c = *cache;
  const skinny_kv_batch& b = *batch;
  if (!qkv || !q_out) return SKINNY_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > c.head_dim || (rotary_dim > 0) != (inv_freq != nullptr) ||
      (interleaved != 0 && interleaved != 1))
    return SKINNY_ERR_INVALID_ARG;
  if (rotary_dim % kUnit != 0) return SKINNY_ERR_UNSUPPORTED;
  if (!aligned(qkv, 16) || !aligned(q_out, 16) || (inv_freq && !aligned(inv_freq, 4)))
    return SKINNY_ERR_UNSUPPORTED;
  const size_t width = (size_t)(q_heads + 2 * c.kv_heads) * c.head_dim;
  const Range xr = range_of(qkv, b.tokens * width * 2);
  const Range fr = range_of(inv_freq, (size_t)rotary_dim / 2 * 4);
  const Range qr = range_of(q_out, (size_t)b.tokens * q_heads * c.head_dim * 2);
  Range sh[kSharedRanges + 2];
  Range base[kSharedRanges];
  shared_ranges(c, b, base);
  for (int i = 0; i < kSharedRanges; ++i) sh[i] = base[i];
  sh[kSharedRanges] = xr;
  sh[kSharedRanges + 1] = fr;
  if (meets(qr, sh, kSharedRanges + 2)) return SKINNY_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)                       // the pools and scales are written too
    if (sh[i].lo != sh[i].hi && meets(sh[i], sh + i + 1, kSharedRanges + 1 - i))
      return SKINNY_ERR_INVALID_ARG;
  const bool fp8 = c.dtype == SKINNY_KV_FP8;
  const int most = b.tokens < c.page_tokens ? b.tokens : c.page_tokens;   // rows of a page
  const size_t rows = fp8 ? (size_t)most * c.head_dim * 4 : 0;
  const bool few = b.tokens <= kFewRows && rows <= kFewLds;
  // n rows of a sequence fall into at most n pages, and at most (n - 2) / P + 2.
  const long long seqs = b.seqs < b.tokens ? b.seqs : b.tokens;
  long long units = b.tokens / c.page_tokens + 2 * seqs;
  if (units > b.tokens) units = b.tokens;
  const long long kvb = units * c.kv_heads * 2;
  const long long qb = few
      ? (long long)b.tokens * ((q_heads + kQHeadsPerBlock - 1) / kQHeadsPerBlock)
      : (b.tokens + kQRows - 1) / kQRows;
  if ((kvb + qb) * kThreads > 0xffffffffLL) return SKINNY_ERR_UNSUPPORTED;   // threads of a launch
  DeviceInfo d;
  st = device_info(&d);
  if (st != SKINNY_OK) return st;
  if (!d.gfx950) return SKINNY_ERR_UNSUPPORTED;

  AppendArgs a;
  a.kv = kv_args(c, b, q_heads / c.kv_heads);
  a.qkv = (const __bf16*)qkv;
  a.q_out = (__bf16*)q_out;
  a.inv_freq = inv_freq;
  a.q_heads = q_heads;
  a.head_dim = c.head_dim;
  a.rot = rotary_dim;
  a.interleaved = interleaved;
  a.kv_blocks = (int)kvb;
  const dim3 all((unsigned)(kvb + qb)), threads(kThreads);
  const hipStream_t hs = (hipStream_t)stream;
  if (few) {
    const size_t turns = (size_t)rotary_dim * 8;    // cos and sin in fp64
    const size_t lds = rows > turns ? rows : turns;
    if (fp8) hipLaunchKernelGGL(skinny_kv_append_few<kFP8>, all, threads, lds, hs, a);
    else hipLaunchKernelGGL(skinny_kv_append_few<kBF16>, all, threads, lds, hs, a);
    return hipGetLastError() == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP;
  }
  const int step = kThreads * kUnit / c.head_dim;   // rows of a pass
  const int passes = (most + step - 1) / step;      // at most 8
  const Kernel fn = fp8 ? append_many<kFP8>(passes, interleaved) : append_many<kBF16>(passes, interleaved);
  const size_t lds = (size_t)(step > kQRows ? step : kQRows) * rotary_dim * 8;   // cos and sin in fp64
  hipLaunchKernelGGL(fn, all, threads, lds, hs, a);
  return hipGetLastError() == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP;
}

size_t skinny_kv_attention_workspace_bytes(const skinny_kv_cache* cache,
                                           const skinny_kv_batch* batch, int q_heads) {
  if (check_cache(cache) != SKINNY_OK || check_batch(*cache, batch) != SKINNY_OK ||
      check_heads(*cache, q_heads) != SKINNY_OK)
    return 0;
  const size_t b = attention_workspace(*cache, *batch, q_heads);
  if (b == 0) return 0;
  return b > SKINNY_MIN_WORKSPACE_BYTES ? b : SKINNY_MIN_WORKSPACE_BYTES;
}

skinny_status skinny_kv_attention(const skinny_kv_cache* cache, const skinny_kv_batch* batch,
                                  const void* q, int q_heads, float scale, void* out,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  skinny_status st = check_cache(cache);
  if (st == SKINNY_OK) st = check_batch(*cache, batch);
  if (st == SKINNY_OK) st = check_heads(*cache, q_heads);
  if (st != SKINNY_OK) return st;
  const skinny_kv_cache& c = *cache;
  const skinny_kv_batch& b = *batch;
  const float log2_scale = scale * 1.44269504088896340736f;   // the kernel's softmax is in exp2
  if (!q || !out || !(log2_scale - log2_scale == 0.0f)) return SKINNY_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16)) return SKINNY_ERR_UNSUPPORTED;
  const RowCut r = row_cut(c, b, q_heads);
  const long long work = max_work(c, b, q_heads, r);
  if (work >= kMaxCount) return SKINNY_ERR_UNSUPPORTED;
  if (!workspace ||
      workspace_bytes < skinny_kv_attention_workspace_bytes(cache, batch, q_heads))
    return SKINNY_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SKINNY_ERR_UNSUPPORTED;
  const size_t row_bytes = (size_t)b.tokens * q_heads * c.head_dim * 2;
  const Range qr = range_of(q, row_bytes), yr = range_of(out, row_bytes);
  const Range wr = range_of(workspace, workspace_bytes);
  Range sh[kSharedRanges];
  shared_ranges(c, b, sh);
  if (overlap(yr, qr) || overlap(yr, wr) || overlap(wr, qr) || meets(yr, sh, kSharedRanges) ||
      meets(wr, sh, kSharedRanges))
    return SKINNY_ERR_INVALID_ARG;
  DeviceInfo d;
  st = device_info(&d);
  if (st != SKINNY_OK) return st;
  if (!d.gfx950) return SKINNY_ERR_UNSUPPORTED;

  AttnArgs a;
  a.kv = kv_args(c, b, q_heads / c.kv_heads);
  a.q = (const __bf16*)q;
  a.out = (__bf16*)out;
  a.splits = (Split*)workspace;
  a.part = (float*)((unsigned char*)workspace + kSplitBytes);
  a.scale = log2_scale;
  long long groups = d.cus < kMaxGroups ? d.cus : kMaxGroups;
  const long long items = max_items(c, b, q_heads, r);
  a.whole = stays_whole(c, b, r, items, groups);
  const long long parts = a.whole ? items : work;
  if (groups > parts) groups = parts;
  a.groups = (int)groups;
  const long long rows = (long long)b.tokens * (q_heads / c.kv_heads);
  const int most = rows < 128 ? (int)rows : 128;     // rows of an item at most
  if (c.dtype == SKINNY_KV_FP8)
    return launch_dim<kFP8>(a, c.head_dim, r, most, (hipStream_t)stream);
  return launch_dim<kBF16>(a, c.head_dim, r, most, (hipStream_t)stream);
}

}  // extern "C"
