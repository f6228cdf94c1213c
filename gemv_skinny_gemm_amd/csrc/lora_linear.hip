// lora_linear.hip - low-rank adapters of many requests beside a shared projection
// (skinny_lora_linear), on MI355X (gfx950).

#include <hip/hip_runtime.h>

#include "host_util.h"
#include "skinny_gemm.h"

namespace {

using skinny_host::DeviceInfo;
using skinny_host::Range;
using skinny_host::aligned;
using skinny_host::device_info;
using skinny_host::overlap;
using skinny_host::range_of;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));   // y's rows of an odd width
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRowBlock = 64;          // rows whose adapters a wave looks over at once
constexpr int kPiece = 64;             // values of K per row and wave at a time: a cache line
constexpr int kCols = 64;              // columns of y of a wave
constexpr int kMaxSlices = SKINNY_LORA_MAX_SLICES;

struct LoraArgs {
  const __bf16* x;
  const __bf16* base;
  __bf16* y;
  const int* ids;
  const int* ranks;
  const float* scale;
  float* part;                         // [splits][slices][rows][rank]
  const __bf16* a[kMaxSlices];
  const __bf16* b[kMaxSlices];
  int n[kMaxSlices], col[kMaxSlices];  // columns of a slice, and the first one's number in y
  int tile[kMaxSlices + 1];            // first column tile of a slice
  int rows, adapters, rank, K, N, slices;
  int splits, pieces;                  // of K, and pieces of a split
  int rank_groups;                     // of 16 MT ranks
  int ordinals;                        // workgroups that share a row block's adapters
  int copy;                            // base is not y: rows without an adapter are copied
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, bf16x2{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ float bf16_lo(unsigned u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) {
  return __builtin_bit_cast(float, u & 0xffff0000u);
}

__device__ __forceinline__ unsigned upper_halves(float a, float b) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, b), __builtin_bit_cast(unsigned, a),
                               0x07060302u);
}
// x - part; 0 for infinities, which part has in full.
__device__ __forceinline__ float rest_of(float x, float part) {
  const float r = x - part;
  return r - r == 0.0f ? r : 0.0f;
}

// The rows of a block that share an adapter.
struct Group {
  int adapter;                         // -1: the rows without one
  unsigned long long lanes;            // bit l: row l of the block
};

// The adapters of a row block, one after the other: lane l holds row l's.
struct Adapters {
  int id;                              // of the lane's row; -1: none
  unsigned long long rest;             // rows with an adapter that has not come yet
  unsigned long long none;             // rows without one
  __device__ __forceinline__ Adapters(const LoraArgs& a, int block) {
    const int t = block * kRowBlock + (threadIdx.x & 63);
    id = t < a.rows ? a.ids[t] : -1;
    if (id < 0 || id >= a.adapters) id = -1;
    rest = __ballot(id >= 0);
    none = __ballot(id < 0 && t < a.rows);
  }
  __device__ __forceinline__ Group next() {
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(rest));
    const unsigned long long same = __ballot(id == e);
    rest &= ~same;
    return Group{e, same};
  }
};

__device__ __forceinline__ int rank_of(const LoraArgs& a, int adapter) {
  return a.ranks ? min(max(uniform(a.ranks[adapter]), 0), a.rank) : a.rank;
}

// Row numbers of a group's rows, side by side, the last one again behind them.
__device__ __forceinline__ void list_rows(const Group& g, int block, int (&list)[kRowBlock]) {
  const int lane = threadIdx.x & 63;
  const int count = __popcll(g.lanes);
  const int at = __popcll(g.lanes & ((1ull << lane) - 1));
  if (threadIdx.x < 64) {
    if (g.lanes >> lane & 1) list[at] = block * kRowBlock + lane;
    if (lane >= count) list[lane] = block * kRowBlock + 63 - __builtin_clzll(g.lanes);
  }
}

// A x for RT tiles of 16 rows and MT tiles of 16 ranks over a split's share of K:
// the waves take pieces of K in turn, and their sums are added in order.
template <int MT, int RT>
__device__ __forceinline__ void shrink(const LoraArgs& a, const __bf16* w, int rank, int r0,
                                       int count, int split, int slice, const int* list,
                                       float* sums) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  f32x4 acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
  const __bf16* xp[RT];
  const __bf16* wp[MT];
#pragma unroll
  for (int t = 0; t < RT; ++t) xp[t] = a.x + (size_t)list[16 * t + c] * a.K + 8 * g;
#pragma unroll
  for (int m = 0; m < MT; ++m) wp[m] = w + (size_t)min(r0 + 16 * m + c, rank - 1) * a.K + 8 * g;
  const int end = min((split + 1) * a.pieces * kPiece, a.K);
  for (int k = (split * a.pieces + wave) * kPiece; k < end; k += kWaves * kPiece) {
    u32x4 xf[2][RT], wf[2][MT];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool in = k + 32 * u + 8 * g < end;
#pragma unroll
      for (int t = 0; t < RT; ++t)
        xf[u][t] = in ? *reinterpret_cast<const u32x4*>(xp[t] + k + 32 * u) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int m = 0; m < MT; ++m)
        wf[u][m] = in ? *reinterpret_cast<const u32x4*>(wp[m] + k + 32 * u) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[m][t] = mfma_bf16(wf[u][m], xf[u][t], acc[m][t]);
  }
  // Lane (c, g), register r holds rank 4g + r of row c.
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < RT; ++t)
      *reinterpret_cast<f32x4*>(sums + ((wave * MT + m) * RT + t) * 256 + lane * 4) = acc[m][t];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * RT * 64; i += kThreads) {
    const int l = i & 63, t = i / 64 % RT, m = i / 64 / RT;
    const int row = 16 * t + (l & 15), r = r0 + 16 * m + 4 * (l >> 4);
    if (row >= count || r >= rank) continue;
    f32x4 s{0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < kWaves; ++v)
      s += *reinterpret_cast<const f32x4*>(sums + ((v * MT + m) * RT + t) * 256 + l * 4);
    *reinterpret_cast<f32x4*>(
        a.part + ((size_t)(split * a.slices + slice) * a.rows + list[row]) * a.rank + r) = s;
  }
  __syncthreads();
}

template <int MT>
__global__ __launch_bounds__(kThreads) void skinny_lora_shrink(const LoraArgs a) {
  __shared__ int list[kRowBlock];
  __shared__ __attribute__((aligned(16))) float sums[kWaves * MT * 4 * 256];
  // Splits of one item run on neighbouring workgroups.
  int i = blockIdx.x;
  const int split = i % a.splits;
  i /= a.splits;
  const int r0 = i % a.rank_groups * 16 * MT;
  i /= a.rank_groups;
  const int slice = i % a.slices;
  i /= a.slices;
  const int ordinal = i % a.ordinals;
  const int block = i / a.ordinals;
  if (!a.a[slice]) return;
  Adapters all(a, block);
  for (int d = 0; all.rest; ++d) {
    const Group grp = all.next();
    if (d % a.ordinals != ordinal) continue;
    const int rank = rank_of(a, grp.adapter);
    if (r0 >= rank) continue;
    list_rows(grp, block, list);
    __syncthreads();
    const int count = __popcll(grp.lanes);
    const __bf16* w = a.a[slice] + (size_t)grp.adapter * a.rank * a.K;
    if (count <= 16) shrink<MT, 1>(a, w, rank, r0, count, split, slice, list, sums);
    else if (count <= 32) shrink<MT, 2>(a, w, rank, r0, count, split, slice, list, sums);
    else shrink<MT, 4>(a, w, rank, r0, count, split, slice, list, sums);
  }
}

// y of RT tiles of 16 rows in the wave's columns.
template <int RT>
__device__ __forceinline__ void expand(const LoraArgs& a, const __bf16* w, int rank, int n0, int n,
                                       int col, int count, const int* list, const unsigned* hi,
                                       const unsigned* lo, int stride) {
  const int lane = threadIdx.x & 63;
  const int c = lane & 15, g = lane >> 4;
  f32x4 acc[RT][4];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[t][j] = f32x4{0, 0, 0, 0};
  // Product j's row i is column 16 (i / 4) + 4 j + i % 4, so that a lane ends with
  // 16 neighbouring columns of one row of y.
  const __bf16* wp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = n0 + 16 * (c >> 2) + 4 * j + (c & 3);
    wp[j] = w + (size_t)min(at, n - 1) * a.rank;
  }
  for (int k = 0; k < rank; k += 32) {
    const int at = k + 8 * g;
    u32x4 wf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      wf[j] = at < rank ? *reinterpret_cast<const u32x4*>(wp[j] + at) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e) {    // columns past the adapter's own, whatever they hold
        if (at + 2 * e >= rank) wf[j][e] = 0;
        else if (at + 2 * e + 1 >= rank) wf[j][e] &= 0xffffu;
      }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int v = (16 * t + c) * stride + at / 2;
      const u32x4 vh = *reinterpret_cast<const u32x4*>(hi + v);
      const u32x4 vl = *reinterpret_cast<const u32x4*>(lo + v);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = mfma_bf16(wf[j], vh, acc[t][j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = mfma_bf16(wf[j], vl, acc[t][j]);
    }
  }
  const int first = n0 + 16 * g;
  const int cols = min(n - first, 16);
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (16 * t + c >= count || cols <= 0) continue;
    const size_t at = (size_t)list[16 * t + c] * a.N + col + first;
    if (cols == 16) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        u32x4 v = *reinterpret_cast<const u32x4_any*>(a.base + at + 8 * p);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = pack_bf16(bf16_lo(v[e]) + acc[t][2 * p + e / 2][2 * (e % 2)],
                           bf16_hi(v[e]) + acc[t][2 * p + e / 2][2 * (e % 2) + 1]);
        *reinterpret_cast<u32x4_any*>(a.y + at + 8 * p) = v;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (e < cols) a.y[at + e] = (__bf16)((float)a.base[at + e] + acc[t][e / 4][e % 4]);
    }
  }
}

// Rows that have no adapter, in the workgroup's columns.
__device__ __forceinline__ void copy_rows(const LoraArgs& a, unsigned long long lanes, int block,
                                          int col, int cols) {
  while (lanes) {
    const int l = __builtin_ctzll(lanes);
    lanes &= lanes - 1;
    const size_t at = (size_t)(block * kRowBlock + l) * a.N + col;
    for (int i = threadIdx.x; i < cols; i += kThreads) a.y[at + i] = a.base[at + i];
  }
}

__global__ __launch_bounds__(kThreads) void skinny_lora_expand(const LoraArgs a) {
  __shared__ int list[kRowBlock];
  extern __shared__ __attribute__((aligned(16))) unsigned low[];   // A x in two parts
  int i = blockIdx.x;
  const int tiles = a.tile[a.slices];
  const int tile = i % tiles;
  i /= tiles;
  const int ordinal = i % a.ordinals;
  const int block = i / a.ordinals;
  int slice = 0;
  while (tile >= a.tile[slice + 1]) ++slice;
  const int n = a.n[slice], col = a.col[slice];
  const int tile0 = (tile - a.tile[slice]) * kCols * kWaves;
  const int lane_tile = tile0 + uniform(threadIdx.x >> 6) * kCols;
  const int width = min(n - tile0, kCols * kWaves);
  const bool bare = !a.a[slice];
  const int padded = (a.rank + 31) / 32 * 32;
  const int stride = padded / 2 + 4;                 // dwords of a row, kept off the same banks
  unsigned* hi = low;
  unsigned* lo = low + kRowBlock * stride;

  Adapters all(a, block);
  unsigned long long rest = all.none;
  if (bare) rest |= all.rest;
  if (a.copy && ordinal == 0 && rest) copy_rows(a, rest, block, col + tile0, width);
  if (bare) return;
  for (int d = 0; all.rest; ++d) {
    const Group grp = all.next();
    if (d % a.ordinals != ordinal) continue;
    const int rank = rank_of(a, grp.adapter);
    if (rank == 0) {
      if (a.copy) copy_rows(a, grp.lanes, block, col + tile0, width);
      continue;
    }
    list_rows(grp, block, list);
    __syncthreads();
    const int count = __popcll(grp.lanes);
    const float scale = a.scale ? a.scale[grp.adapter] : 1.0f;
    // Pairs of ranks of every row, up to a whole product of 32.
    const int pairs = (rank + 31) / 32 * 16, tall = (count + 15) / 16 * 16;
    for (int p = threadIdx.x; p < tall * pairs; p += kThreads) {
      const int row = p / pairs, r = p % pairs * 2;
      float s0 = 0.0f, s1 = 0.0f;
      if (row < count && r < rank) {
        const float* src = a.part + ((size_t)slice * a.rows + list[row]) * a.rank + r;
        for (int k = 0; k < a.splits; ++k) {
          const float2 v = *reinterpret_cast<const float2*>(
              src + (size_t)k * a.slices * a.rows * a.rank);
          s0 += v.x;
          s1 += v.y;
        }
        s0 *= scale;
        s1 = r + 1 < rank ? s1 * scale : 0.0f;
      }
      // The upper half of the fp32 number, and what that leaves of it, rounded.
      const unsigned h = upper_halves(s0, s1);
      hi[row * stride + r / 2] = h;
      lo[row * stride + r / 2] = pack_bf16(rest_of(s0, bf16_lo(h)), rest_of(s1, bf16_hi(h)));
    }
    __syncthreads();
    const __bf16* w = a.b[slice] + (size_t)grp.adapter * n * a.rank;
    if (lane_tile < n) {
      if (count <= 16) expand<1>(a, w, rank, lane_tile, n, col, count, list, hi, lo, stride);
      else if (count <= 32) expand<2>(a, w, rank, lane_tile, n, col, count, list, hi, lo, stride);
      else expand<4>(a, w, rank, lane_tile, n, col, count, list, hi, lo, stride);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host side.

struct Cut {
  int splits, pieces, rank_tiles, ordinals;
};

// How a call is cut: from the sizes alone, so that the workspace is known.
Cut cut_of(const skinny_lora& l, int rows) {
  Cut c;
  const int blocks = (rows + kRowBlock - 1) / kRowBlock;
  const int rank_tiles = (l.rank + 15) / 16;
  c.rank_tiles = rank_tiles >= 4 ? 4 : rank_tiles >= 2 ? 2 : 1;
  const int most = rows < l.adapters ? rows : l.adapters;
  c.ordinals = most < kRowBlock ? most : kRowBlock;
  if (blocks > 4) c.ordinals = c.ordinals < 8 ? c.ordinals : 8;
  if (blocks > 32) c.ordinals = c.ordinals < 2 ? c.ordinals : 2;
  const int pieces = (l.K + kPiece - 1) / kPiece;
  const long long items = (long long)blocks * (blocks > 4 ? 1 : c.ordinals) * l.slices *
                          ((rank_tiles + c.rank_tiles - 1) / c.rank_tiles);
  long long splits = (512 + items - 1) / items;
  const int whole = (pieces + kWaves - 1) / kWaves;  // one piece per wave
  if (splits > whole) splits = whole;
  if (splits < 1) splits = 1;
  c.pieces = (int)((pieces + splits - 1) / splits);
  c.splits = (pieces + c.pieces - 1) / c.pieces;
  return c;
}

skinny_status check_lora(const skinny_lora* l, int rows, long long* width) {
  if (!l || rows < 1) return SKINNY_ERR_INVALID_ARG;
  if (l->adapters < 1 || l->rank < 1 || l->K < 1 || l->slices < 1) return SKINNY_ERR_INVALID_ARG;
  if (l->slices > SKINNY_LORA_MAX_SLICES) return SKINNY_ERR_UNSUPPORTED;
  long long n = 0;
  bool any = false;
  for (int i = 0; i < l->slices; ++i) {
    if (l->n[i] < 1 || (l->a[i] != nullptr) != (l->b[i] != nullptr)) return SKINNY_ERR_INVALID_ARG;
    if (!aligned(l->a[i], 16) || !aligned(l->b[i], 16)) return SKINNY_ERR_UNSUPPORTED;
    n += l->n[i];
    any = any || l->a[i];
  }
  if (!any) return SKINNY_ERR_INVALID_ARG;
  if (rows > SKINNY_LORA_MAX_ROWS || l->adapters > 65536 || l->rank % 8 != 0 ||
      l->rank > SKINNY_LORA_MAX_RANK || l->K % 8 != 0 || l->K > (1 << 28) || n > (1 << 28))
    return SKINNY_ERR_UNSUPPORTED;
  if (!aligned(l->ranks, 4) || !aligned(l->scale, 4)) return SKINNY_ERR_UNSUPPORTED;
  *width = n;
  return SKINNY_OK;
}

size_t workspace_of(const skinny_lora& l, int rows) {
  const Cut c = cut_of(l, rows);
  const size_t bytes = (size_t)c.splits * l.slices * rows * l.rank * sizeof(float);
  return bytes > SKINNY_MIN_WORKSPACE_BYTES ? bytes : SKINNY_MIN_WORKSPACE_BYTES;
}

}  // namespace

extern "C" {

size_t skinny_lora_workspace_bytes(const skinny_lora* lora, int rows) {
  long long n;
  return check_lora(lora, rows, &n) == SKINNY_OK ? workspace_of(*lora, rows) : 0;
}

skinny_status skinny_lora_linear(const skinny_lora* lora, const void* x, const int* ids, int rows,
                                 const void* base, void* y, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  long long width = 0;
  skinny_status st = check_lora(lora, rows, &width);
  if (st != SKINNY_OK) return st;
  const skinny_lora& l = *lora;
  if (!x || !ids || !y) return SKINNY_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(ids, 4) || !aligned(y, 2) || !aligned(base, 2))
    return SKINNY_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < workspace_of(l, rows)) return SKINNY_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SKINNY_ERR_UNSUPPORTED;
  if (!base) base = y;
  const size_t yb = (size_t)rows * width * 2;
  const Range yr = range_of(y, yb), wr = range_of(workspace, workspace_bytes);
  Range in[5 + 2 * SKINNY_LORA_MAX_SLICES];
  int m = 0;
  in[m++] = range_of(x, (size_t)rows * l.K * 2);
  in[m++] = range_of(ids, (size_t)rows * 4);
  if (l.ranks) in[m++] = range_of(l.ranks, (size_t)l.adapters * 4);
  if (l.scale) in[m++] = range_of(l.scale, (size_t)l.adapters * 4);
  for (int i = 0; i < l.slices; ++i) {
    if (!l.a[i]) continue;
    in[m++] = range_of(l.a[i], (size_t)l.adapters * l.rank * l.K * 2);
    in[m++] = range_of(l.b[i], (size_t)l.adapters * l.rank * l.n[i] * 2);
  }
  if (base != y) in[m++] = range_of(base, yb);
  if (overlap(yr, wr)) return SKINNY_ERR_INVALID_ARG;
  for (int i = 0; i < m; ++i)
    if (overlap(yr, in[i]) || overlap(wr, in[i])) return SKINNY_ERR_INVALID_ARG;

  const Cut c = cut_of(l, rows);
  LoraArgs a;
  a.x = (const __bf16*)x;
  a.base = (const __bf16*)base;
  a.y = (__bf16*)y;
  a.ids = ids;
  a.ranks = l.ranks;
  a.scale = l.scale;
  a.part = (float*)workspace;
  a.rows = rows;
  a.adapters = l.adapters;
  a.rank = l.rank;
  a.K = l.K;
  a.N = (int)width;
  a.slices = l.slices;
  a.splits = c.splits;
  a.pieces = c.pieces;
  a.rank_groups = (l.rank + 16 * c.rank_tiles - 1) / (16 * c.rank_tiles);
  a.ordinals = c.ordinals;
  a.copy = base != y;
  int col = 0, tile = 0;
  for (int i = 0; i < kMaxSlices; ++i) {
    const bool in_use = i < l.slices;
    a.a[i] = in_use ? (const __bf16*)l.a[i] : nullptr;
    a.b[i] = in_use ? (const __bf16*)l.b[i] : nullptr;
    a.n[i] = in_use ? l.n[i] : 0;
    a.col[i] = col;
    a.tile[i] = tile;
    col += a.n[i];
    tile += (a.n[i] + kCols * kWaves - 1) / (kCols * kWaves);
  }
  a.tile[kMaxSlices] = tile;
  for (int i = l.slices; i < kMaxSlices; ++i) a.tile[i] = tile;
  const long long blocks = (rows + kRowBlock - 1) / kRowBlock;
  const long long first = blocks * a.ordinals * a.slices * a.rank_groups * a.splits;
  const long long second = blocks * a.ordinals * tile;
  if (first * kThreads > 0xffffffffLL || second * kThreads > 0xffffffffLL)   // threads of a launch
    return SKINNY_ERR_UNSUPPORTED;
  DeviceInfo d;
  st = device_info(&d);
  if (st != SKINNY_OK) return st;
  if (!d.gfx950) return SKINNY_ERR_UNSUPPORTED;

  const hipStream_t hs = (hipStream_t)stream;
  const dim3 grid((unsigned)first), threads(kThreads);
  if (c.rank_tiles == 1) hipLaunchKernelGGL(skinny_lora_shrink<1>, grid, threads, 0, hs, a);
  else if (c.rank_tiles == 2) hipLaunchKernelGGL(skinny_lora_shrink<2>, grid, threads, 0, hs, a);
  else hipLaunchKernelGGL(skinny_lora_shrink<4>, grid, threads, 0, hs, a);
  if (hipGetLastError() != hipSuccess) return SKINNY_ERR_HIP;
  const int padded = (l.rank + 31) / 32 * 32;
  const size_t lds = (size_t)2 * kRowBlock * (padded / 2 + 4) * sizeof(unsigned);
  if (lds > 60 * 1024 &&               // beside the list, more than a launch may have unasked
      hipFuncSetAttribute((const void*)skinny_lora_expand,
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
    return SKINNY_ERR_HIP;
  hipLaunchKernelGGL(skinny_lora_expand, dim3((unsigned)second), threads, lds, hs, a);
  return hipGetLastError() == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP;
}

}  // extern "C"
