// fa_kv8_sched.cuh -- what the two attention kernels of the 8-bit cache share: their parameters, the even
// division of ragged work over the CTAs, and the kernel that merges units cut by it.
#pragma once
#include <algorithm>

#include "fa_internal.h"
#include "fa_kv8.h"
#include "fa_prefill_common.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kSms = 148;
constexpr float kLazy = 8.f;     // log2 units by which a maximum may be exceeded before it is raised
// Weights of O are 2^kHead times the contribution relative to the largest one, so they stay below 2^(kHead + kLazy) = 2^15, half
// of what fp16 holds, and a contribution counts down to 2^-32 of the largest (with a unit of 1 it was lost below
// 2^-25, while the row sum had it: many small keys beside a large one of no value were gone from O).
constexpr float kHead = 7.f;
constexpr float kUnhead = 0x1p-7f;
constexpr float kNone = -1e30f;  // a maximum over nothing (finite, so that differences with -inf are defined)
constexpr int kStatusPageTable = 12;  // FA_ERR_PAGE_TABLE


struct AttParams {
  const void* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const int* table;
  const int* seqlens;
  void* o;
  float* lse;
  float* ws_o;  // [2 * shares, rows of a tile, D]: pieces of units
  float* ws_l;  // [2 * shares, rows of a tile]
  int B, Nq, Hq, Hkv, group, tiles;
  int granule;  // keys
  int over;     // granules that the fixed cost of a unit (queries, the first tiles, the merge) stands for; 0: a
                // granule is a whole unit, and no unit is cut
  int least;    // cost of the smallest share: shorter ones cost more to merge than to read
  int num_pages, page_shift, pps;
  float scale_log2;
  int* status;
};

// The parameters that do not depend on the kernel.
inline AttParams params_of(const Attend8Args& a) {
  AttParams p{};
  p.q = a.q;
  p.k = static_cast<const uint8_t*>(a.c.k);
  p.v = static_cast<const uint8_t*>(a.c.v);
  p.ks = a.c.ks;
  p.vs = a.c.vs;
  p.table = a.c.table;
  p.seqlens = a.c.seqlens;
  p.o = a.o;
  p.lse = a.lse;
  p.B = a.c.B;
  p.Nq = a.Nq;
  p.Hq = a.Hq;
  p.Hkv = a.c.Hkv;
  p.group = a.Hq / a.c.Hkv;
  p.num_pages = a.c.num_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.c.page_size) ++p.page_shift;
  p.pps = a.c.pages_per_seq;
  p.scale_log2 = a.scale * kLog2e;
  p.status = a.status;
  return p;
}

// 2^e as fp32, e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// log2 of a V scale.  A scale of zero stands for values of zero: no weight, and no say in the maximum of O.
__device__ __forceinline__ float log2_scale(float vs) { return vs > 0.f ? lg2(fmaxf(vs, 1.17549435e-38f)) : -INFINITY; }

// Two weights as fp16.  Beyond scores of 10^7, where a step of the score is a factor of two and more, they could pass
// its range: the largest finite value then.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool kFp16>
__device__ __forceinline__ void store2(void* o, size_t at, float a, float b, bool f32) {
  if (f32) *reinterpret_cast<float2*>(static_cast<float*>(o) + at) = make_float2(a, b);
  else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(o) + at) = pack2<kFp16>(a, b);
}

// Keys of batch item b (0 for a length outside its range).
__device__ __forceinline__ int keys_of(const AttParams& p, int b) {
  const int cap = p.pps << p.page_shift;
  if (!p.seqlens) return cap;
  const int len = __ldg(p.seqlens + b);
  return len < 0 || len > cap ? 0 : len;
}

// Keys that a row sees (rows of a token see the same ones), and granules of a row tile.
__device__ __forceinline__ int row_limit(const AttParams& p, int len, int row) { return max(0, len - p.Nq + row / p.group + 1); }
template <int kRows>
__device__ __forceinline__ int tile_keys(const AttParams& p, int len, int tile) {
  return row_limit(p, len, min(p.Nq * p.group, (tile + 1) * kRows) - 1);
}
template <int kRows>
__device__ __forceinline__ int tile_granules(const AttParams& p, int len, int tile) {
  return (tile_keys<kRows>(p, len, tile) + p.granule - 1) / p.granule;
}
// Cost of an item: the granules of its units and the units' fixed costs (a unit without granules has none).
template <int kRows>
__device__ __forceinline__ long long item_cost(const AttParams& p, int len) {
  long long n = 0;
  for (int i = 0; i < p.tiles; ++i) {
    const int m = tile_granules<kRows>(p, len, i);
    n += m > 0 ? m + p.over : 0;
  }
  return n * p.Hkv;
}

// Where a share begins: item b, `off` of the item's cost.
struct Place {
  long long total;  // cost of all items
  long long off;
  int b;
  bool short_items;  // some item has fewer keys than queries (or a length out of range)
};

template <int kThreads>
struct ScanMem {
  long long sums[kThreads / 32];
  long long off;
  int b;
};

// Number of shares of a total cost, and where share c begins.
__device__ __forceinline__ int shares_of(const AttParams& p, long long total, int grid) {
  return static_cast<int>(min(static_cast<long long>(grid), (total + p.least - 1) / p.least));
}
__device__ __forceinline__ long long share_begin(long long total, int shares, int c) {
  if (total < (1LL << 31)) {  // (a 64-bit division takes a hundred instructions)
    const unsigned q = static_cast<unsigned>(total) / static_cast<unsigned>(shares), r = static_cast<unsigned>(total) % static_cast<unsigned>(shares);
    return static_cast<long long>(q) * c + min(c, static_cast<int>(r));
  }
  return total / shares * c + min(static_cast<long long>(c), total % shares);
}

// The place where share c begins: a scan of the items' costs, a CTA's worth at a time, once
// for the total and (with more items than threads) once to find the place.  Collective.
template <int kRows, int kThreads>
__device__ __forceinline__ Place find_place(const AttParams& p, int grid, int c, ScanMem<kThreads>& sm) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Place r;
  long long mine = 0, sum = 0;
  bool few = false;
  for (int b = tid; b < p.B; b += kThreads) {
    const int len = keys_of(p, b);
    few |= len < p.Nq;
    sum += (mine = item_cost<kRows>(p, len));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sm.sums[warp] = sum;
  r.short_items = __syncthreads_or(few) != 0;
  r.total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) r.total += sm.sums[w];
  const int shares = shares_of(p, r.total, grid);
  r.b = -1;
  r.off = 0;
  if (c >= shares) return r;  // uniform: this CTA has no share
  const long long want = share_begin(r.total, shares, c);
  long long before = 0;
  for (int base = 0; base < p.B; base += kThreads) {
    const int b = base + tid;
    const long long n = p.B <= kThreads ? (b < p.B ? mine : 0) : (b < p.B ? item_cost<kRows>(p, keys_of(p, b)) : 0);
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();  // sums were read
    if (lane == 31) sm.sums[warp] = x;
    __syncthreads();
    long long all = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) x += sm.sums[w];
      all += sm.sums[w];
    }
    x += before;  // cost up to and with this item
    if (want < x && want >= x - n) {
      sm.b = b;
      sm.off = want - (x - n);
    }
    before = all;
    if (want < all) break;  // uniform
  }
  __syncthreads();
  r.b = sm.b;
  r.off = sm.off;
  return r;
}

// The unit (row tile, KV head) that `off` of the cost of an item with len keys lies in, its granules, and the
// place inside it: r of its cost, where the fixed cost comes first, so granule max(0, r - over).
struct Unit {
  int tile, hk, n, r, g0;
};
template <int kRows>
__device__ __forceinline__ Unit unit_at(const AttParams& p, int len, long long off) {
  Unit u;
  for (u.tile = 0;; ++u.tile) {
    u.n = tile_granules<kRows>(p, len, u.tile);
    const long long here = u.n > 0 ? static_cast<long long>(u.n + p.over) * p.Hkv : 0;
    if (off < here) break;
    off -= here;
  }
  const unsigned cost = u.n + p.over;
  if (off < (1LL << 31)) {
    u.hk = static_cast<int>(static_cast<unsigned>(off) / cost);
    u.r = static_cast<int>(static_cast<unsigned>(off) % cost);
  } else {
    u.hk = static_cast<int>(off / cost);
    u.r = static_cast<int>(off % cost);
  }
  u.g0 = max(0, u.r - p.over);
  return u;
}

// Index of a row among the rows of O [B, Nq, Hq, D], and of its LSE [B, Hq, Nq].
__device__ __forceinline__ size_t o_row(const AttParams& p, int b, int hk, int row) {
  return (static_cast<size_t>(b) * p.Nq + row / p.group) * p.Hq + hk * p.group + row % p.group;
}
__device__ __forceinline__ size_t lse_row(const AttParams& p, int b, int hk, int row) {
  return (static_cast<size_t>(b) * p.Hq + hk * p.group + row % p.group) * p.Nq + row / p.group;
}

// A share under way: the items' costs that are left of it, from `off` in item b on.
struct Walk {
  long long left, off;
  int b;
};

// One piece of a share: keys [lo, hi) of a unit.
struct Piece {
  int b, hk, row0, len, lo, hi;
  int slot;   // of the workspace (0: the share's first piece, 1: its last one that begins its unit)
  bool whole;  // the unit lies in this share
};

__device__ __forceinline__ Walk walk_of(const AttParams& p, const Place& place, int grid, int c) {
  const int shares = shares_of(p, place.total, grid);
  Walk w;
  w.left = share_begin(place.total, shares, c + 1) - share_begin(place.total, shares, c);
  w.off = place.off;
  w.b = place.b;
  return w;
}

template <int kRows>
__device__ __forceinline__ bool next_piece(const AttParams& p, Walk& w, Piece& s) {
  while (w.left > 0) {
    const int len = keys_of(p, w.b);
    if (w.off >= item_cost<kRows>(p, len)) {  // (items without granules are passed over)
      ++w.b;
      w.off = 0;
      continue;
    }
    const Unit u = unit_at<kRows>(p, len, w.off);
    const int use = static_cast<int>(min(w.left, static_cast<long long>(u.n + p.over - u.r)));
    const int take = max(0, u.r + use - p.over) - u.g0;
    w.left -= use;
    w.off += use;
    if (take == 0) continue;  // a share that ends in the fixed cost of a unit leaves the unit to the next
    s.b = w.b;
    s.hk = u.hk;
    s.row0 = u.tile * kRows;
    s.len = len;
    s.lo = u.g0 * p.granule;
    s.hi = static_cast<int>(min(static_cast<long long>(tile_keys<kRows>(p, len, u.tile)), static_cast<long long>(s.lo) + static_cast<long long>(take) * p.granule));
    s.slot = u.g0 == 0 ? 1 : 0;
    s.whole = u.g0 == 0 && take == u.n;
    return true;
  }
  return false;
}

// O = 0 and LSE = -inf for the rows of tiles that see no key (only items with fewer keys than queries have any), and
// the report of lengths out of range.  An item with few such rows is left to one CTA, many rows are spread over the
// grid; a warp looks at 32 items at once.
template <bool kFp16, int D, int kRows>
__device__ __forceinline__ void write_tiles_without_keys(const AttParams& p, int o_fp32) {
  const int rows = p.Nq * p.group, lane = threadIdx.x & 31;
  // rows of the first Nq - len tokens see no key; of those, the ones in tiles that hold nothing else
  auto dead_rows = [&](int len) {
    const long long none = static_cast<long long>(p.Nq - len) * p.group;
    return none >= rows ? rows : static_cast<int>(none / kRows * kRows);
  };
  for (int base = 0; base < p.B; base += 32) {
    const int mine = base + lane, len_l = mine < p.B ? keys_of(p, mine) : p.Nq;
    const bool few = len_l < p.Nq;
    if (few && p.seqlens && blockIdx.x == 0 && threadIdx.x < 32) {
      const int given = __ldg(p.seqlens + mine);
      if (given < 0 || given > (p.pps << p.page_shift)) record_status(p.status, kStatusCuSeqlens);
    }
    const bool spread = few && static_cast<long long>(dead_rows(len_l)) * p.Hkv > 256;
    unsigned todo = __ballot_sync(0xffffffffu, few && (spread || mine % static_cast<int>(gridDim.x) == static_cast<int>(blockIdx.x)));
    const unsigned wide = __ballot_sync(0xffffffffu, spread);
    while (todo) {
      const int at_lane = __ffs(todo) - 1, b = base + at_lane;
      todo &= todo - 1;
      const bool all = (wide >> at_lane) & 1;
      const long long n = static_cast<long long>(dead_rows(__shfl_sync(0xffffffffu, len_l, at_lane))) * p.Hkv * (D / 8);
      const long long first = all ? static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x : threadIdx.x;
      const long long step = all ? static_cast<long long>(gridDim.x) * blockDim.x : blockDim.x;
      for (long long i = first; i < n; i += step) {
        const unsigned r = static_cast<unsigned>(i / (D / 8));
        const int row = static_cast<int>(r / static_cast<unsigned>(p.Hkv)), hk = static_cast<int>(r % static_cast<unsigned>(p.Hkv)), d = static_cast<int>(i % (D / 8)) * 8;
        const size_t at = o_row(p, b, hk, row);
        if (!idx_ok(p.status, at, 1, static_cast<long long>(p.B) * p.Nq * p.Hq)) continue;
#pragma unroll
        for (int e = 0; e < 8; e += 2) store2<kFp16>(p.o, at * D + d + e, 0.f, 0.f, o_fp32 != 0);
        if (d == 0) p.lse[lse_row(p, b, hk, row)] = -INFINITY;
      }
    }
  }
}

// Merges the pieces of the units that lie in more than one share.  CTA i looks at the border between
// shares i and i + 1 and takes the unit it cuts, if no earlier border cuts the same one: piece 0 is the
// end of share i, the others are the beginnings of shares i + 1, i + 2, ...  O = sum_s exp(lse_s - M) o_s /
// sum_s exp(lse_s - M), LSE = M + ln of that sum; two rows to a warp, eight of a tile to a CTA.  kMany, for long
// contexts of few heads, which come in a hundred pieces and more: two rows to a CTA, whose warps take a
// quarter of the pieces each (2 x 95246 keys, 10 rows: 58 us without it, 36 with it).
constexpr int kCombineThreads = 128;
template <bool kMany>
constexpr int kCombineRows = kMany ? 2 : 8;

template <bool kFp16, int D, int kRows, bool kMany>
__global__ void __launch_bounds__(kCombineThreads) kv8_combine_kernel(const AttParams p, const int o_fp32, const int grid) {
  constexpr int kPart = kCombineRows<kMany>, kWarps = kCombineThreads / 32;
  constexpr int PER = D / 32, RPW = 2;        // rows of a warp, both under way at once
  constexpr int kStride = kMany ? 1 : kWarps;  // between them
  __shared__ ScanMem<kCombineThreads> scan;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x + 1;
  const Place place = find_place<kRows, kCombineThreads>(p, grid, c, scan);
  // what follows this kernel must find the first one done, also where no border cuts a unit
  if (blockIdx.x == 0 && blockIdx.y == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (place.b < 0) return;
  const int shares = shares_of(p, place.total, grid);
  const Unit u = unit_at<kRows>(p, keys_of(p, place.b), place.off);
  const long long begin = share_begin(place.total, shares, c) - u.r, end = begin + u.n + p.over;
  if (u.g0 == 0 || share_begin(place.total, shares, c - 1) > begin + p.over) return;
  int pieces = 1;  // beside the first
  while (c + pieces < shares && share_begin(place.total, shares, c + pieces) < end) ++pieces;
  auto slot = [&](int s) { return static_cast<size_t>(s == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + s)) * kRows; };
  const int rows = min(kRows, p.Nq * p.group - u.tile * kRows), part = blockIdx.y * kPart;
  if (part >= rows) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are written

  const int each = kMany ? (pieces + kWarps) / kWarps : pieces + 1;  // pieces of this warp
  const int from = kMany ? warp * each : 0, to = min(from + each, pieces + 1);
  float M[RPW], sum[RPW], acc[RPW][PER];
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    const int row = part + (kMany ? 0 : warp) + i * kStride;
    M[i] = kNone;
    for (int s = from + lane; s < to && row < rows; s += 32) M[i] = fmaxf(M[i], p.ws_l[slot(s) + row] * kLog2e);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M[i] = fmaxf(M[i], __shfl_xor_sync(0xffffffffu, M[i], o));
    sum[i] = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[i][e] = 0.f;
  }
  // eight pieces' loads are under way at once
  for (int s0 = from; s0 < to; s0 += 8) {
    float w[RPW][8];
    float2 x[RPW][8][PER / 2];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        const int row = part + (kMany ? 0 : warp) + i * kStride;
        const bool in = s0 + k < to && row < rows;
        const size_t at = slot(in ? s0 + k : 0) + (in ? row : 0);
        w[i][k] = in ? p.ws_l[at] : -INFINITY;
        const float2* src = reinterpret_cast<const float2*>(p.ws_o + at * D) + lane * (PER / 2);
#pragma unroll
        for (int e = 0; e < PER / 2; ++e) x[i][k][e] = in ? src[e] : make_float2(0.f, 0.f);
      }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        const float f = ex2(w[i][k] * kLog2e - M[i]);
        sum[i] += f;
#pragma unroll
        for (int e = 0; e < PER / 2; ++e) {
          acc[i][2 * e] = fmaf(f, x[i][k][e].x, acc[i][2 * e]);
          acc[i][2 * e + 1] = fmaf(f, x[i][k][e].y, acc[i][2 * e + 1]);
        }
      }
  }
  if constexpr (kMany) {  // the warps' sums, in order
    __shared__ float part_m[kWarps][RPW], part_sum[kWarps][RPW], part_acc[kWarps][RPW][D];
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      part_m[warp][i] = M[i];
      part_sum[warp][i] = sum[i];
#pragma unroll
      for (int e = 0; e < PER; ++e) part_acc[warp][i][lane * PER + e] = acc[i][e];
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M[i] = fmaxf(M[i], part_m[w][i]);
      sum[i] = 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[i][e] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(part_m[w][i] - M[i]);
        sum[i] = fmaf(f, part_sum[w][i], sum[i]);
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[i][e] = fmaf(f, part_acc[w][i][lane * PER + e], acc[i][e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    const int row = part + (kMany ? 0 : warp) + i * kStride, rr = u.tile * kRows + row;
    if (row >= rows) continue;
    const bool none = sum[i] == 0.f;  // (not by M: a NaN leaves that where it was)
    const float inv = none ? 0.f : 1.f / sum[i];
    const size_t at = o_row(p, place.b, u.hk, rr);
    if (!idx_ok(p.status, at, 1, static_cast<long long>(p.B) * p.Nq * p.Hq)) continue;
#pragma unroll
    for (int e = 0; e < PER / 2; ++e)
      store2<kFp16>(p.o, at * D + lane * PER + 2 * e, acc[i][2 * e] * inv, acc[i][2 * e + 1] * inv, o_fp32 != 0);
    if (lane == 0) p.lse[lse_row(p, place.b, u.hk, rr)] = none ? -INFINITY : (M[i] + lg2(sum[i])) * kLn2;
  }
}

// Launched while the first kernel still runs: it finds its place meanwhile and waits for the pieces.
template <bool kFp16, int D, int kRows, bool kMany = false>
int launch_combine8(const AttParams& p, int o_fp32, int grid, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const long long rows = std::min<long long>(kRows, static_cast<long long>(p.Nq) * p.group);  // of the largest tile
  cfg.gridDim = dim3(grid - 1, static_cast<unsigned>((rows + kCombineRows<kMany> - 1) / kCombineRows<kMany>));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kv8_combine_kernel<kFp16, D, kRows, kMany>, p, o_fp32, grid));
}

}  // namespace
}  // namespace fa
