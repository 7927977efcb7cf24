// fa_kv8_attend.cu -- attention of the newest tokens of each sequence over its paged 8-bit cache.
//
// Codes c and one fp32 scale per (16 tokens, head): K_j = ks(j) ck_j, V_j = vs(j) cv_j.  A code has at
// most 8 significant bits and is exact in fp16, so both products run on fp16 tensor-core operands
// straight from the codes, and the scales enter in fp32 around them, once per 16 keys:
//   s_j  = (q . ck_j) * ks(j) * scale            (fp32; a bf16 query row is first multiplied by a power
//                                                 of two that brings its largest value below 2^15: its
//                                                 8-bit significands are exact in fp16)
//   m    = running max of s_j, l = sum 2^(s_j - m)
//   mo   = running max of s_j + log2 vs(j), O = sum 2^(s_j + log2 vs(j) - mo) cv_j
// O has a maximum of its own: its weights carry the value scales, so they are rounded to fp16 (11
// significant bits) relative to the largest contribution whatever the scales are, and nothing
// overflows.  At the end O * 2^(mo - m) / l.  Both maxima are raised lazily (by more than 2^8 only).
//
// Rows: the G = Hq / Hkv query heads of a KV head times the Nq tokens, token-major, in tiles of 8, 16, 24 or 32:
// keys are the M of the warp MMAs and rows their N, so that few rows waste little of the tensor pipe (a
// 16-row M took 275 of its cycles per block where 8 rows take 138):
//   S^T [16 keys x 8 rows]   = K [16 keys x D] Q^T,   O^T [D x 8 rows] += V^T [D x 16 keys] W^T [16 keys x 8 rows];
// the weights go from the accumulator's layout to the operand's with a movmatrix.
// Work is cut evenly over the CTAs (two to four per SM), whatever the lengths are: the
// granules (64 keys) of all units (sequence, row tile, KV head) are numbered through, with a few more for
// each unit's fixed cost, and CTA c takes the c-th equal share, which may begin and end inside a unit, and finds its place with a scan over the
// lengths.  A unit that lies in one share is written at once; the pieces of the others go to the
// workspace (at most two per CTA) and are merged in order by a second kernel.  Warp w of the four takes every
// fourth block of 16 keys: a block has one scale per pool and lies in one page, so a warp needs nothing
// from the others until the end of a unit.  It streams its blocks (16 x D bytes of K and of V, contiguous in a
// page) through a ring of its own in shared memory with 16-byte cp.async, keys past the end filled with
// zeros, and reads them back as 16-byte (K) and 16- or 8-byte (V) pieces of a row: which k slot of an
// MMA a value takes is free as long as both operands agree, so no transposition is needed but of the
// byte pairs of V (two PRMT per eight codes).  The ring's 16-byte chunks are swizzled so that both reads
// are free of bank conflicts.  Warps and pieces are merged by their (m, l, mo, O).
#include <algorithm>

#include "fa_internal.h"
#include "fa_kv8.h"
#include "fa_prefill_common.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLazy = 8.f;  // log2 units by which a maximum may be exceeded before it is raised
constexpr float kNone = -1e30f;  // a maximum over nothing (finite, so that differences with -inf are defined)
constexpr int kStatusPageTable = 12;  // FA_ERR_PAGE_TABLE
constexpr int kSms = 148;
constexpr int kGranule = 64;      // keys: one block of 16 for each warp
constexpr int kMinShare = 8;      // granules (a unit's fixed cost included) of a share: shorter ones cost more to merge than to read
constexpr int kUnitCost = 4;      // granules that the fixed cost of a unit (queries, filling the ring, merging the warps) stands for
constexpr int kShortKeys = 512;   // tables up to this many keys: a granule is a whole unit, and nothing is merged

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
  int over;     // kUnitCost, or 0 where a granule is a whole unit
  int num_pages, page_shift, pps;
  float scale_log2;
  int* status;
};

// CTAs per SM for tiles of NG * 8 rows (O takes 32 registers per eight rows at D = 128), and the ring.  Four of
// one group leave 128 registers and less overlap inside a warp: 200 us where three take 193 (4 x 131072).
template <int NG>
constexpr int kPerSm = NG <= 2 ? 3 : 2;

template <int D, int NG>
struct Ring {
  static constexpr int kRows = 8 * NG;
  static constexpr int kBlock = kKv8Block * D;  // bytes of 16 keys of K or V
  static constexpr int kStage = 2 * kBlock;
  static constexpr int kRoom = (227 * 1024 / kPerSm<NG> - 2048) / kWarps - 128;
  static constexpr int kStages = kRoom / kStage < 8 ? kRoom / kStage : 8;
  static constexpr int kWarp = kStages * kStage + 128;  // the stages, then (ks, vs) of each, 16 bytes apart
  static constexpr int kMerge = kWarps * kRows * (D + 3) * 4;
  static constexpr int kSmem = kWarps * kWarp > kMerge ? kWarps * kWarp : kMerge;
  static_assert(kStages >= 3 && kStages * 16 <= 128, "stages, and their scales");
};

// Byte offset of 16-byte chunk ch of row r of a 16 x D block.  D = 128: a row is one 128-byte line; rows
// 2i and 2i + 1 differ in bit 2 of the chunk (K: lanes read four chunks of two rows at once) and rows 2t
// (or 2t + 1), t = 0..3, in bits 1-2 (V: two chunks of four rows).  D = 64: two rows share a line.
template <int D>
__device__ __forceinline__ uint32_t ring_off(int r, int ch) {
  if constexpr (D == 128) return r * 128 + ((ch ^ (2 * (((r >> 1) & 3) ^ ((r & 1) << 1)))) << 4);
  else return (r >> 1) * 128 + ((((r & 1) * 4 + ch) ^ (2 * ((r >> 1) & 3))) << 4);
}

// Float of row r, column d in the merge buffer: 16-byte chunks swizzled so that the eight lanes that store
// at once (two columns D / 8 apart, rows 2t) do not share banks.
template <int D>
__device__ __forceinline__ int merge_at(int r, int d) {
  const int ch = d >> 2, t = (r >> 1) & 3;
  return r * D + ((ch ^ (D == 128 ? t : (t & 1) | ((t >> 1) << 2))) << 2) + (d & 3);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4_or_zero(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(full ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Four codes as fp16 pairs: e4m3 codes (0, 1) and (2, 3) of the word by the hardware's conversion (2.9 clocks
// per warp and pair), int8 codes (0, 2) and (1, 3): code + 128 in the mantissa of 1024, less 1152, all exact.
template <bool kInt8>
__device__ __forceinline__ void halves_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kInt8) {
    lo = (w & 0x00FF00FFu) ^ 0x64806480u;
    hi = ((w >> 8) & 0x00FF00FFu) ^ 0x64806480u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&lo), off), y = __hsub2(*reinterpret_cast<__half2*>(&hi), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
  }
}

// Bytes 2i, 2i + 1 of two words so that halves_of gives (x, y) pairs of byte 2i (lo) and 2i + 1 (hi).
template <bool kInt8, int i>
__device__ __forceinline__ uint32_t pair_bytes(uint32_t x, uint32_t y) {
  return __byte_perm(x, y, kInt8 ? (i ? 0x7632 : 0x5410) : (i ? 0x7362 : 0x5140));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}

// 2^e as fp32, e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

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
};

struct ScanMem {
  long long sums[kWarps];
  long long off;
  int b;
};

// Number of shares of a total cost, and where share c begins.
__device__ __forceinline__ int shares_of(const AttParams& p, long long total, int grid) {
  const int least = p.over ? kMinShare : 1;
  return static_cast<int>(min(static_cast<long long>(grid), (total + least - 1) / least));
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
template <int kRows>
__device__ __forceinline__ Place find_place(const AttParams& p, int grid, int c, ScanMem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Place r;
  long long mine = 0, sum = 0;
  for (int b = tid; b < p.B; b += kThreads) sum += (mine = item_cost<kRows>(p, keys_of(p, b)));
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sm.sums[warp] = sum;
  __syncthreads();
  r.total = sm.sums[0] + sm.sums[1] + sm.sums[2] + sm.sums[3];
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

template <bool kFp16, bool kInt8, int D, int NG>
__global__ void __launch_bounds__(kThreads, kPerSm<NG>) kv8_attend_kernel(const AttParams p, const int o_fp32) {
  using R = Ring<D, NG>;
  constexpr int kRows = R::kRows, kStages = R::kStages;
  constexpr int LD = D / 64;  // 16-byte pieces of a K row per lane
  constexpr int MT = D / 16;  // 16-column tiles of O (M of the second product)
  constexpr int kDShift = D == 128 ? 7 : 6;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ScanMem scan;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rows = p.Nq * p.group;
  const long long outs = static_cast<long long>(p.B) * p.Nq * p.Hq;
  const long long pool = (static_cast<long long>(p.num_pages) * p.Hkv) << p.page_shift;

  // rows of tiles that see no key at all, and lengths out of range (reported)
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (p.seqlens && tid == 0) {
      const int len = __ldg(p.seqlens + b);
      if (len < 0 || len > (p.pps << p.page_shift)) record_status(p.status, kStatusCuSeqlens);
    }
    const int len = keys_of(p, b);
    for (int tile = 0; tile < p.tiles && tile_keys<kRows>(p, len, tile) == 0; ++tile) {
      const int n = min(rows - tile * kRows, kRows) * p.Hkv;
      for (int i = tid; i < n * (D / 2); i += kThreads) {
        const int row = tile * kRows + i / (D / 2) / p.Hkv, hk = i / (D / 2) % p.Hkv, d = i % (D / 2) * 2;
        const size_t at = o_row(p, b, hk, row);
        if (!idx_ok(p.status, at, 1, outs)) continue;
        store2<kFp16>(p.o, at * D + d, 0.f, 0.f, o_fp32 != 0);
        if (d == 0) p.lse[lse_row(p, b, hk, row)] = -INFINITY;
      }
    }
  }

  asm volatile("griddepcontrol.launch_dependents;");
  const Place place = find_place<kRows>(p, gridDim.x, blockIdx.x, scan);
  if (place.b < 0) return;
  const int shares = shares_of(p, place.total, gridDim.x);
  long long left = share_begin(place.total, shares, blockIdx.x + 1) - share_begin(place.total, shares, blockIdx.x);
  long long off = place.off;
  int b = place.b;

  const uint32_t ring = smem_addr(smem) + warp * R::kWarp, ring_s = ring + kStages * R::kStage;

  while (left > 0) {
    const int len = keys_of(p, b);
    if (off >= item_cost<kRows>(p, len)) {  // (items without granules are passed over)
      ++b;
      off = 0;
      continue;
    }
    const Unit u = unit_at<kRows>(p, len, off);
    const int use = static_cast<int>(min(left, static_cast<long long>(u.n + p.over - u.r)));
    const int take = max(0, u.r + use - p.over) - u.g0;
    left -= use;
    off += use;
    if (take == 0) continue;  // a share that ends in the fixed cost of a unit leaves the unit to the next
    const int row0 = u.tile * kRows, hk = u.hk;
    const int tile_end = tile_keys<kRows>(p, len, u.tile), tile_all = row_limit(p, len, row0);
    const int lo = u.g0 * p.granule;
    const int hi = static_cast<int>(min(static_cast<long long>(tile_end), static_cast<long long>(lo) + static_cast<long long>(take) * p.granule));
    const bool whole = u.g0 == 0 && take == u.n;

    // the first blocks are on their way before the queries are read
    const int blocks = ((hi - lo + kKv8Block - 1) / kKv8Block - warp + kWarps - 1) / kWarps;
    const int* table = p.table + static_cast<long long>(b) * p.pps;
    const int key_w = lo + warp * kKv8Block;  // first key of this warp's block 0
    auto page_of = [&](int i) {               // page of block i (-1: none)
      return i < blocks ? __ldg(table + ((key_w + i * (kWarps * kKv8Block)) >> p.page_shift)) : -1;
    };
    auto fetch = [&](int i, int st, int page) {  // block i into stage st
      if (i < blocks) {
        const int key0 = key_w + i * (kWarps * kKv8Block);
        bool ok = page >= 0 && page < p.num_pages;
        if (!ok) {
          if (lane == 0) record_status(p.status, kStatusPageTable);
          page = 0;
        }
        // first row of the block among the pool's rows
        const long long row = ((static_cast<long long>(page) * p.Hkv + hk) << p.page_shift) + (key0 & ((1 << p.page_shift) - 1));
        ok = ok && idx_ok(p.status, row, kKv8Block, pool);
        const uint8_t* ksrc = p.k + (row << kDShift) + lane * 16;
        const uint8_t* vsrc = p.v + (row << kDShift) + lane * 16;
        const uint32_t dst = ring + st * R::kStage;
        if (ok && key0 + kKv8Block <= hi) {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint32_t at = dst + ring_off<D>((j * 32 + lane) / (D / 16), lane % (D / 16));
            cp16(at, ksrc + j * 512);
            cp16(at + R::kBlock, vsrc + j * 512);
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const int r = (j * 32 + lane) / (D / 16);
            const uint32_t at = dst + ring_off<D>(r, lane % (D / 16));
            cp16_or_zero(at, ksrc + j * 512, ok && key0 + r < hi);
            cp16_or_zero(at + R::kBlock, vsrc + j * 512, ok && key0 + r < hi);
          }
        }
        if (lane < 2) cp4_or_zero(ring_s + st * 16 + lane * 4, (lane ? p.vs : p.ks) + (row >> 4), ok);
      }
      cp_commit();
    };
    int next = page_of(0);
    for (int i = 0; i < kStages - 1; ++i) {
      const int page = next;
      next = page_of(i + 1);
      fetch(i, i, page);
    }

    // queries: B operand, row 8 n + g, 16 values from d = 16 (t + 4 c); the scales of the rows 8 n + 2 t + e that
    // this lane holds in the accumulators come from the lanes that read them
    uint32_t qb[NG][LD][4][2];
    float qs[NG][2];
    int lim[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int row = row0 + 8 * n + g;
      const bool in = row < rows;
      const size_t at = o_row(p, b, hk, in ? row : row0) * D;
      uint32_t w[LD][8];
#pragma unroll
      for (int c = 0; c < LD; ++c) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at + 16 * (t + 4 * c));
        const bool ok = in && idx_ok(p.status, at + 16 * (t + 4 * c), 16, outs * D);
        const uint4 x = ok ? __ldg(src) : make_uint4(0, 0, 0, 0), y = ok ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
        w[c][0] = x.x; w[c][1] = x.y; w[c][2] = x.z; w[c][3] = x.w;
        w[c][4] = y.x; w[c][5] = y.y; w[c][6] = y.z; w[c][7] = y.w;
      }
      float down = p.scale_log2;
      if constexpr (!kFp16) {
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < LD; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = unpack2<false>(w[c][j]);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112), 126);
        const float up = pow2i(14 - e);
        down *= pow2i(e - 14);
#pragma unroll
        for (int c = 0; c < LD; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = unpack2<false>(w[c][j]);
            w[c][j] = pack2<true>(f.x * up, f.y * up);
          }
      }
#pragma unroll
      for (int c = 0; c < LD; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // the four values that a word of K meets, in the order of halves_of
          qb[n][c][j][0] = kInt8 ? __byte_perm(w[c][2 * j], w[c][2 * j + 1], 0x5410) : w[c][2 * j];
          qb[n][c][j][1] = kInt8 ? __byte_perm(w[c][2 * j], w[c][2 * j + 1], 0x7632) : w[c][2 * j + 1];
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = row0 + 8 * n + 2 * t + e;
        qs[n][e] = __shfl_sync(0xffffffffu, down, (2 * t + e) * 4);
        lim[n][e] = r < rows ? min(row_limit(p, len, r), hi) : 0;
      }
    }

    float o[NG][MT][4];
    float m[NG][2], mo[NG][2], l[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
      m[n][0] = m[n][1] = mo[n][0] = mo[n][1] = kNone;
      l[n][0] = l[n][1] = 0.f;
    }

    int st = 0, st_in = kStages - 1;  // stages of block i and of block i + kStages - 1
    for (int i = 0; i < blocks; ++i) {
      {
        const int page = next;
        next = page_of(i + kStages);
        fetch(i + kStages - 1, st_in, page);
      }
      cp_wait<kStages - 1>();
      __syncwarp();
      const uint32_t kb = ring + st * R::kStage, vb = kb + R::kBlock;
      float ks, vs;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs) : "r"(ring_s + st * 16) : "memory");
      const int key0 = key_w + i * (kWarps * kKv8Block);

      // S^T: element e of accumulator n: key g + 8 (e >> 1), row 8 n + 2 t + (e & 1)
      float sc[NG][4] = {};
#pragma unroll
      for (int c = 0; c < LD; ++c) {
        const uint4 x = lds128(kb + ring_off<D>(g, t + 4 * c)), y = lds128(kb + ring_off<D>(g + 8, t + 4 * c));
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0, a1, a2, a3;
          halves_of<kInt8>(xw[j], a0, a2);
          halves_of<kInt8>(yw[j], a1, a3);
#pragma unroll
          for (int n = 0; n < NG; ++n) mma_f16(sc[n], a0, a1, a2, a3, qb[n][c][j][0], qb[n][c][j][1]);
        }
      }

      const bool edge = key0 + kKv8Block > min(tile_all, hi);
      const float lv = lg2(fmaxf(vs, 1.17549435e-38f));  // a scale of zero stands for values of zero
      uint32_t wb[NG][2];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const float f[2] = {qs[n][0] * ks, qs[n][1] * ks};
        if (edge) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + g + 8 * (e >> 1) >= lim[n][e & 1]) sc[n][e] = -INFINITY;
        }
        // the maxima are raised when a score of any lane passes them by more than 2^8 (rare after a few blocks)
        float mx[2];
        bool past = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float top = fmaxf(sc[n][e], sc[n][2 + e]);
          mx[e] = top == -INFINITY ? -INFINITY : top * f[e];  // (-inf stays what it is where the scale is zero)
          past |= mx[e] > fminf(m[n][e], mo[n][e] - lv) + kLazy;
        }
        if (__any_sync(0xffffffffu, past)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int s2 = 4; s2 <= 16; s2 <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], s2));
            if (mx[e] > m[n][e]) {
              l[n][e] *= ex2(m[n][e] - mx[e]);
              m[n][e] = mx[e];
            }
            const float mv = mx[e] + lv;
            if (mv > mo[n][e]) {
              const float a = ex2(mo[n][e] - mv);
#pragma unroll
              for (int i2 = 0; i2 < MT; ++i2) {
                o[n][i2][e] *= a;
                o[n][i2][2 + e] *= a;
              }
              mo[n][e] = mv;
            }
          }
        }
        float p2[4], w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p2[e] = fmaf(sc[n][e], f[e & 1], -m[n][e & 1]);
          w[e] = fmaf(sc[n][e], f[e & 1], lv - mo[n][e & 1]);
        }
        if (edge) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (sc[n][e] == -INFINITY) p2[e] = w[e] = -INFINITY;
        }
        l[n][0] += ex2(p2[0]) + ex2(p2[2]);
        l[n][1] += ex2(p2[1]) + ex2(p2[3]);
        wb[n][0] = transpose8x8(pack2<true>(ex2(w[0]), ex2(w[1])));  // keys 0..7 of the block
        wb[n][1] = transpose8x8(pack2<true>(ex2(w[2]), ex2(w[3])));  // keys 8..15
      }

      // O^T += V^T W^T: this lane's keys 2t, 2t + 1 of both halves of the block, D / 8 columns from d = (D / 8) g;
      // tile i: its rows g and g + 8 are the columns 2 i and 2 i + 1 of those
      uint32_t v[4][D / 32];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = (k >> 1) * 8 + 2 * t + (k & 1);
        if constexpr (D == 128) {
          const uint4 x = lds128(vb + ring_off<D>(r, g));
          v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
        } else {
          const uint2 x = lds64(vb + ring_off<D>(r, g >> 1) + (g & 1) * 8);
          v[k][0] = x.x; v[k][1] = x.y;
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t a0, a1, a2, a3;
        halves_of<kInt8>(pair_bytes<kInt8, 0>(v[0][w], v[1][w]), a0, a1);
        halves_of<kInt8>(pair_bytes<kInt8, 0>(v[2][w], v[3][w]), a2, a3);
#pragma unroll
        for (int n = 0; n < NG; ++n) mma_f16(o[n][2 * w], a0, a1, a2, a3, wb[n][0], wb[n][1]);
        halves_of<kInt8>(pair_bytes<kInt8, 1>(v[0][w], v[1][w]), a0, a1);
        halves_of<kInt8>(pair_bytes<kInt8, 1>(v[2][w], v[3][w]), a2, a3);
#pragma unroll
        for (int n = 0; n < NG; ++n) mma_f16(o[n][2 * w + 1], a0, a1, a2, a3, wb[n][0], wb[n][1]);
      }
      st_in = st;
      st = st + 1 == kStages ? 0 : st + 1;
      __syncwarp();  // every lane has read the stage before the next fetch writes it
    }
    cp_wait<0>();
    __syncthreads();

    // merge of the four warps through shared memory: O [warp][row][d], then m, l, mo [warp][row]; a row's
    // factors (one per warp) and its place take the room of the latter
    float* ro = reinterpret_cast<float*>(smem);
    float* rm = ro + kWarps * kRows * D;
    float* rl = rm + kWarps * kRows;
    float* rw = rl + kWarps * kRows;
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
#pragma unroll
        for (int s2 = 4; s2 <= 16; s2 <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s2);
        const int row = warp * kRows + 8 * n + 2 * t + e;
        if (g == 0) {
          rm[row] = m[n][e];
          rl[row] = sum;
          rw[row] = mo[n][e];
        }
#pragma unroll
        for (int i = 0; i < MT; i += 2)
          *reinterpret_cast<float4*>(ro + merge_at<D>(row, (D / 8) * g + 2 * i)) =
              make_float4(o[n][i][e], o[n][i][2 + e], o[n][i + 1][e], o[n][i + 1][2 + e]);
      }
    __syncthreads();
    const int slot = 2 * blockIdx.x + (u.g0 == 0 ? 1 : 0);  // of a piece
    if (tid < kRows && row0 + tid < rows) {
      const int rr = row0 + tid;
      float M = kNone, W = kNone, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        M = fmaxf(M, rm[w * kRows + tid]);
        W = fmaxf(W, rw[w * kRows + tid]);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += ex2(rm[w * kRows + tid] - M) * rl[w * kRows + tid];
      const bool none = M == kNone;
      const float f = none ? 0.f : ex2(W - M) / sum;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) rw[w * kRows + tid] = ex2(rw[w * kRows + tid] - W) * f;
      const float ls = none ? -INFINITY : (M + lg2(sum)) * kLn2;
      if (whole) {
        const size_t at = lse_row(p, b, hk, rr);
        if (idx_ok(p.status, at, 1, outs)) p.lse[at] = ls;
        reinterpret_cast<int*>(rl)[tid] = static_cast<int>(o_row(p, b, hk, rr));  // (below 2^31)
      } else if (idx_ok(p.status, static_cast<long long>(slot) * kRows + tid, 1, 2LL * gridDim.x * kRows)) {
        p.ws_l[static_cast<size_t>(slot) * kRows + tid] = ls;
      }
    }
    __syncthreads();
    for (int i = tid; i < min(kRows, rows - row0) * (D / 4); i += kThreads) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = rw[w * kRows + row];
        const float4 y = *reinterpret_cast<const float4*>(ro + merge_at<D>(w * kRows + row, d));
        x.x = fmaf(f, y.x, x.x);
        x.y = fmaf(f, y.y, x.y);
        x.z = fmaf(f, y.z, x.z);
        x.w = fmaf(f, y.w, x.w);
      }
      if (whole) {
        const size_t at = static_cast<size_t>(reinterpret_cast<const int*>(rl)[row]);
        if (!idx_ok(p.status, at, 1, outs)) continue;
        store2<kFp16>(p.o, at * D + d, x.x, x.y, o_fp32 != 0);
        store2<kFp16>(p.o, at * D + d + 2, x.z, x.w, o_fp32 != 0);
      } else {
        const size_t at = static_cast<size_t>(slot) * kRows + row;
        if (idx_ok(p.status, at, 1, 2LL * gridDim.x * kRows)) *reinterpret_cast<float4*>(p.ws_o + at * D + d) = x;
      }
    }
    __syncthreads();  // the merge buffers are the ring of the next unit
  }
}

// Merges the pieces of the units that lie in more than one share.  CTA i looks at the border between
// shares i and i + 1 and takes the unit it cuts, if no earlier border cuts the same one: piece 0 is the
// end of share i, the others are the beginnings of shares i + 1, i + 2, ...  O = sum_s exp(lse_s - M) o_s /
// sum_s exp(lse_s - M), LSE = M + ln of that sum; one warp per row.
template <bool kFp16, int D, int NG>
__global__ void __launch_bounds__(kThreads) kv8_combine_kernel(const AttParams p, const int o_fp32, const int grid) {
  constexpr int kRows = 8 * NG, PER = D / 32, RPW = 2 * NG;  // rows of a warp, all under way at once
  __shared__ ScanMem scan;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x + 1;
  const Place place = find_place<kRows>(p, grid, c, scan);
  if (place.b < 0) return;
  const int shares = shares_of(p, place.total, grid);
  const Unit u = unit_at<kRows>(p, keys_of(p, place.b), place.off);
  const long long begin = share_begin(place.total, shares, c) - u.r, end = begin + u.n + p.over;
  if (u.g0 == 0 || share_begin(place.total, shares, c - 1) > begin + p.over) return;
  int pieces = 1;  // beside the first
  while (c + pieces < shares && share_begin(place.total, shares, c + pieces) < end) ++pieces;
  auto slot = [&](int s) { return static_cast<size_t>(s == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + s)) * kRows; };
  const int rows = min(kRows, p.Nq * p.group - u.tile * kRows);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are written

  float M[RPW], sum[RPW], acc[RPW][PER];
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    M[i] = kNone;
    sum[i] = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[i][e] = 0.f;
  }
  for (int s = 0; s <= pieces; ++s)
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int row = warp + i * kWarps;
      if (row < rows) M[i] = fmaxf(M[i], p.ws_l[slot(s) + row] * kLog2e);
    }
  for (int s = 0; s <= pieces; ++s)
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int row = warp + i * kWarps;
      if (row >= rows) continue;
      const float w = ex2(p.ws_l[slot(s) + row] * kLog2e - M[i]);
      sum[i] += w;
      const float2* x = reinterpret_cast<const float2*>(p.ws_o + (slot(s) + row) * D) + lane * (PER / 2);
#pragma unroll
      for (int e = 0; e < PER / 2; ++e) {
        const float2 y = x[e];
        acc[i][2 * e] = fmaf(w, y.x, acc[i][2 * e]);
        acc[i][2 * e + 1] = fmaf(w, y.y, acc[i][2 * e + 1]);
      }
    }
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    const int row = warp + i * kWarps, rr = u.tile * kRows + row;
    if (row >= rows) continue;
    const bool none = M[i] == kNone;
    const float inv = none ? 0.f : 1.f / sum[i];
    const size_t at = o_row(p, place.b, u.hk, rr);
    if (!idx_ok(p.status, at, 1, static_cast<long long>(p.B) * p.Nq * p.Hq)) continue;
#pragma unroll
    for (int e = 0; e < PER / 2; ++e)
      store2<kFp16>(p.o, at * D + lane * PER + 2 * e, acc[i][2 * e] * inv, acc[i][2 * e + 1] * inv, o_fp32 != 0);
    if (lane == 0) p.lse[lse_row(p, place.b, u.hk, rr)] = none ? -INFINITY : (M[i] + lg2(sum[i])) * kLn2;
  }
}

// Rows of a tile, in groups of eight: as many tiles as 32 rows each take, of even size.
int groups_for(int Nq, int group) {
  const long long all = (static_cast<long long>(Nq) * group + 7) / 8, tiles = (all + 3) / 4;
  return static_cast<int>((all + tiles - 1) / tiles);
}

template <bool kFp16, bool kInt8, int D, int NG>
int launch_t(const Attend8Args& a, AttParams& p, cudaStream_t stream) {
  using R = Ring<D, NG>;
  constexpr int kCtas = kPerSm<NG> * kSms;
  auto kern = kv8_attend_kernel<kFp16, kInt8, D, NG>;
  static PerContext<int> configured;
  int unused = 0;
  const int ce = configured.get(
      &unused, [&](int*) { return static_cast<int>(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem)); });
  if (ce != 0) return ce;
  p.tiles = static_cast<int>((static_cast<long long>(a.Nq) * p.group + R::kRows - 1) / R::kRows);
  p.ws_o = static_cast<float*>(a.ws);
  p.ws_l = p.ws_o + static_cast<size_t>(2) * kCtas * R::kRows * D;
  const long long cap = static_cast<long long>(a.c.pages_per_seq) * a.c.page_size;
  p.granule = cap <= kShortKeys ? kShortKeys : kGranule;
  p.over = p.granule == kGranule ? kUnitCost : 0;
  // no more CTAs than the fullest tables could give work to
  const long long most = ((cap + p.granule - 1) / p.granule + p.over) * p.B * p.Hkv * p.tiles;
  const int grid = static_cast<int>(std::min<long long>(kCtas, p.over ? (most + kMinShare - 1) / kMinShare : most));
  kern<<<grid, kThreads, R::kSmem, stream>>>(p, a.o_fp32);
  if (p.granule == kGranule && grid > 1) {
    // launched while the first kernel still runs: it finds its place meanwhile and waits for the pieces
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid - 1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_combine_kernel<kFp16, D, NG>, static_cast<const AttParams&>(p), static_cast<int>(a.o_fp32), grid);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  return static_cast<int>(cudaGetLastError());
}

template <bool kFp16, bool kInt8, int D>
int launch_rows(const Attend8Args& a, AttParams& p, cudaStream_t stream) {
  switch (groups_for(a.Nq, p.group)) {
    case 1: return launch_t<kFp16, kInt8, D, 1>(a, p, stream);
    case 2: return launch_t<kFp16, kInt8, D, 2>(a, p, stream);
    case 3: return launch_t<kFp16, kInt8, D, 3>(a, p, stream);
    default: return launch_t<kFp16, kInt8, D, 4>(a, p, stream);
  }
}

}  // namespace

size_t kv8_attend_ws_bytes(int B, int Nq, int Hq, int Hkv, int D) {
  const int n = groups_for(Nq, Hq / Hkv), per_sm = n == 1 ? kPerSm<1> : n == 2 ? kPerSm<2> : n == 3 ? kPerSm<3> : kPerSm<4>;
  return static_cast<size_t>(2) * per_sm * kSms * 8 * n * (D + 1) * sizeof(float);
}

int launch_kv8_attend(const Attend8Args& a, cudaStream_t stream) {
  AttParams p;
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
  if (a.c.D == 64) {
    if (a.c.int8) return a.fp16 ? launch_rows<true, true, 64>(a, p, stream) : launch_rows<false, true, 64>(a, p, stream);
    return a.fp16 ? launch_rows<true, false, 64>(a, p, stream) : launch_rows<false, false, 64>(a, p, stream);
  }
  if (a.c.int8) return a.fp16 ? launch_rows<true, true, 128>(a, p, stream) : launch_rows<false, true, 128>(a, p, stream);
  return a.fp16 ? launch_rows<true, false, 128>(a, p, stream) : launch_rows<false, false, 128>(a, p, stream);
}

}  // namespace fa
