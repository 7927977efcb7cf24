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
// O has a maximum of its own: its weights carry the value scales, so their rounding to fp16 is relative to the largest
// contribution whatever the scales are, and nothing overflows: 11 significant bits down to 2^-21 of the largest one, fewer
// down to 2^-32 (kHead).  mo is kept as dm = mo - m and a weight taken as 2^((s_j - m) + (log2 vs(j) - dm)), from the very s_j - m
// that the row sum takes: with an mo of its own, rounded at the size of the scores, the two drift apart by half a step of
// the score (O 4 % off at scores of 10^6).  At the end O * 2^dm / l.  Both maxima are raised lazily (by more than 2^8 only).
//
// Rows: the G = Hq / Hkv query heads of a KV head times the Nq tokens, token-major, in tiles of 8, 16, 24 or 32:
// keys are the M of the warp MMAs and rows their N, so that few rows waste little of the tensor pipe (16 keys
// against 8 rows take 138 of its cycles, against an M of 16 rows 275):
//   S^T [16 keys x 8 rows]   = K [16 keys x D] Q^T,   O^T [D x 8 rows] += V^T [D x 16 keys] W^T [16 keys x 8 rows];
// the weights go from the accumulator's layout to the operand's with a movmatrix.
// Work is cut evenly over the CTAs (three per SM for up to 16 rows, else two), whatever the lengths are:
// the granules (64 keys) of all units (sequence, row tile, KV head) are numbered through, with a few more
// for each unit's fixed cost, and CTA c takes the c-th equal share, which may begin and end inside a unit,
// and finds its place with a scan over the lengths.  A unit that lies in one share is written at once; the pieces of the others go to the
// workspace (at most two per CTA) and are merged in order by a second kernel.  Warp w of the four takes every
// fourth block of 16 keys: a block has one scale per pool and lies in one page, so a warp needs nothing
// from the others until the end of a unit.  It streams its blocks (16 x D bytes of K and of V, contiguous in a
// page) through a ring of its own in shared memory with 16-byte cp.async, keys past the end filled with
// zeros, and reads them back as 16-byte (K) and 16- or 8-byte (V) pieces of a row: which k slot of an
// MMA a value takes is free as long as both operands agree, so no transposition is needed but of the
// byte pairs of V (two PRMT per eight codes).  The ring's 16-byte chunks are swizzled so that both reads
// are free of bank conflicts.  Warps and pieces are merged by their (m, l, mo, O).
// What bounds it: up to 16 rows the reads (4 x 131072 keys, 32 heads, int8: 178 us, 6.0 TB/s, e4m3 182; without
// any arithmetic 164 us), above that the instructions of two warps per scheduler, which depend on one another from the first
// product over the softmax to the second (24 rows: about 430 instructions for a block of 16 keys, one every 1170 cycles
// on a scheduler, so 2340 for each of its two warps; neither fewer matrix products nor fewer conversions or exponentials
// make it shorter).
#include <algorithm>

#include "fa_internal.h"
#include "fa_kv8.h"
#include "fa_kv8_sched.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kGranule = 64;  // keys
constexpr int kUnitCost = 4;  // granules that a unit's fixed cost stands for (2 and 8: 102 and 96 us where 4 takes 94, B64 ragged 8192)
constexpr int kMinShare = 8;
constexpr int kWholeKeys = 1024;  // tables up to this many keys: a granule is a whole unit, nothing is merged
constexpr int kManyPieces = 16;  // CTAs per unit from which on tiles of up to 16 rows are merged by many CTAs (32: 4 x 32768 keys,
                                 // 4 heads 37 us where 16 takes 34; 24 rows, 8 x 20221: 39 us with them, 33 without)
constexpr int kWarpRows = 64;  // more rows per KV head than this take the tcgen05 kernel (B8, 8 KV heads, D 128; 40 rows,
                               // 8192 keys: 85 us here, 107 there; 64, 4096: 65 and 67; 96, 2048: 58 and 52)

// CTAs per SM for tiles of NG * 8 rows (O takes 32 registers per eight rows at D = 128), and the ring.  Four of
// one group left 128 registers and less overlap inside a warp: 200 us where three took 193 (4 x 131072, int8).
template <int D, int NG>
struct Ring {
  static constexpr int kPerSm = NG <= 2 ? 3 : 2;
  static constexpr int kRows = 8 * NG;
  static constexpr bool kQSmem = NG >= 2;       // their registers are needed for O (with registers 71 us where this takes 64: 64 rows, 4096 keys, B8)
  static constexpr int kBlock = kKv8Block * D;  // bytes of 16 keys of K or V
  static constexpr int kStage = 2 * kBlock;
  static constexpr int kQ = kQSmem ? kRows * (D * 2 + 4) : 0;
  static constexpr int kRoom = (227 * 1024 / kPerSm - 2048 - kQ) / kWarps - 128;
  static constexpr int kStages = kRoom / kStage < 8 ? kRoom / kStage : 8;
  static constexpr int kWarp = kStages * kStage + 128;  // the stages, then (ks, vs) of each, 16 bytes apart
  static constexpr int kMerge = kWarps * kRows * (D + 3) * 4;
  static constexpr int kRings = kWarps * kWarp > kMerge ? kWarps * kWarp : kMerge;
  static constexpr int kSmem = kRings + kQ;
  static_assert(kStages >= 3 && kStages * 16 <= 128, "stages, and their scales");
  static_assert(kPerSm * (kSmem + 2048) <= 227 * 1024 + 1024, "room");
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
// per warp and pair), int8 codes (0, 2) and (1, 3): code + 128 in the mantissa of 1024, less 1152, all exact
// (three byte permutes and logic operations per word; with masks and shifts five, and 194 us where 4 x 131072 take 176).
template <bool kInt8>
__device__ __forceinline__ void halves_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kInt8) {
    w ^= 0x80808080u;
    lo = __byte_perm(w, 0x64646464u, 0x4240);
    hi = __byte_perm(w, 0x64646464u, 0x4341);
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool kFp16, bool kInt8, int D, int NG>
__global__ void __launch_bounds__(kThreads, Ring<D, NG>::kPerSm) kv8_attend_kernel(const __grid_constant__ AttParams p, const int o_fp32) {
  using R = Ring<D, NG>;
  constexpr int kRows = R::kRows, kStages = R::kStages;
  constexpr int LD = D / 64;  // 16-byte pieces of a K row per lane
  constexpr int MT = D / 16;  // 16-column tiles of O (M of the second product)
  constexpr int kDShift = D == 128 ? 7 : 6;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ScanMem<kThreads> scan;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rows = p.Nq * p.group;
  const long long outs = static_cast<long long>(p.B) * p.Nq * p.Hq;
  const long long pool = (static_cast<long long>(p.num_pages) * p.Hkv) << p.page_shift;

  asm volatile("griddepcontrol.launch_dependents;");
  const Place place = find_place<kRows, kThreads>(p, gridDim.x, blockIdx.x, scan);
  if (place.short_items) write_tiles_without_keys<kFp16, D, kRows>(p, o_fp32);
  if (place.b < 0) return;
  Walk walk = walk_of(p, place, gridDim.x, blockIdx.x);

  const uint8_t* own_ring = smem + warp * R::kWarp;
  const uint32_t ring = smem_addr(own_ring), ring_s = ring + kStages * R::kStage;

  Piece pc;
  while (next_piece<kRows>(p, walk, pc)) {
    const int b = pc.b, hk = pc.hk, row0 = pc.row0, len = pc.len, lo = pc.lo, hi = pc.hi;
    const bool whole = pc.whole;
    const int tile_all = row_limit(p, len, row0);  // keys that every row of the tile sees

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

    // queries: B operand, row 8 n + g, 16 values from d = 16 (t + 4 c); in the order of halves_of, a word of K meets
    // four values.  In registers, or (large tiles) in shared memory, as 16 bytes for each lane.
    uint4* qsm = reinterpret_cast<uint4*>(smem + R::kRings);
    float* qscale = reinterpret_cast<float*>(smem + R::kRings + kRows * D * 2);
    uint4 qb[R::kQSmem ? 1 : NG][LD][2];
    float qs[NG][2];
    int lim[NG][2];
    auto load_q = [&](int n, uint4 (&out)[LD][2]) {  // returns the factor that a score of row 8 n + g takes
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
        for (int j = 0; j < 2; ++j) {
          const uint32_t *x = w[c] + 4 * j;
          out[c][j] = kInt8 ? make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                                         __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[2], x[3], 0x7632))
                            : make_uint4(x[0], x[1], x[2], x[3]);
        }
      return down;
    };
    if constexpr (R::kQSmem) {
      if (warp < NG) {
        const float down = load_q(warp, qb[0]);
#pragma unroll
        for (int c = 0; c < LD; ++c)
#pragma unroll
          for (int j = 0; j < 2; ++j) qsm[((warp * LD + c) * 2 + j) * 32 + lane] = qb[0][c][j];
        if (t == 0) qscale[8 * warp + g] = down;
      }
      __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      float down = 0.f;
      if constexpr (!R::kQSmem) down = load_q(n, qb[n]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // the rows that this lane holds in the accumulators
        const int r = 8 * n + 2 * t + e;
        if constexpr (R::kQSmem) qs[n][e] = qscale[r];
        else qs[n][e] = __shfl_sync(0xffffffffu, down, (2 * t + e) * 4);
        lim[n][e] = row0 + r < rows ? min(row_limit(p, len, row0 + r), hi) : 0;
      }
    }

    float o[NG][MT][4];
    float m[NG][2], dm[NG][2], l[NG][2];  // dm: mo - m - kHead (before the first key any finite number)
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
      m[n][0] = m[n][1] = kNone;
      dm[n][0] = dm[n][1] = 0.f;
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
      const uint8_t *kb = own_ring + st * R::kStage, *vb = kb + R::kBlock;
      const float2 kvs = *reinterpret_cast<const float2*>(own_ring + kStages * R::kStage + st * 16);
      const float ks = kvs.x, vs = kvs.y;
      const int key0 = key_w + i * (kWarps * kKv8Block);

      // S^T: element e of accumulator n: key g + 8 (e >> 1), row 8 n + 2 t + (e & 1)
      float sc[NG][4] = {};
#pragma unroll
      for (int c = 0; c < LD; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(kb + ring_off<D>(g, t + 4 * c)), y = *reinterpret_cast<const uint4*>(kb + ring_off<D>(g + 8, t + 4 * c));
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t a[2][4];
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            halves_of<kInt8>(xw[2 * j + i2], a[i2][0], a[i2][2]);
            halves_of<kInt8>(yw[2 * j + i2], a[i2][1], a[i2][3]);
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const uint4 q = R::kQSmem ? qsm[((n * LD + c) * 2 + j) * 32 + lane] : qb[R::kQSmem ? 0 : n][c][j];
            mma_f16(sc[n], a[0][0], a[0][1], a[0][2], a[0][3], q.x, q.y);
            mma_f16(sc[n], a[1][0], a[1][1], a[1][2], a[1][3], q.z, q.w);
          }
        }
      }

      const bool edge = key0 + kKv8Block > min(tile_all, hi);
      const float lv = log2_scale(vs);
      uint32_t wb[NG][2];
      float f[NG][2], mx[NG][2];
      bool past = false;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        if (edge) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + g + 8 * (e >> 1) >= lim[n][e & 1]) sc[n][e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[n][e] = qs[n][e] * ks;
          const float top = fmaxf(sc[n][e], sc[n][2 + e]);
          mx[n][e] = top == -INFINITY ? -INFINITY : top * f[n][e];  // (-inf stays what it is where the scale is zero)
          past |= mx[n][e] > m[n][e] + fminf(kLazy, dm[n][e] - (lv - (kHead + kLazy)));
        }
      }
      // the maxima are raised when a score of any lane passes them by more than 2^8 (rare after a few blocks; one vote for
      // all rows, so that everything behind it is straight code)
      if (__any_sync(0xffffffffu, past)) {
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = mx[n][e];
#pragma unroll
            for (int s2 = 4; s2 <= 16; s2 <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s2));
            if (top > m[n][e]) {  // (mo stays what it is)
              const float by = m[n][e] - top;
              l[n][e] *= ex2(by);
              dm[n][e] += by;
              m[n][e] = top;
            }
            const float mv = (top - m[n][e]) + (lv - kHead);
            if (mv > dm[n][e]) {
              const float a = ex2(dm[n][e] - mv);
#pragma unroll
              for (int i2 = 0; i2 < MT; ++i2) {
                o[n][i2][e] *= a;
                o[n][i2][2 + e] *= a;
              }
              dm[n][e] = mv;
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float p2[4], w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p2[e] = fmaf(sc[n][e], f[n][e & 1], -m[n][e & 1]);
        if (edge) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (sc[n][e] == -INFINITY) p2[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = p2[e] + (lv - dm[n][e & 1]);
        l[n][0] += ex2(p2[0]) + ex2(p2[2]);
        l[n][1] += ex2(p2[1]) + ex2(p2[3]);
        wb[n][0] = transpose8x8(pack_weights(ex2(w[0]), ex2(w[1])));  // keys 0..7 of the block
        wb[n][1] = transpose8x8(pack_weights(ex2(w[2]), ex2(w[3])));  // keys 8..15
      }

      // O^T += V^T W^T: this lane's keys 2t, 2t + 1 of both halves of the block, D / 8 columns from d = (D / 8) g;
      // tile i: its rows g and g + 8 are the columns 2 i and 2 i + 1 of those
      uint32_t v[4][D / 32];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = (k >> 1) * 8 + 2 * t + (k & 1);
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(vb + ring_off<D>(r, g));
          v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(vb + ring_off<D>(r, g >> 1) + (g & 1) * 8);
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

    // merge of the four warps through shared memory: O [warp][row][d], then m, l, dm [warp][row]; a row's
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
          rw[row] = dm[n][e];
        }
#pragma unroll
        for (int i = 0; i < MT; i += 2)
          *reinterpret_cast<float4*>(ro + merge_at<D>(row, (D / 8) * g + 2 * i)) =
              make_float4(o[n][i][e] * kUnhead, o[n][i][2 + e] * kUnhead, o[n][i + 1][e] * kUnhead, o[n][i + 1][2 + e] * kUnhead);
      }
    __syncthreads();
    const int slot = 2 * blockIdx.x + pc.slot;
    if (tid < kRows && row0 + tid < rows) {
      const int rr = row0 + tid;
      float M = kNone, W = kNone, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, rm[w * kRows + tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {  // mo - M of each warp, and the largest
        const float d = rw[w * kRows + tid] += rm[w * kRows + tid] - M;
        W = fmaxf(W, d);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += ex2(rm[w * kRows + tid] - M) * rl[w * kRows + tid];
      const bool none = sum == 0.f;  // (not by M: scores of NaN leave that where it was)
      const float f = none ? 0.f : ex2(W + kHead) / sum;
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

// Which kernel takes a call, by its rows per KV head.
bool on_chunk_kernel(int Nq, int group) { return static_cast<long long>(Nq) * group > kWarpRows; }

// Rows of a tile, in groups of eight: as many tiles as 32 rows each take, of even size.
int groups_for(int Nq, int group) {
  const long long all = (static_cast<long long>(Nq) * group + 7) / 8, tiles = (all + 3) / 4;
  return static_cast<int>((all + tiles - 1) / tiles);
}

template <bool kFp16, bool kInt8, int D, int NG>
int launch_t(const Attend8Args& a, AttParams& p, cudaStream_t stream) {
  using R = Ring<D, NG>;
  constexpr int kCtas = R::kPerSm * kSms;
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
  p.granule = cap <= kWholeKeys ? kWholeKeys : kGranule;
  p.over = p.granule == kGranule ? kUnitCost : 0;
  p.least = p.over ? kMinShare : 1;
  // no more CTAs than the fullest tables could give work to
  const long long most = ((cap + p.granule - 1) / p.granule + p.over) * p.B * p.Hkv * p.tiles;
  const int grid = static_cast<int>(std::min<long long>(kCtas, (most + p.least - 1) / p.least));
  kern<<<grid, kThreads, R::kSmem, stream>>>(p, a.o_fp32);
  if (p.over && grid > 1) {
    const bool many = NG <= 2 && static_cast<long long>(p.B) * p.Hkv * p.tiles * kManyPieces <= grid;
    const int e = many ? launch_combine8<kFp16, D, R::kRows, NG <= 2>(p, a.o_fp32, grid, stream)
                       : launch_combine8<kFp16, D, R::kRows>(p, a.o_fp32, grid, stream);
    if (e != 0) return e;
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
  if (on_chunk_kernel(Nq, Hq / Hkv)) return kv8_chunk_ws_bytes(D);
  const int n = groups_for(Nq, Hq / Hkv), per_sm = n <= 2 ? Ring<128, 1>::kPerSm : Ring<128, 3>::kPerSm;
  return static_cast<size_t>(2) * per_sm * kSms * 8 * n * (D + 1) * sizeof(float);
}

int launch_kv8_attend(const Attend8Args& a, cudaStream_t stream) {
  if (on_chunk_kernel(a.Nq, a.Hq / a.c.Hkv)) return launch_kv8_chunk(a, stream);
  AttParams p = params_of(a);
  if (a.c.D == 64) {
    if (a.c.int8) return a.fp16 ? launch_rows<true, true, 64>(a, p, stream) : launch_rows<false, true, 64>(a, p, stream);
    return a.fp16 ? launch_rows<true, false, 64>(a, p, stream) : launch_rows<false, false, 64>(a, p, stream);
  }
  if (a.c.int8) return a.fp16 ? launch_rows<true, true, 128>(a, p, stream) : launch_rows<false, true, 128>(a, p, stream);
  return a.fp16 ? launch_rows<true, false, 128>(a, p, stream) : launch_rows<false, false, 128>(a, p, stream);
}

}  // namespace fa
