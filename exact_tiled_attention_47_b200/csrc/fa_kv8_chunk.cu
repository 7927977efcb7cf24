// fa_kv8_chunk.cu -- attention over the paged 8-bit cache for many query rows per KV head (chunks of prompts,
// long drafts): the mathematics of fa_kv8_attend.cu on tcgen05 tensor cores.
//
// The scheme is that of the prefill kernel (fa_prefill_sm100.cu): two 128-row Q tiles per CTA, a softmax
// warpgroup and an MMA-issuing thread each, S and O in tensor memory, P in shared memory as the A operand of
// P V, S(j+1) issued as soon as S(j) is in registers.  What differs:
//   - K and V tiles are made by a warpgroup of its own: it loads the codes of 128 keys from their pages with
//     16-byte loads one tile ahead, converts them to fp16 (exact) and stores them where TMA would have put
//     them (128-byte rows, 16-byte chunks XOR-ed with the row).  It also brings the queries to fp16 (bf16
//     rows times a power of two) and the scales to shared memory.
//   - a tile has eight blocks of 16 keys with a scale each.  With f = q scale * ks and the maxima m (of the
//     scores) and mo (of score + log2 vs, less kHead), a weight is w = 2^(s f + log2 vs - mo): one fma and one ex2 as
//     before, with other constants for each block; the row sum takes it back to 2^(s f - m) with the factor
//     2^(mo - m - log2 vs) in the same instruction that adds it.  Where a block's vs is 2^64 or more below
//     the row's largest contribution, that factor could meet a weight that was flushed to zero: then the
//     row sums of the tile are computed from exponentials of their own.
//   - the grid is one CTA per SM and shares the work evenly (fa_kv8_sched.cuh), pieces of cut units are
//     merged by a second kernel.
// Tensor memory: S0 S1 [0, 256), O0 O1 [256, 256 + 2 D).  Warps 0-3 and 4-7: softmax of tile 0 and 1; 8 and 9: MMA
// issue (10 and 11 idle); 12-15: conversion.  16 warps share the registers, so a row of S is never held as a whole: its
// two halves are read for the maxima, the second is turned into weights and stored, the first is read again.
// A step of 128 keys takes about 5800 cycles (1024 tokens behind 15360 cached keys, two sequences: 718 us, 742 TFLOP/s), of
// which the MUFU needs 2180 and the tensor core 2100: what is left is latency inside the softmax warps, of which the
// registers allow two per scheduler.
#include <algorithm>

#include "fa_internal.h"
#include "fa_kv8.h"
#include "fa_kv8_sched.cuh"
#include "fa_prefill_common.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kBM = 128;          // rows of a tile
constexpr int kBN = 128;          // keys of a block
constexpr int kUnitRows = 2 * kBM;
constexpr int kChunkThreads = 512;
constexpr int kMmaWarp = 8;       // owns TMEM; issues the MMAs of tile 0 (warp 9 those of tile 1)
constexpr int kConvWarp = 12;
constexpr uint32_t kTmemCols = 512;
constexpr int kPanelBytes = kBM * 128;  // 64 fp16 columns of a tile
constexpr int kChunkUnitCost = 2;       // blocks that the fixed cost of a unit stands for
constexpr int kChunkWholeKeys = 512;    // tables up to this many keys: a granule is a whole unit, nothing is merged
constexpr int kChunkMinShare = 4;       // (Nq 244, 1 head of each group, 1248 keys, B3: 43 us, with 8 53)
// Registers: launched with kLaunchRegs per thread; the MMA warpgroup gives some to the others.  The sum must not
// exceed the launch allocation, else setmaxnreg.inc would wait forever; the host confirms that allocation once per
// device.  (Of the splits that leave little in local memory this one was the fastest: chunk of 1024 behind 16384
// keys 717 us, with 160 / 56 / 136 727, with 168 / 56 / 120 737.)
constexpr int kLaunchRegs = 128;
constexpr int kSoftmaxRegs = 144;
constexpr int kControlRegs = 80;
constexpr int kConvRegs = 144;
static_assert(2 * kSoftmaxRegs + kControlRegs + kConvRegs <= 4 * kLaunchRegs, "register split");

template <int D>
struct ChunkCfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kBM * D * 2;
  static constexpr int kPBytes = kBM * kBN * 2;
  // D = 128 has room for one K and two V stages beside Q and P (K_{j+1} is needed a whole step after S(j))
  static constexpr int kKStages = D == 64 ? 2 : 1;
  static constexpr int kVStages = 2;
  static constexpr int kKOff = 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kPOff = kVOff + kVStages * kTileBytes;
  static constexpr int kBarOff = kPOff + 2 * kPBytes;
  static constexpr int kSmemBytes = kBarOff + 2048 + 1024;  // barriers, scales; alignment slack
  __device__ static constexpr uint32_t col_s(int t) { return t ? 128u : 0u; }
  __device__ static constexpr uint32_t col_o(int t) { return 256u + (t ? static_cast<uint32_t>(D) : 0u); }
};
static_assert(ChunkCfg<64>::kSmemBytes <= 232448 && ChunkCfg<128>::kSmemBytes <= 232448, "shared memory budget");

struct ChunkBars {
  uint64_t q_full;   // piece s is in piece[s % 2], its queries are in place
  uint64_t q_taken;  // every warp is done with it (so that none falls a phase behind)
  uint64_t k_full[2], v_full[2];
  uint64_t k_empty[2][2], v_empty[2][2];  // [tile][stage]
  uint64_t s_full[2], s_free[2], p_full[2], o_done[2], drain[2];
  uint32_t tmem_base;
  int abort_flag;
  // The pieces, walked by the conversion warps and handed on to the others (no keys left: the end).  With the walk in
  // every warp's registers it was spilled into the inner loops, whose local memory misses the small L1 that the
  // tiles leave: 938 us where this took 710 (chunk of 1024 behind 16384 keys, B2).
  Piece piece[2];
  Walk walk[4];
  union {
    ScanMem<kChunkThreads> scan;  // before the roles part
    struct {
      float2 scale[4][8];              // (ks, log2 vs) of the eight blocks of key block n % 4
      signed char qexp[2][kUnitRows];  // the rows of piece s % 2 were multiplied by 2^-qexp
    };
  };
};
static_assert(sizeof(ChunkBars) <= 2048, "barrier block too large");

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 16 bytes that this SM reads once: not kept in the little L1 that the tiles leave.
__device__ __forceinline__ uint4 ldg_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// D (+)= A B with the operands' descriptors (smem_desc_sw128) as their low words, the high word is common: the
// issuing thread shares its sub-partition with computing warps, so it gets few instructions per MMA.
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Address of 16-byte chunk ch (8 columns) of row r of a tile of 64-column panels, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int r, int ch) {
  return base + (ch >> 3) * kPanelBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// Four codes as two fp16 pairs in memory order.
template <bool kInt8>
__device__ __forceinline__ void halves_in_order(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kInt8) {
    w ^= 0x80808080u;
    lo = __byte_perm(w, 0x64646464u, 0x4140);
    hi = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&lo), off), y = __hsub2(*reinterpret_cast<__half2*>(&hi), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
  }
}

// (ks, log2 vs) of block h of those whose pairs begin at this shared-memory address.
__device__ __forceinline__ float2 scale_at(uint32_t scale, int h) {
  float2 r;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(scale + h * 8));
  return r;
}

// Weights of columns 32 ch ... 32 ch + 31 of 64 (two blocks of keys) of a row, their share of the row sum, packed to fp16.
// kOwnSum: the row sum from exponentials of its own (see above).
// (The prefill's cubic for a part of the exponentials is off by up to 7.5e-5 relative: too much for the fp32 LSE of
// a row that sees few keys, so all of them run on the MUFU here.)
template <bool kOwnSum>
__device__ __forceinline__ void weights32(const uint32_t (&sr)[64], int ch, uint32_t scale, float qs, float m, float mo, uint64_t& acc0,
                                          uint64_t& acc1, uint32_t (&pk)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 sc = scale_at(scale, h);
    const float f = fmaxf(qs * sc.x, 1.17549435e-38f), e = kOwnSum ? -m : sc.y - mo;
    const float d = kOwnSum ? sc.y - (mo - m) : ex2(mo - m - sc.y);
    const uint64_t f2v = f2(f, f), e2v = f2(e, e), d2v = f2(d, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = ch * 32 + h * 16 + 2 * i;
      const uint64_t s2 = f2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
      uint64_t x = f2_fma(s2, f2v, e2v);
      float x0, x1;
      if constexpr (kOwnSum) {  // the weight from the s f - m of the row sum: rounded once, at the size of the score
        f2_split(x, x0, x1);
        acc0 = f2_add(acc0, f2(ex2(x0), ex2(x1)));
        x = f2_add(x, d2v);
      }
      f2_split(x, x0, x1);
      const float p0 = ex2(x0), p1 = ex2(x1);
      const uint64_t pe = f2(p0, p1);
      if constexpr (kOwnSum) {
      } else if (i & 1) {
        acc1 = f2_fma(pe, d2v, acc1);
      } else {
        acc0 = f2_fma(pe, d2v, acc0);
      }
      pk[h * 8 + i] = pack_weights(p0, p1);
    }
  }
}

template <bool kFp16, bool kInt8, int D>
__global__ void __launch_bounds__(kChunkThreads, 1) kv8_chunk_kernel(const __grid_constant__ AttParams p, const int o_fp32) {
  using C = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  ChunkBars* bars = reinterpret_cast<ChunkBars*>(smem + C::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.Nq * p.group;

  asm volatile("griddepcontrol.launch_dependents;");
  const Place place = find_place<kUnitRows, kChunkThreads>(p, gridDim.x, blockIdx.x, bars->scan);
  if (place.short_items) write_tiles_without_keys<kFp16, D, kUnitRows>(p, o_fp32);
  if (place.b < 0) return;  // uniform
  __syncthreads();  // scan and what lies in its place may be written
  if (threadIdx.x < 4) bars->walk[threadIdx.x] = walk_of(p, place, gridDim.x, blockIdx.x);

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 4);
    mbar_init(&bars->q_taken, 10);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->k_full[s], 4);
      mbar_init(&bars->v_full[s], 4);
      for (int t = 0; t < 2; ++t) {
        mbar_init(&bars->k_empty[t][s], 1);
        mbar_init(&bars->v_empty[t][s], 1);
      }
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->s_free[t], 4);
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->o_done[t], 1);
      mbar_init(&bars->drain[t], 1);
    }
    bars->abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;
  volatile int* abort_flag = &bars->abort_flag;
  const uint32_t sQ = smem_addr(smem), sK = sQ + C::kKOff, sV = sQ + C::kVOff, sP = sQ + C::kPOff;
  int n0 = 0;  // key blocks of the pieces before this one

  if (warp >= kConvWarp) {
    if constexpr (kConvRegs > kLaunchRegs) regs_increase<kConvRegs>();
    else if constexpr (kConvRegs < kLaunchRegs) regs_decrease<kConvRegs>();
    // ================================ conversion =================================================
    const int cw = warp - kConvWarp;
    const int r8 = lane >> 2, c4 = lane & 3;  // row of a group of eight, 16-code chunk of a 64-column panel
    const long long pool = (static_cast<long long>(p.num_pages) * p.Hkv) << p.page_shift;
    bool ok = true;
    for (int s = 0; ok; ++s) {
      Piece pc;
      if (lane == 0) {
        if (!next_piece<kUnitRows>(p, bars->walk[cw], pc)) pc.lo = pc.hi = 0;  // the end
        if (cw == 0) bars->piece[s & 1] = pc;  // (piece s - 2 was taken before s - 1 was handed on)
      }
      if (n0 > 0) {  // the MMAs of the piece before must be done with its queries
        const int last = n0 - 1;
        for (int t = 0; t < 2 && ok; ++t)
          ok = warp_wait(&bars->k_empty[t][last % C::kKStages], (last / C::kKStages) & 1, abort_flag, p.status);
      }
      if (!ok) break;
      // Hands the piece on.  Every warp waits for each phase of q_taken before it lets the next one begin.
      auto publish = [&]() {
        if (s > 0 && !warp_wait(&bars->q_taken, (s - 1) & 1, abort_flag, p.status)) return false;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full);
        return true;
      };
      const int lo = __shfl_sync(0xffffffffu, pc.lo, 0), hi = __shfl_sync(0xffffffffu, pc.hi, 0), blocks = (hi - lo + kBN - 1) / kBN;
      if (blocks == 0) {
        publish();
        break;
      }
      pc.b = __shfl_sync(0xffffffffu, pc.b, 0);
      pc.row0 = __shfl_sync(0xffffffffu, pc.row0, 0);
      const int hk = __shfl_sync(0xffffffffu, pc.hk, 0);
      const int* table = p.table + static_cast<long long>(pc.b) * p.pps;
      // Row of the pool where this warp's 16 keys [key0, key0 + 16) lie, -1 if there are none (a bad entry is
      // reported: nothing is read through it).
      auto pool_row = [&](int key0) -> long long {
        if (key0 >= hi) return -1;
        const int page = __ldg(table + (key0 >> p.page_shift));
        if (page < 0 || page >= p.num_pages) {
          if (lane == 0) record_status(p.status, kStatusPageTable);
          return -1;
        }
        const long long row = ((static_cast<long long>(page) * p.Hkv + hk) << p.page_shift) + (key0 & ((1 << p.page_shift) - 1));
        return idx_ok(p.status, row, kKv8Block, pool) ? row : -1;
      };
      long long row[2];            // of this warp's two blocks of 16 keys
      uint4 kx[4][C::kPanels], vx[4][C::kPanels];
      auto load = [&](const uint8_t* src, uint4 (&x)[4][C::kPanels], int key0) {
        const int left = hi - key0 - r8;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn) {
            const long long at = row[i >> 1];
            const int r = (i & 1) * 8 + r8;
            x[i][pn] = make_uint4(0, 0, 0, 0);  // keys past the end: zeros
            if (at >= 0 && i * 8 < left) x[i][pn] = ldg_once(src + (at + r) * D + pn * 64 + c4 * 16);
          }
      };
      auto store = [&](uint32_t tile, const uint4 (&x)[4][C::kPanels]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn) {
            const uint32_t w[4] = {x[i][pn].x, x[i][pn].y, x[i][pn].z, x[i][pn].w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) halves_in_order<kInt8>(w[k], h[2 * k], h[2 * k + 1]);
            const int r = cw * 32 + i * 8 + r8, ch = pn * 8 + c4 * 2;
            sts128(tile_at(tile, r, ch), h[0], h[1], h[2], h[3]);
            sts128(tile_at(tile, r, ch + 1), h[4], h[5], h[6], h[7]);
          }
      };
      float2 sc = make_float2(0.f, 0.f);  // lanes 0 and 1: scales of this warp's two blocks
      auto fetch = [&](int j) {
        const int key0 = lo + j * kBN + cw * 32;
        row[0] = pool_row(key0);
        row[1] = pool_row(key0 + 16);
        load(p.k, kx, key0);
        if (lane < 2) {
          const long long at = lane ? row[1] : row[0];
          sc = make_float2(0.f, 1.f);  // (of a block behind the keys: any that is no extreme)
          if (at >= 0) sc = make_float2(__ldg(p.ks + (at >> 4)), __ldg(p.vs + (at >> 4)));
        }
      };
      // the queries (before the first codes are loaded: both at once would not fit the registers), a tile's 32 rows
      // of this warp at once
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        if (pc.row0 + t * kBM >= rows) break;
        uint32_t w[4][D / 8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = pc.row0 + t * kBM + cw * 32 + i * 8 + r8;
          const bool in = q < rows;
          const size_t at = o_row(p, pc.b, hk, in ? q : pc.row0) * D + c4 * (D / 4);
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const bool rd = in && idx_ok(p.status, at + 8 * k, 8, static_cast<long long>(p.B) * p.Nq * p.Hq * D);
            const uint4 x = rd ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at) + k) : make_uint4(0, 0, 0, 0);
            w[i][4 * k] = x.x; w[i][4 * k + 1] = x.y; w[i][4 * k + 2] = x.z; w[i][4 * k + 3] = x.w;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = cw * 32 + i * 8 + r8;
          int down = 0;
          if constexpr (!kFp16) {
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
              const float2 f = unpack2<false>(w[i][k]);
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112), 126);
            const float up = pow2i(14 - e);
            down = e - 14;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
              const float2 f = unpack2<false>(w[i][k]);
              w[i][k] = pack2<true>(f.x * up, f.y * up);
            }
          }
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            sts128(tile_at(sQ + t * C::kTileBytes, r, c4 * (D / 32) + k), w[i][4 * k], w[i][4 * k + 1], w[i][4 * k + 2], w[i][4 * k + 3]);
          if (c4 == 0) bars->qexp[s & 1][t * kBM + r] = static_cast<signed char>(down);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      fetch(0);
      load(p.v, vx, lo + cw * 32);
      if (!(ok = publish())) break;

      for (int j = 0; j < blocks; ++j) {
        const int n = n0 + j, ks = n % C::kKStages, vs = n % C::kVStages, ku = n / C::kKStages, vu = n / C::kVStages;
        if (ku > 0) {
          for (int t = 0; t < 2 && ok; ++t) ok = warp_wait(&bars->k_empty[t][ks], (ku - 1) & 1, abort_flag, p.status);
          if (!ok) break;
        }
        store(sK + ks * C::kTileBytes, kx);
        if (lane < 2) bars->scale[n & 3][cw * 2 + lane] = make_float2(sc.x, log2_scale(sc.y));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->k_full[ks]);
        if (j + 1 < blocks) fetch(j + 1);
        if (vu > 0) {
          for (int t = 0; t < 2 && ok; ++t) ok = warp_wait(&bars->v_empty[t][vs], (vu - 1) & 1, abort_flag, p.status);
          if (!ok) break;
        }
        store(sV + vs * C::kTileBytes, vx);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->v_full[vs]);
        if (j + 1 < blocks) load(p.v, vx, lo + (j + 1) * kBN + cw * 32);
      }
      n0 += blocks;
    }
  } else if (warp >= 8) {
    regs_decrease<kControlRegs>();
    if (warp < kMmaWarp + 2 && lane == 0) {
      // ================================ MMA issue ================================================
      constexpr uint32_t idesc_qk = instr_desc_f16(kBM, kBN, 0, 0);
      constexpr uint32_t idesc_pv = instr_desc_f16(kBM, D, 0, 1);
      const int t = warp - kMmaWarp;
      // low words of the operands' descriptors (K-major Q, K, P; V with its panels kPanelBytes apart)
      const uint32_t q_lo = static_cast<uint32_t>(smem_desc_sw128(sQ + t * C::kTileBytes, 16, 1024)), k_lo = static_cast<uint32_t>(smem_desc_sw128(sK, 16, 1024));
      const uint32_t p_lo = static_cast<uint32_t>(smem_desc_sw128(sP + t * C::kPBytes, 16, 1024)), v_lo = static_cast<uint32_t>(smem_desc_sw128(sV, kPanelBytes, 1024));
      const uint32_t kDescHi = static_cast<uint32_t>(smem_desc_sw128(0, 16, 1024) >> 32);
      int c0 = 0;  // steps of this tile before this piece
      bool ok = true;
      for (int s = 0; ok; ++s) {
        if (!(ok = mbar_wait(&bars->q_full, s & 1, abort_flag, p.status))) break;
        const int blocks = (bars->piece[s & 1].hi - bars->piece[s & 1].lo + kBN - 1) / kBN;
        const bool mine = bars->piece[s & 1].row0 + t * kBM < rows;
        if (blocks == 0) break;
        mbar_arrive(&bars->q_taken);
        auto wait_k = [&](int j) {
          const int n = n0 + j;
          return mbar_wait(&bars->k_full[n % C::kKStages], (n / C::kKStages) & 1, abort_flag, p.status);
        };
        auto wait_v = [&](int j) {
          const int n = n0 + j;
          return mbar_wait(&bars->v_full[n % C::kVStages], (n / C::kVStages) & 1, abort_flag, p.status);
        };
        if (!mine) {  // no such tile in this unit: its share of the stages is free at once
          for (int j = 0; ok && j < blocks; ++j) {
            if (!(ok = wait_k(j))) break;
            mbar_arrive(&bars->k_empty[t][(n0 + j) % C::kKStages]);
            if (!(ok = wait_v(j))) break;
            mbar_arrive(&bars->v_empty[t][(n0 + j) % C::kVStages]);
          }
          n0 += blocks;
          continue;
        }
        auto issue_s = [&](int j) {
          const int st = (n0 + j) % C::kKStages;
          const uint32_t a = q_lo, b = k_lo + st * (C::kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {  // 16 columns are 32 bytes of a row, 64 a panel
            const uint32_t off = ((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4;
            mma_ss_lo(tbase + C::col_s(t), a + off, b + off, kDescHi, idesc_qk, kk > 0 ? 1u : 0u);
          }
          mma_commit(&bars->s_full[t]);
          mma_commit(&bars->k_empty[t][st]);
        };
        auto issue_pv = [&](int j) {
          const int st = (n0 + j) % C::kVStages;
          const uint32_t a = p_lo, b = v_lo + st * (C::kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk) {  // 16 keys are two 1024-byte atoms of V
            const uint32_t off = ((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4;
            mma_ss_lo(tbase + C::col_o(t), a + off, b + ((kk * 2048) >> 4), kDescHi, idesc_pv, kk > 0 ? 1u : (j > 0 ? 1u : 0u));
          }
          mma_commit(&bars->o_done[t]);
          mma_commit(&bars->v_empty[t][st]);
        };
        if (!(ok = wait_k(0))) break;
        // the last scores of the piece before have been read
        if (c0 > 0 && !(ok = mbar_wait(&bars->s_free[t], (c0 - 1) & 1, abort_flag, p.status))) break;
        tc_fence_after();
        issue_s(0);
        for (int j = 0; j < blocks; ++j) {
          if (j + 1 < blocks) {
            if (!(ok = mbar_wait(&bars->s_free[t], (c0 + j) & 1, abort_flag, p.status) && wait_k(j + 1))) break;
            tc_fence_after();
            issue_s(j + 1);
          }
          if (!(ok = mbar_wait(&bars->p_full[t], (c0 + j) & 1, abort_flag, p.status) && wait_v(j))) break;
          tc_fence_after();
          issue_pv(j);
        }
        c0 += blocks;
        n0 += blocks;
      }
      // no tensor-core work of this thread may still be in flight when TMEM and shared memory are released
      mma_commit(&bars->drain[t]);
      drain_wait(&bars->drain[t], 0);
    }
  } else {
    regs_increase<kSoftmaxRegs>();
    // ================================ softmax / epilogue =========================================
    const int t = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tbase + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t pbase = sP + t * C::kPBytes, scale0 = smem_addr(bars->scale);
    int c0 = 0;
    bool ok = true;
    for (int s = 0; ok; ++s) {
      if (!(ok = warp_wait(&bars->q_full, s & 1, abort_flag, p.status))) break;
      const Piece& pc = bars->piece[s & 1];
      const int lo = pc.lo, blocks = (pc.hi - lo + kBN - 1) / kBN;
      if (blocks == 0) break;
      const int tile0 = pc.row0 + t * kBM, row = tile0 + r;
      if (tile0 >= rows) {
        n0 += blocks;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_taken);
        continue;
      }
      // keys visible to this row, and to every row of the tile (rows behind the last one are zeros and see all)
      const int lim = row < rows ? min(row_limit(p, pc.len, row), pc.hi) : pc.hi;
      const int all = min(row_limit(p, pc.len, tile0), pc.hi);
      float m = kNone, mo = kNone, qs = 0.f;  // (mo: less kHead)
      uint64_t lsum = f2(0.f, 0.f);
      for (int j = 0; j < blocks; ++j) {
        if (!(ok = warp_wait(&bars->s_full[t], (c0 + j) & 1, abort_flag, p.status))) break;
        tc_fence_after();
        if (j == 0) qs = p.scale_log2 * pow2i(bars->qexp[s & 1][t * kBM + r]);
        const uint32_t scale = scale0 + ((n0 + j) & 3) * 64;  // of the block's eight pairs
        const int key0 = lo + j * kBN;
        const bool masked = key0 + kBN > all;
        uint32_t sr[64];
        auto read = [&](int half) {
          tmem_ld64_sync(lane_base + C::col_s(t) + half * 64, sr);
          if (masked) {
            const int n = lim - key0 - half * 64;
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c >= n) sr[c] = __float_as_uint(-INFINITY);
          }
        };
        float mx = -INFINITY, mv = -INFINITY, lv_min = INFINITY;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          read(half);
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float2 sc = scale_at(scale, half * 4 + h);
            const int c = 16 * h;
            float b0 = fmax3(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]), __uint_as_float(sr[c + 2]));
#pragma unroll
            for (int i = 3; i < 15; i += 2) b0 = fmax3(b0, __uint_as_float(sr[c + i]), __uint_as_float(sr[c + i + 1]));
            b0 = fmaxf(b0, __uint_as_float(sr[c + 15])) * fmaxf(qs * sc.x, 1.17549435e-38f);
            mx = fmaxf(mx, b0);
            mv = fmaxf(mv, b0 + sc.y);
            lv_min = fminf(lv_min, sc.y);
          }
        }
        // The maxima are raised when they are exceeded by more than 2^8 (warp-uniform); O waits below until
        // the product before has landed.
        const bool past = mx > m + kLazy || mv > mo + (kHead + kLazy);
        float alpha = 1.f;
        bool rescale = false;
        if (__any_sync(0xffffffffu, past)) {
          rescale = j > 0;
          if (past) {
            const float m_new = fmaxf(m, mx), mo_new = fmaxf(mo, mv - kHead), a = ex2(m - m_new);
            alpha = ex2(mo - mo_new);
            float l0, l1;
            f2_split(lsum, l0, l1);
            lsum = f2(l0 * a, l1 * a);
            m = m_new;
            mo = mo_new;
          }
        }
        uint64_t acc0 = f2(0.f, 0.f), acc1 = f2(0.f, 0.f);
        const bool own = __any_sync(0xffffffffu, mo - m > lv_min + 64.f);
        uint32_t pk[2][16];
        auto weigh = [&](int half) {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const uint32_t sc = scale + (half * 4 + ch * 2) * 8;
            if (own) weights32<true>(sr, ch, sc, qs, m, mo, acc0, acc1, pk[ch]);
            else weights32<false>(sr, ch, sc, qs, m, mo, acc0, acc1, pk[ch]);
          }
        };
        auto put = [&](int half) {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              sts128(tile_at(pbase, r, half * 8 + ch * 4 + q), pk[ch][4 * q], pk[ch][4 * q + 1], pk[ch][4 * q + 2], pk[ch][4 * q + 3]);
        };
        weigh(1);
        if (j > 0) {  // P and O belong to the product before until it is done
          if (!(ok = warp_wait(&bars->o_done[t], (c0 + j - 1) & 1, abort_flag, p.status))) break;
          tc_fence_after();
        }
        put(1);
        if (rescale) {
#pragma unroll
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t orr[32];
            tmem_ld32_sync(lane_base + C::col_o(t) + ch * 32, orr);
#pragma unroll
            for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha);
            tmem_st32(lane_base + C::col_o(t) + ch * 32, orr);
          }
        }
        read(0);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_free[t]);
        weigh(0);
        put(0);
        lsum = f2_add(lsum, f2_add(acc0, acc1));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (rescale) tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t]);
      }
      if (!ok) break;
      if (!(ok = warp_wait(&bars->o_done[t], (c0 + blocks - 1) & 1, abort_flag, p.status))) break;
      tc_fence_after();
      c0 += blocks;
      n0 += blocks;
      float l0, l1;
      f2_split(lsum, l0, l1);
      const bool none = l0 + l1 == 0.f;  // (not by m: scores of NaN leave that where it was)
      const float f = none ? 0.f : ex2(mo - m + kHead) / (l0 + l1), ls = none ? -INFINITY : (m + lg2(l0 + l1)) * kLn2;
      const int slot = 2 * blockIdx.x + pc.slot;
      const size_t at = pc.whole ? o_row(p, pc.b, pc.hk, min(row, rows - 1)) : static_cast<size_t>(slot) * kUnitRows + t * kBM + r;
      const bool st = row < rows && idx_ok(p.status, at, 1, pc.whole ? static_cast<long long>(p.B) * p.Nq * p.Hq : 2LL * gridDim.x * kUnitRows);
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t orr[32];
        tmem_ld32_sync(lane_base + C::col_o(t) + ch * 32, orr);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(orr[i]) * kUnhead;
        if (!st) {
          // nothing of this row is stored (the loads of O are collective)
        } else if (!pc.whole || o_fp32) {
          float4* out = reinterpret_cast<float4*>((pc.whole ? static_cast<float*>(p.o) : p.ws_o) + at * D + ch * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i) out[i] = make_float4(x[4 * i] * f, x[4 * i + 1] * f, x[4 * i + 2] * f, x[4 * i + 3] * f);
        } else {
          uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + at * D + ch * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            out[i] = make_uint4(pack2<kFp16>(x[8 * i] * f, x[8 * i + 1] * f), pack2<kFp16>(x[8 * i + 2] * f, x[8 * i + 3] * f),
                                pack2<kFp16>(x[8 * i + 4] * f, x[8 * i + 5] * f), pack2<kFp16>(x[8 * i + 6] * f, x[8 * i + 7] * f));
        }
      }
      tc_fence_before();  // O was read before the next piece's products are let go (by p_full)
      if (st) (pc.whole ? p.lse[lse_row(p, pc.b, pc.hk, row)] : p.ws_l[at]) = ls;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->q_taken);
    }
  }

  // ---- teardown -------------------------------------------------------------------------------
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

template <bool kFp16, bool kInt8, int D>
int launch_t(const Attend8Args& a, AttParams& p, cudaStream_t stream) {
  auto kern = kv8_chunk_kernel<kFp16, kInt8, D>;
  static PerContext<int> configured;
  int unused = 0;
  const int ce = configured.get(&unused, [&](int*) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<D>::kSmemBytes);
    if (e != cudaSuccess) return static_cast<int>(e);
    cudaFuncAttributes fattr;
    e = cudaFuncGetAttributes(&fattr, kern);
    if (e != cudaSuccess) return static_cast<int>(e);
    return fattr.numRegs == kLaunchRegs ? 0 : static_cast<int>(cudaErrorInvalidConfiguration);
  });
  if (ce != 0) return ce;
  p.tiles = static_cast<int>((static_cast<long long>(a.Nq) * p.group + kUnitRows - 1) / kUnitRows);
  p.ws_o = static_cast<float*>(a.ws);
  p.ws_l = p.ws_o + static_cast<size_t>(2) * kSms * kUnitRows * D;
  const long long cap = static_cast<long long>(a.c.pages_per_seq) * a.c.page_size;
  p.granule = cap <= kChunkWholeKeys ? kChunkWholeKeys : kBN;
  p.over = p.granule == kBN ? kChunkUnitCost : 0;
  p.least = p.over ? kChunkMinShare : 1;
  const long long most = ((cap + p.granule - 1) / p.granule + p.over) * p.B * p.Hkv * p.tiles;
  const int grid = static_cast<int>(std::min<long long>(kSms, (most + p.least - 1) / p.least));
  kern<<<grid, kChunkThreads, ChunkCfg<D>::kSmemBytes, stream>>>(p, a.o_fp32);
  if (p.over && grid > 1)
    if (const int e = launch_combine8<kFp16, D, kUnitRows>(p, a.o_fp32, grid, stream)) return e;
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

size_t kv8_chunk_ws_bytes(int D) { return static_cast<size_t>(2) * kSms * kUnitRows * (D + 1) * sizeof(float); }

int launch_kv8_chunk(const Attend8Args& a, cudaStream_t stream) {
  AttParams p = params_of(a);
  if (a.c.D == 64) {
    if (a.c.int8) return a.fp16 ? launch_t<true, true, 64>(a, p, stream) : launch_t<false, true, 64>(a, p, stream);
    return a.fp16 ? launch_t<true, false, 64>(a, p, stream) : launch_t<false, false, 64>(a, p, stream);
  }
  if (a.c.int8) return a.fp16 ? launch_t<true, true, 128>(a, p, stream) : launch_t<false, true, 128>(a, p, stream);
  return a.fp16 ? launch_t<true, false, 128>(a, p, stream) : launch_t<false, false, 128>(a, p, stream);
}

}  // namespace fa
