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
// Rows: the G = Hq / Hkv query heads of a KV head times the Nq tokens, token-major, in tiles of 16 (the M
// of a warp MMA).  CTA = (row tile, KV head; split of the keys; sequence), four warps.  Warp w takes every
// fourth block of 16 keys: a block has one scale per pool and lies in one page, so a warp needs nothing
// from the others until the end.  It streams its blocks (16 x D bytes of K and of V, contiguous in a
// page) through a ring of its own in shared memory with 16-byte cp.async, keys past the end filled with
// zeros, and reads them back as 16-byte (K) and 16- or 8-byte (V) pieces of a row: which k slot of an
// MMA a value takes is free as long as both operands agree, so no transposition is needed but of the
// byte pairs of V (two PRMT per eight codes).  The ring's 16-byte chunks are swizzled so that both reads
// are free of bank conflicts.  Warps and splits are merged by their (m, l, mo, O).
#include <algorithm>

#include "fa_internal.h"
#include "fa_kv8.h"
#include "fa_prefill_common.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kRows = 16;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 6;
constexpr float kLazy = 8.f;  // log2 units by which a maximum may be exceeded before it is raised
constexpr int kStatusPageTable = 12;  // FA_ERR_PAGE_TABLE
constexpr int kMaxSplits = 64;
constexpr int kSplitKeys = 256;  // a split covers at least this many keys

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
  float* ws_o;  // [B * Nq * Hq, S, D]
  float* ws_l;  // [B * Nq * Hq, S]
  int B, Nq, Hq, Hkv, group, tiles, S;
  int num_pages, page_shift, pps;
  float scale_log2;
  int* status;
};

template <int D>
struct Ring {
  static constexpr int kBlock = kKv8Block * D;    // bytes of 16 keys of K or V
  static constexpr int kStage = 2 * kBlock;
  static constexpr int kWarp = kStages * kStage + 128;  // the stages, then (ks, vs) of each, 16 bytes apart
  static constexpr int kMerge = kWarps * kRows * (D + 3) * 4;
  static constexpr int kSmem = kWarps * kWarp > kMerge ? kWarps * kWarp : kMerge;
  static_assert(kStages * 16 <= 128, "scales of the stages");
};

// Byte offset of 16-byte chunk ch of row r of a 16 x D block.  D = 128: a row is one 128-byte line; rows
// 2i and 2i + 1 differ in bit 2 of the chunk (K: lanes read four chunks of two rows at once) and rows 2t
// (or 2t + 1), t = 0..3, in bits 1-2 (V: two chunks of four rows).  D = 64: two rows share a line.
template <int D>
__device__ __forceinline__ uint32_t ring_off(int r, int ch) {
  if constexpr (D == 128) return r * 128 + ((ch ^ (2 * (((r >> 1) & 3) ^ ((r & 1) << 1)))) << 4);
  else return (r >> 1) * 128 + ((((r & 1) * 4 + ch) ^ (2 * ((r >> 1) & 3))) << 4);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(full ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two codes (the low 16 bits) as two fp16 values.
template <bool kInt8>
__device__ __forceinline__ uint32_t half2_of(uint32_t two) {
  uint32_t h;
  if constexpr (kInt8) {
    // code + 128 in the mantissa of 1024: 1024 + (code + 128) - 1152, all exact
    h = __byte_perm(two ^ 0x8080u, 0x64646464u, 0x4140);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
    h = *reinterpret_cast<const uint32_t*>(&x);
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  }
  return h;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <bool kFp16, bool kInt8, int D>
__global__ void __launch_bounds__(kThreads, 2) kv8_attend_kernel(const AttParams p, const int o_fp32) {
  using R = Ring<D>;
  constexpr int LD = D / 64;  // 16-byte pieces of a K row per lane
  constexpr int NT = D / 8;   // 8-column tiles of O
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int tile = blockIdx.x % p.tiles, hk = blockIdx.x / p.tiles, split = blockIdx.y, b = blockIdx.z;
  const int rows = p.Nq * p.group, row0 = tile * kRows;

  const long long cap = static_cast<long long>(p.pps) << p.page_shift;
  int len = static_cast<int>(cap);
  if (p.seqlens) {
    len = __ldg(p.seqlens + b);
    if (len < 0 || len > cap) {
      if (tid == 0 && split == 0 && blockIdx.x == 0) record_status(p.status, kStatusCuSeqlens);
      len = 0;
    }
  }
  // keys that a row of token i sees: len - Nq + i + 1; of the tile: those its last and its first row see
  auto limit = [&](int row) { return max(0, len - p.Nq + row / p.group + 1); };
  const int tile_end = limit(min(rows, row0 + kRows) - 1), tile_all = limit(row0);
  const int per = (max((tile_end + p.S - 1) / p.S, kSplitKeys) + 63) & ~63;
  const int lo = static_cast<int>(min(static_cast<long long>(tile_end), static_cast<long long>(split) * per));
  const int hi = min(tile_end, lo + per);
  int lim[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = row0 + g + 8 * r;
    lim[r] = row < rows ? limit(row) : 0;
  }

  // queries: A operand of row g (and g + 8); piece i of 16 values from d = 16 (t + 4 i)
  uint32_t qa[LD][4][4];
  float qs[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = row0 + g + 8 * r;
    const bool in = row < rows;
    const size_t at = ((static_cast<size_t>(b) * p.Nq + row / p.group) * p.Hq + hk * p.group + row % p.group) * D;
    uint32_t u[LD][8];
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at + 16 * (t + 4 * i));
      const bool ok = in && idx_ok(p.status, at + 16 * (t + 4 * i), 16, static_cast<long long>(p.B) * p.Nq * p.Hq * D);
      const uint4 a = ok ? __ldg(src) : make_uint4(0, 0, 0, 0), c = ok ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
      u[i][0] = a.x; u[i][1] = a.y; u[i][2] = a.z; u[i][3] = a.w;
      u[i][4] = c.x; u[i][5] = c.y; u[i][6] = c.z; u[i][7] = c.w;
    }
    qs[r] = p.scale_log2;
    if constexpr (!kFp16) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < LD; ++i)
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 f = unpack2<false>(u[i][w]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112), 126);
      const float up = pow2i(14 - e);
      qs[r] *= pow2i(e - 14);
#pragma unroll
      for (int i = 0; i < LD; ++i)
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 f = unpack2<false>(u[i][w]);
          u[i][w] = pack2<true>(f.x * up, f.y * up);
        }
    }
#pragma unroll
    for (int i = 0; i < LD; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        qa[i][j][r] = u[i][2 * j];
        qa[i][j][2 + r] = u[i][2 * j + 1];
      }
  }

  float o[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, mo[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  const uint32_t ring = smem_addr(smem) + warp * R::kWarp, ring_s = ring + kStages * R::kStage;
  const int blocks = lo < hi ? ((hi - lo + kKv8Block - 1) / kKv8Block - warp + kWarps - 1) / kWarps : 0;
  const long long pool = (static_cast<long long>(p.num_pages) * p.Hkv) << p.page_shift;
  const int* table = p.table + static_cast<long long>(b) * p.pps;

  auto page_of = [&](int i) {  // page of this warp's block i (-1: none)
    return i < blocks ? __ldg(table + ((lo + (warp + i * kWarps) * kKv8Block) >> p.page_shift)) : -1;
  };
  auto fetch = [&](int i, int page) {
    if (i < blocks) {
      const int key0 = lo + (warp + i * kWarps) * kKv8Block;
      bool ok = page >= 0 && page < p.num_pages;
      if (!ok) {
        if (lane == 0) record_status(p.status, kStatusPageTable);
        page = 0;
      }
      const size_t head = static_cast<size_t>(page) * p.Hkv + hk;
      const int in_page = key0 & ((1 << p.page_shift) - 1);
      const size_t at = ((head << p.page_shift) + in_page) * D;
      const size_t sc = head * ((1 << p.page_shift) / kKv8Block) + in_page / kKv8Block;
      ok = ok && idx_ok(p.status, at, R::kBlock, pool * D) && idx_ok(p.status, sc, 1, pool / kKv8Block);
      const int st = i % kStages;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const int c = j * 32 + lane, r = c / (D / 16), ch = c % (D / 16);
        const bool full = ok && key0 + r < hi;
        const uint32_t dst = ring + st * R::kStage + ring_off<D>(r, ch);
        cp16(dst, p.k + at + c * 16, full);
        cp16(dst + R::kBlock, p.v + at + c * 16, full);
      }
      if (lane < 2) cp4(ring_s + st * 16 + lane * 4, (lane ? p.vs : p.ks) + sc, ok);
    }
    cp_commit();
  };

  int next = page_of(0);
  for (int i = 0; i < kStages - 1; ++i) {
    const int page = next;
    next = page_of(i + 1);
    fetch(i, page);
  }
  for (int i = 0; i < blocks; ++i) {
    {
      const int page = next;
      next = page_of(i + kStages);
      fetch(i + kStages - 1, page);
    }
    cp_wait<kStages - 1>();
    __syncwarp();
    const uint32_t kb = ring + (i % kStages) * R::kStage, vb = kb + R::kBlock;
    float ks, vs;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs) : "r"(ring_s + (i % kStages) * 16) : "memory");
    const int key0 = lo + (warp + i * kWarps) * kKv8Block;

    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int c = 0; c < LD; ++c) {
        const uint4 u = lds128(kb + ring_off<D>(n * 8 + g, t + 4 * c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f16(sc[n], qa[c][j], half2_of<kInt8>(w[j] & 0xFFFFu), half2_of<kInt8>(w[j] >> 16));
      }

    const bool edge = key0 + kKv8Block > min(tile_all, hi);
    const float lv = lg2(fmaxf(vs, 1.17549435e-38f));  // a scale of zero stands for values of zero
    uint32_t pa[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float f = qs[r] * ks;
      float x[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[2 * n + e] = sc[n][2 * r + e] * f;
          if (edge && key0 + 8 * n + 2 * t + e >= min(lim[r], hi)) x[2 * n + e] = -INFINITY;
        }
      float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (mx > m[r] + kLazy) {  // (false while both are -inf)
        l[r] *= ex2(m[r] - mx);
        m[r] = mx;
      }
      const float mv = mx + lv;
      if (mv > mo[r] + kLazy) {
        const float a = ex2(mo[r] - mv);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][2 * r] *= a;
          o[j][2 * r + 1] *= a;
        }
        mo[r] = mv;
      }
      const float mm = m[r] == -INFINITY ? 0.f : m[r], mw = mo[r] == -INFINITY ? 0.f : mo[r] - lv;
      float w[4];
#pragma unroll
      for (int i2 = 0; i2 < 4; ++i2) {
        l[r] += ex2(x[i2] - mm);
        w[i2] = ex2(x[i2] - mw);
      }
      pa[r] = pack2<true>(w[0], w[1]);
      pa[2 + r] = pack2<true>(w[2], w[3]);
    }

    // O += W V: this lane's four keys (2t, 2t + 1 of both halves of the block), D / 8 columns from d = (D / 8) g
    uint32_t v[4][D / 32];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = (k >> 1) * 8 + 2 * t + (k & 1);
      if constexpr (D == 128) {
        const uint4 u = lds128(vb + ring_off<D>(r, g));
        v[k][0] = u.x; v[k][1] = u.y; v[k][2] = u.z; v[k][3] = u.w;
      } else {
        const uint2 u = lds64(vb + ring_off<D>(r, g >> 1) + (g & 1) * 8);
        v[k][0] = u.x; v[k][1] = u.y;
      }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5140), a1 = __byte_perm(v[0][w], v[1][w], 0x7362);
      const uint32_t b0 = __byte_perm(v[2][w], v[3][w], 0x5140), b1 = __byte_perm(v[2][w], v[3][w], 0x7362);
      mma_f16(o[4 * w], pa, half2_of<kInt8>(a0 & 0xFFFFu), half2_of<kInt8>(b0 & 0xFFFFu));
      mma_f16(o[4 * w + 1], pa, half2_of<kInt8>(a0 >> 16), half2_of<kInt8>(b0 >> 16));
      mma_f16(o[4 * w + 2], pa, half2_of<kInt8>(a1 & 0xFFFFu), half2_of<kInt8>(b1 & 0xFFFFu));
      mma_f16(o[4 * w + 3], pa, half2_of<kInt8>(a1 >> 16), half2_of<kInt8>(b1 >> 16));
    }
    __syncwarp();  // every lane has read the stage before the next fetch writes it
  }
  cp_wait<0>();
  __syncthreads();

  // merge of the four warps through shared memory: O [warp][row][d], then m, l, mo [warp][row]
  float* ro = reinterpret_cast<float*>(smem);
  float* rm = ro + kWarps * kRows * D;
  float* rl = rm + kWarps * kRows;
  float* rw = rl + kWarps * kRows;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int row = warp * kRows + g + 8 * r;
    if (t == 0) {
      rm[row] = m[r];
      rl[row] = l[r];
      rw[row] = mo[r];
    }
    // n-tile j, column 2t + e holds d = (D / 8) (2t + e) + j
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < NT; j += 4)
        *reinterpret_cast<float4*>(ro + static_cast<size_t>(row) * D + NT * (2 * t + e) + j) =
            make_float4(o[j][2 * r + e], o[j + 1][2 * r + e], o[j + 2][2 * r + e], o[j + 3][2 * r + e]);
  }
  __syncthreads();
  for (int i = tid; i < kRows * D / 2; i += kThreads) {
    const int row = i / (D / 2), d = i % (D / 2) * 2, rr = row0 + row;
    if (rr >= rows) break;
    float M = -INFINITY, W = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      M = fmaxf(M, rm[w * kRows + row]);
      W = fmaxf(W, rw[w * kRows + row]);
    }
    float sum = 0.f, a = 0.f, c = 0.f;
    if (M > -INFINITY) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        sum += ex2(rm[w * kRows + row] - M) * rl[w * kRows + row];
        const float f = ex2(rw[w * kRows + row] - W);
        const float2 x = *reinterpret_cast<const float2*>(ro + static_cast<size_t>(w * kRows + row) * D + d);
        a += f * x.x;
        c += f * x.y;
      }
      const float f = ex2(W - M) / sum;
      a *= f;
      c *= f;
    }
    const float ls = M > -INFINITY ? (M + lg2(sum)) * kLn2 : -INFINITY;
    const int tok = rr / p.group, hq = hk * p.group + rr % p.group;
    const size_t out = (static_cast<size_t>(b) * p.Nq + tok) * p.Hq + hq;
    const long long outs = static_cast<long long>(p.B) * p.Nq * p.Hq;
    if (!idx_ok(p.status, out, 1, outs)) continue;
    if (p.S == 1) {
      store2<kFp16>(p.o, out * D + d, a, c, o_fp32 != 0);
      if (d == 0) p.lse[(static_cast<size_t>(b) * p.Hq + hq) * p.Nq + tok] = ls;
    } else {
      *reinterpret_cast<float2*>(p.ws_o + (out * p.S + split) * D + d) = make_float2(a, c);
      if (d == 0) p.ws_l[out * p.S + split] = ls;
    }
  }
}

// One warp per output row: O = sum_s exp(lse_s - M) o_s / sum_s exp(lse_s - M), LSE = M + ln of that sum.
template <bool kFp16, int D>
__global__ void __launch_bounds__(128) kv8_combine_kernel(const AttParams p, const int o_fp32) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.B) * p.Nq * p.Hq) return;
  const float* wl = p.ws_l + row * p.S;
  float M = -INFINITY;
  for (int s = lane; s < p.S; s += 32) M = fmaxf(M, wl[s] * kLog2e);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[D / 32] = {}, sum = 0.f;
  if (M > -INFINITY) {
    for (int s = 0; s < p.S; ++s) {
      const float w = ex2(wl[s] * kLog2e - M);
      if (w == 0.f) continue;
      sum += w;
      const float2* x = reinterpret_cast<const float2*>(p.ws_o + (row * p.S + s) * D) + lane * (D / 64);
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        acc[2 * e] = fmaf(w, x[e].x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(w, x[e].y, acc[2 * e + 1]);
      }
    }
    const float inv = 1.f / sum;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] *= inv;
  }
#pragma unroll
  for (int e = 0; e < D / 64; ++e) store2<kFp16>(p.o, row * D + lane * (D / 32) + 2 * e, acc[2 * e], acc[2 * e + 1], o_fp32 != 0);
  if (lane == 0) {
    const int hq = static_cast<int>(row % p.Hq);
    const long long tok = row / p.Hq;
    p.lse[(tok / p.Nq * p.Hq + hq) * p.Nq + tok % p.Nq] = M > -INFINITY ? (M + lg2(sum)) * kLn2 : -INFINITY;
  }
}

// Splits of the keys: enough CTAs for four per SM, at most kMaxSplits.
int splits_for(int B, int Nq, int Hq, int Hkv) {
  const long long units = static_cast<long long>(B) * Hkv * ((static_cast<long long>(Nq) * (Hq / Hkv) + kRows - 1) / kRows);
  return static_cast<int>(std::max(1LL, std::min<long long>(kMaxSplits, (148 * 4 + units - 1) / units)));
}

template <bool kFp16, bool kInt8, int D>
int launch_t(const Attend8Args& a, const AttParams& p, cudaStream_t stream) {
  auto kern = kv8_attend_kernel<kFp16, kInt8, D>;
  static PerContext<int> configured;
  int unused = 0;
  const int ce = configured.get(&unused, [&](int*) {
    return static_cast<int>(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D>::kSmem));
  });
  if (ce != 0) return ce;
  const long long gx = static_cast<long long>(p.tiles) * p.Hkv;
  if (gx > 0x7fffffffLL) return static_cast<int>(cudaErrorInvalidConfiguration);
  kern<<<dim3(static_cast<unsigned>(gx), p.S, p.B), kThreads, Ring<D>::kSmem, stream>>>(p, a.o_fp32);
  if (p.S > 1) {
    const long long rows = static_cast<long long>(p.B) * p.Nq * p.Hq;
    kv8_combine_kernel<kFp16, D><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, stream>>>(p, a.o_fp32);
  }
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

size_t kv8_attend_ws_bytes(int B, int Nq, int Hq, int Hkv, int D) {
  const int S = splits_for(B, Nq, Hq, Hkv);
  if (S == 1) return 256;
  const size_t n = static_cast<size_t>(S) * B * Nq * Hq;
  return (n * (D + 1) * sizeof(float) + 255) & ~static_cast<size_t>(255);
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
  p.tiles = static_cast<int>((static_cast<long long>(a.Nq) * p.group + kRows - 1) / kRows);
  p.S = splits_for(p.B, p.Nq, p.Hq, p.Hkv);
  p.num_pages = a.c.num_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.c.page_size) ++p.page_shift;
  p.pps = a.c.pages_per_seq;
  p.scale_log2 = a.scale * kLog2e;
  p.ws_o = static_cast<float*>(a.ws);
  p.ws_l = p.ws_o + static_cast<size_t>(p.S) * p.B * p.Nq * p.Hq * a.c.D;
  p.status = a.status;
  if (a.c.D == 64) {
    if (a.c.int8) return a.fp16 ? launch_t<true, true, 64>(a, p, stream) : launch_t<false, true, 64>(a, p, stream);
    return a.fp16 ? launch_t<true, false, 64>(a, p, stream) : launch_t<false, false, 64>(a, p, stream);
  }
  if (a.c.int8) return a.fp16 ? launch_t<true, true, 128>(a, p, stream) : launch_t<false, true, 128>(a, p, stream);
  return a.fp16 ? launch_t<true, false, 128>(a, p, stream) : launch_t<false, false, 128>(a, p, stream);
}

}  // namespace fa
