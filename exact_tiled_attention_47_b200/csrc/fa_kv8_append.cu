// fa_kv8_append.cu -- writes new K and V rows into a paged 8-bit cache.
//
// A block is 16 consecutive tokens of one head; its codes share one fp32 scale.  With a = max |x| over
// the block's new values, the block's scale is the smallest power of two s with a <= qmax * s (qmax =
// 448 for e4m3, 127 for int8), at least 2^-126, and not below the scale that older rows of the block
// already have; code = round-to-nearest-even(x / s).  When a newer row raises the scale, the older
// codes are requantised by old / new.  Powers of two keep all of this exact but for the one rounding to
// 8 bits: x / s only moves the exponent, and an e4m3 code that is divided by a power of two loses bits
// only where it becomes subnormal, so a row's value does not drift as later rows come in.  The price is
// up to one bit of an int8 code's range (e4m3 loses nothing but range).
//
// One warp takes one (block, head, K or V): rows are read in 32-byte pieces per lane (D/16 lanes per
// row), the 16 x D values stay in registers between the maximum and the rounding, and each lane writes
// 16 codes at once.  Bound by HBM for prompts (two bytes read and one written per value) and by launch
// latency for single tokens.
#include "fa_internal.h"
#include "fa_kv8.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kAppendWarps = 8;
constexpr int kStatusPageTable = 12;  // FA_ERR_PAGE_TABLE
constexpr int kStatusNonFinite = 13;  // FA_ERR_NONFINITE

struct AppendParams {
  const void* k;
  const void* v;
  void* k_pages;
  void* v_pages;
  float* k_scales;
  float* v_scales;
  const int* table;
  const int* seqlens;
  const int* new_lens;
  int B, Nt, Hkv, num_pages, page_shift, pps, blocks;  // blocks: 16-token blocks that Nt rows can touch
  int* status;
};

// Smallest power of two s >= 2^-126 with a <= qmax * s, for finite a >= 0: the exponent of a, one more
// if its mantissa is above qmax's, less qmax's own exponent.
template <bool kInt8>
__device__ __forceinline__ float block_scale(float a) {
  constexpr uint32_t qmant = kInt8 ? 0x7E0000u : 0x600000u;  // 127 = 1.984375 * 2^6, 448 = 1.75 * 2^8
  constexpr int qexp = kInt8 ? 6 : 8;
  const uint32_t up = __float_as_uint(a) + (0x7FFFFFu - qmant);
  const int e = max(static_cast<int>(up >> 23) - qexp, 1);
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// 1 / s where s is a power of two with a normal reciprocal, else 0 (divide then).
__device__ __forceinline__ float exact_reciprocal(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x807FFFFFu) == 0u && u >= 0x00800000u && u <= 0x7E800000u ? __uint_as_float(0x7F000000u - u) : 0.f;
}

template <bool kInt8>
__device__ __forceinline__ uint32_t code2(float a, float b) {
  if constexpr (kInt8) {
    const int x = __float2int_rn(fminf(fmaxf(a, -127.f), 127.f)), y = __float2int_rn(fminf(fmaxf(b, -127.f), 127.f));
    return (static_cast<uint32_t>(x) & 0xFFu) | ((static_cast<uint32_t>(y) & 0xFFu) << 8);
  } else {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
  }
}

template <bool kInt8>
__device__ __forceinline__ float2 value2(uint32_t two) {  // two codes in the low 16 bits
  if constexpr (kInt8) {
    return make_float2(static_cast<float>(static_cast<int8_t>(two & 0xFFu)), static_cast<float>(static_cast<int8_t>((two >> 8) & 0xFFu)));
  } else {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return unpack2<true>(h);
  }
}

template <bool kFp16, bool kInt8, int D>
__global__ void __launch_bounds__(kAppendWarps * 32, 4) kv8_append_kernel(const AppendParams p) {
  constexpr int LPR = D / 16;        // lanes per row
  constexpr int RPI = 32 / LPR;      // rows per step
  constexpr int IT = kKv8Block / RPI;
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  const int h = static_cast<int>(unit % p.Hkv);
  long long rest = unit / p.Hkv;
  const int kv = static_cast<int>(rest & 1);
  rest >>= 1;
  const int blk = static_cast<int>(rest % p.blocks);
  const long long bl = rest / p.blocks;
  if (bl >= p.B) return;
  const int b = static_cast<int>(bl);
  const uint16_t* x = static_cast<const uint16_t*>(kv ? p.v : p.k);
  uint8_t* pages = static_cast<uint8_t*>(kv ? p.v_pages : p.k_pages);
  float* scales = kv ? p.v_scales : p.k_scales;
  const bool speaks = lane == 0 && h == 0 && kv == 0 && blk == 0;

  const int len = __ldg(p.seqlens + b), n = p.new_lens ? __ldg(p.new_lens + b) : p.Nt;
  if (n < 0 || n > p.Nt || len < n || static_cast<long long>(len) > (static_cast<long long>(p.pps) << p.page_shift)) {
    if (speaks) record_status(p.status, kStatusCuSeqlens);
    return;
  }
  const int first = len - n;
  const int row0 = (first / kKv8Block + blk) * kKv8Block;  // first token of this block
  if (row0 >= len) return;
  const int lo = max(first, row0), hi = min(len, row0 + kKv8Block);
  if (lo >= hi) return;
  const int page = __ldg(p.table + static_cast<long long>(b) * p.pps + (row0 >> p.page_shift));
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) record_status(p.status, kStatusPageTable);
    return;
  }
  const int in_page = row0 & ((1 << p.page_shift) - 1);
  const size_t head = static_cast<size_t>(page) * p.Hkv + h;
  uint8_t* codes = pages + ((head << p.page_shift) + in_page) * D;
  float* scale_at = scales + head * ((1 << p.page_shift) / kKv8Block) + in_page / kKv8Block;
  const long long pool = (static_cast<long long>(p.num_pages) * p.Hkv) << p.page_shift;  // rows of the pool
  if (!idx_ok(p.status, codes - pages, kKv8Block * D, pool * D) ||
      !idx_ok(p.status, scale_at - scales, 1, pool / kKv8Block))
    return;

  // the block's new rows, 16 values of a row per lane and step (row r of the block: step r / RPI)
  const int c = lane % LPR;
  uint32_t raw[IT][8];
  uint32_t most = 0;  // the largest magnitudes: 16-bit values without their sign compare as integers, two at once
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int row = row0 + i * RPI + lane / LPR;
    const size_t at = ((static_cast<size_t>(b) * p.Nt + (row - first)) * p.Hkv + h) * D + c * 16;
    const bool mine = row >= lo && row < hi && idx_ok(p.status, at, 16, static_cast<long long>(p.B) * p.Nt * p.Hkv * D);
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (mine) {
      const uint4* src = reinterpret_cast<const uint4*>(x + at);
      u0 = __ldcs(src);
      u1 = __ldcs(src + 1);
    }
    raw[i][0] = u0.x; raw[i][1] = u0.y; raw[i][2] = u0.z; raw[i][3] = u0.w;
    raw[i][4] = u1.x; raw[i][5] = u1.y; raw[i][6] = u1.z; raw[i][7] = u1.w;
#pragma unroll
    for (int w = 0; w < 8; ++w) most = __vmaxu2(most, raw[i][w] & 0x7FFF7FFFu);
  }
  most = __reduce_max_sync(0xffffffffu, max(most & 0xFFFFu, most >> 16));
  float top = unpack2<kFp16>(most).x;
  const bool finite = most < (kFp16 ? 0x7C00u : 0x7F80u);
  if (!finite) {  // the block holds an infinity or a NaN, which the maximum passes over
    top = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float2 f = unpack2<kFp16>(raw[i][w]);
        const float ax = fabsf(f.x), ay = fabsf(f.y);
        top = fmaxf(top, fmaxf(ax < INFINITY ? ax : 0.f, ay < INFINITY ? ay : 0.f));
      }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) record_status(p.status, kStatusNonFinite);
  }

  float scale = block_scale<kInt8>(top);
  const bool older = first > row0;  // rows of an earlier append share the block
  if (older) {
    const float old = *scale_at;
    scale = fmaxf(scale, old);
    if (scale != old) {  // (warp-uniform) the older codes are rounded again on the larger scale
      const float by = __fdiv_rn(old, scale);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + lane / LPR;
        if (row0 + r < first) {
          uint4* at = reinterpret_cast<uint4*>(codes + r * D + c * 16);
          const uint4 u = *at;
          const uint32_t in[4] = {u.x, u.y, u.z, u.w};
          uint32_t out[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 e = value2<kInt8>(in[w] & 0xFFFFu), f = value2<kInt8>(in[w] >> 16);
            out[w] = code2<kInt8>(e.x * by, e.y * by) | (code2<kInt8>(f.x * by, f.y * by) << 16);
          }
          *at = make_uint4(out[0], out[1], out[2], out[3]);
        }
      }
    }
  }
  __syncwarp();
  if (lane == 0) *scale_at = scale;
  const float inv = exact_reciprocal(scale);
  if (finite && inv != 0.f) {  // every value is at most qmax * scale
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int row = row0 + i * RPI + lane / LPR;
      if (row < lo || row >= hi) continue;
      uint32_t out[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 e = unpack2<kFp16>(raw[i][2 * w]), f = unpack2<kFp16>(raw[i][2 * w + 1]);
        if constexpr (kInt8) {  // x / scale + 1.5 * 2^23 is rounded to an integer, whose low byte is the code
          constexpr float kRound = 12582912.f;
          const uint32_t lo2 = __byte_perm(__float_as_uint(fmaf(e.x, inv, kRound)), __float_as_uint(fmaf(e.y, inv, kRound)), 0x0040);
          const uint32_t hi2 = __byte_perm(__float_as_uint(fmaf(f.x, inv, kRound)), __float_as_uint(fmaf(f.y, inv, kRound)), 0x0040);
          out[w] = __byte_perm(lo2, hi2, 0x5410);
        } else {
          out[w] = __byte_perm(code2<false>(e.x * inv, e.y * inv), code2<false>(f.x * inv, f.y * inv), 0x5410);
        }
      }
      *reinterpret_cast<uint4*>(codes + (row - row0) * D + c * 16) = make_uint4(out[0], out[1], out[2], out[3]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int row = row0 + i * RPI + lane / LPR;
    if (row < lo || row >= hi) continue;
    uint32_t out[4];
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      float2 f = unpack2<kFp16>(raw[i][w]);
      if (f.x != f.x) f.x = 0.f;  // a NaN is stored as zero, an infinity as the largest code
      if (f.y != f.y) f.y = 0.f;
      f.x = inv != 0.f ? f.x * inv : __fdiv_rn(f.x, scale);
      f.y = inv != 0.f ? f.y * inv : __fdiv_rn(f.y, scale);
      const uint32_t two = code2<kInt8>(f.x, f.y);
      out[w / 2] = (w & 1) ? out[w / 2] | (two << 16) : two;
    }
    *reinterpret_cast<uint4*>(codes + (row - row0) * D + c * 16) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

}  // namespace

int launch_kv8_append(const AppendArgs& a, cudaStream_t stream) {
  AppendParams p;
  p.k = a.k;
  p.v = a.v;
  p.k_pages = a.c.k;
  p.v_pages = a.c.v;
  p.k_scales = a.c.ks;
  p.v_scales = a.c.vs;
  p.table = a.c.table;
  p.seqlens = a.c.seqlens;
  p.new_lens = a.new_lens;
  p.B = a.c.B;
  p.Nt = a.Nt;
  p.Hkv = a.c.Hkv;
  p.num_pages = a.c.num_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.c.page_size) ++p.page_shift;
  p.pps = a.c.pages_per_seq;
  p.blocks = (a.Nt + 2 * kKv8Block - 2) / kKv8Block;  // Nt rows from any row of a block
  p.status = a.status;
  const long long units = static_cast<long long>(p.B) * p.blocks * 2 * p.Hkv;
  const long long grid = (units + kAppendWarps - 1) / kAppendWarps;
  if (grid > 0x7fffffffLL) return static_cast<int>(cudaErrorInvalidConfiguration);
  auto go = [&](auto kern) { kern<<<static_cast<unsigned>(grid), kAppendWarps * 32, 0, stream>>>(p); };
  if (a.c.D == 64) {
    if (a.c.int8) a.fp16 ? go(kv8_append_kernel<true, true, 64>) : go(kv8_append_kernel<false, true, 64>);
    else a.fp16 ? go(kv8_append_kernel<true, false, 64>) : go(kv8_append_kernel<false, false, 64>);
  } else {
    if (a.c.int8) a.fp16 ? go(kv8_append_kernel<true, true, 128>) : go(kv8_append_kernel<false, true, 128>);
    else a.fp16 ? go(kv8_append_kernel<true, false, 128>) : go(kv8_append_kernel<false, false, 128>);
  }
  return static_cast<int>(cudaGetLastError());
}

}  // namespace fa
