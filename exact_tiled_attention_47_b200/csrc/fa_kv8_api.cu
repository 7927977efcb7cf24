// fa_kv8_api.cu -- the extern "C" boundary of the paged 8-bit cache and of the page operations
// (declared in include/fa.h).  Checks run on the host in the boundary's order: null pointers, element
// types, head dimension, shapes and scale, alignment, workspace, then the device.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_kv8.h"

namespace {

constexpr int64_t k2p31 = static_cast<int64_t>(1) << 31;
constexpr int64_t kMaxKeys = static_cast<int64_t>(1) << 30;

bool page_size_ok(int page_size) { return page_size >= 16 && page_size <= (1 << 16) && (page_size & (page_size - 1)) == 0; }

// Types, head dimension and shapes that the append and the attention share.
int cache_check(int in_dtype, int kv_dtype, int D, int B, int Hkv, int num_pages, int page_size, int pages_per_seq) {
  if (in_dtype != FA_BF16 && in_dtype != FA_FP16) return FA_ERR_DTYPE;
  if (kv_dtype != FA_E4M3 && kv_dtype != FA_INT8) return FA_ERR_DTYPE;
  if (D != 64 && D != 128) return FA_ERR_HEADDIM;
  if (B < 1 || B > 65535 || Hkv < 1 || Hkv > 65535 || num_pages < 1 || pages_per_seq < 1) return FA_ERR_SHAPE;
  if (!page_size_ok(page_size)) return FA_ERR_SHAPE;
  if (static_cast<int64_t>(num_pages) * page_size >= (static_cast<int64_t>(1) << 40) / Hkv) return FA_ERR_SHAPE;
  if (static_cast<int64_t>(pages_per_seq) * page_size > kMaxKeys || static_cast<int64_t>(B) * pages_per_seq >= k2p31)
    return FA_ERR_SHAPE;
  return FA_OK;
}

int launched(int e) {
  if (e == 0) return FA_OK;
  cudaGetLastError();
  return FA_ERR_LAUNCH;
}

fa::Kv8Cache cache_of(const void* k, const void* v, const float* ks, const float* vs, const int* table, const int* seqlens, int B,
                      int Hkv, int num_pages, int page_size, int pages_per_seq, int D, int kv_dtype) {
  fa::Kv8Cache c;
  c.k = const_cast<void*>(k);
  c.v = const_cast<void*>(v);
  c.ks = const_cast<float*>(ks);
  c.vs = const_cast<float*>(vs);
  c.table = table;
  c.seqlens = seqlens;
  c.B = B;
  c.Hkv = Hkv;
  c.D = D;
  c.num_pages = num_pages;
  c.page_size = page_size;
  c.pages_per_seq = pages_per_seq;
  c.int8 = kv_dtype == FA_INT8;
  return c;
}

// Checks that the page operations share: shapes of the state, alignment of its tensors.
int pages_shape(int n, int S, int pages_per_seq, int num_pages, int page_size) {
  if (n < 1 || n > (1 << 20) || S < 1 || S > (1 << 28) || pages_per_seq < 1 || num_pages < 1 || num_pages > (1 << 28)) return FA_ERR_SHAPE;
  if (!page_size_ok(page_size)) return FA_ERR_SHAPE;
  if (static_cast<int64_t>(S) * pages_per_seq >= k2p31 || static_cast<int64_t>(pages_per_seq) * page_size > kMaxKeys) return FA_ERR_SHAPE;
  return FA_OK;
}

int pools_check(const void* const* pools, const size_t* page_bytes, int n_pools) {
  for (int i = 0; i < n_pools; ++i) {
    if (!pools[i]) return FA_ERR_NULL;
    if (page_bytes[i] == 0 || page_bytes[i] > (static_cast<size_t>(1) << 32)) return FA_ERR_SHAPE;
    if (!fa::aligned(pools[i], 4) || page_bytes[i] % 4 != 0) return FA_ERR_ALIGN;
  }
  return FA_OK;
}

int workspace_check(const void* ws, size_t bytes, size_t need) {
  if (!ws || bytes < need) return FA_ERR_WORKSPACE;
  return fa::aligned(ws, 16) ? FA_OK : FA_ERR_ALIGN;
}

bool ints_aligned(std::initializer_list<const int*> ps) {
  for (const int* p : ps)
    if (!fa::aligned(p, 4)) return false;  // (NULL counts as aligned)
  return true;
}

fa::PagesArgs pages_of(int* table, int* seqlens, int* refs, int n, int S, int pages_per_seq, int num_pages, int page_size, void* ws) {
  fa::PagesArgs a{};
  a.table = table;
  a.seqlens = seqlens;
  a.refs = refs;
  a.n = n;
  a.S = S;
  a.pages_per_seq = pages_per_seq;
  a.num_pages = a.dst_pages = num_pages;
  a.page_size = page_size;
  a.ws = static_cast<int*>(ws);
  return a;
}

// The device check and the status word, then the launch.
template <class F, class A>
int run(F launch, A& a, fa_stream_t stream) {
  int dev = -1;
  if (const int st = fa::check_device(&dev)) return st;
  a.status = fa::device_status_ptr();
  if (!a.status) return FA_ERR_LAUNCH;
  return launched(launch(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int fa_kv8_append(const void* k, const void* v, void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                  const int* block_table, const int* seqlens_k, const int* new_lens, int B, int Nt, int Hkv, int num_pages,
                  int page_size, int pages_per_seq, int D, fa_stream_t stream, int in_dtype, int kv_dtype) {
  if (!k || !v || !k_pages || !v_pages || !k_scales || !v_scales || !block_table || !seqlens_k) return FA_ERR_NULL;
  if (const int st = cache_check(in_dtype, kv_dtype, D, B, Hkv, num_pages, page_size, pages_per_seq)) return st;
  if (Nt < 1 || Nt > kMaxKeys) return FA_ERR_SHAPE;
  if (static_cast<int64_t>(B) * (static_cast<int64_t>(Nt) / 16 + 2) * 2 * Hkv >= k2p31 * 8) return FA_ERR_SHAPE;  // one warp each
  if (!fa::aligned(k, 16) || !fa::aligned(v, 16) || !fa::aligned(k_pages, 16) || !fa::aligned(v_pages, 16) || !fa::aligned(k_scales, 4) ||
      !fa::aligned(v_scales, 4) || !ints_aligned({block_table, seqlens_k, new_lens}))
    return FA_ERR_ALIGN;
  fa::AppendArgs a;
  a.c = cache_of(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, Hkv, num_pages, page_size, pages_per_seq, D, kv_dtype);
  a.k = k;
  a.v = v;
  a.new_lens = new_lens;
  a.Nt = Nt;
  a.fp16 = in_dtype == FA_FP16;
  return run(fa::launch_kv8_append, a, stream);
}

size_t fa_kv8_attend_workspace_bytes(int B, int Nq, int Hq, int Hkv, int D) {
  if (B < 1 || Nq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  return fa::kv8_attend_ws_bytes(B, Nq, Hq, Hkv, D);
}

int fa_kv8_attend(const void* q, const void* k_pages, const void* v_pages, const float* k_scales, const float* v_scales,
                  const int* block_table, void* o, float* lse, int B, int Nq, int Hq, int Hkv, int num_pages, int page_size,
                  int pages_per_seq, int D, float scale, const int* seqlens_k, void* workspace, size_t workspace_bytes,
                  fa_stream_t stream, int in_dtype, int kv_dtype, int o_dtype) {
  if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !block_table || !o || !lse) return FA_ERR_NULL;
  if (o_dtype != in_dtype && o_dtype != FA_FP32) return FA_ERR_DTYPE;
  if (const int st = cache_check(in_dtype, kv_dtype, D, B, Hkv, num_pages, page_size, pages_per_seq)) return st;
  if (Nq < 1 || Nq > (1 << 24) || Hq < 1 || Hq > 65535 || Hq % Hkv != 0) return FA_ERR_SHAPE;
  if (static_cast<int64_t>(B) * Nq >= k2p31 / Hq) return FA_ERR_SHAPE;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_SHAPE;
  if (!fa::aligned(q, 16) || !fa::aligned(o, 16) || !fa::aligned(k_pages, 16) || !fa::aligned(v_pages, 16) || !fa::aligned(k_scales, 4) ||
      !fa::aligned(v_scales, 4) || !fa::aligned(lse, 4) || !ints_aligned({block_table, seqlens_k}))
    return FA_ERR_ALIGN;
  if (const int st = workspace_check(workspace, workspace_bytes, fa_kv8_attend_workspace_bytes(B, Nq, Hq, Hkv, D))) return st;
  fa::Attend8Args a;
  a.c = cache_of(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, Hkv, num_pages, page_size, pages_per_seq, D, kv_dtype);
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.ws = workspace;
  a.Nq = Nq;
  a.Hq = Hq;
  a.scale = scale;
  a.fp16 = in_dtype == FA_FP16;
  a.o_fp32 = o_dtype == FA_FP32;
  return run(fa::launch_kv8_attend, a, stream);
}

size_t fa_pages_workspace_bytes(int n, int S, int num_pages) {
  if (n < 1 || n > (1 << 20) || S < 1 || S > (1 << 28) || num_pages < 1 || num_pages > (1 << 28)) return 0;
  return fa::pages_ws_bytes(n, S, num_pages);
}

int fa_pages_extend(int* block_table, int* seqlens, int* refcount, const int* slots, const int* add, int n, int S, int pages_per_seq,
                    int num_pages, int page_size, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (!block_table || !seqlens || !refcount || !add) return FA_ERR_NULL;
  if (const int st = pages_shape(n, S, pages_per_seq, num_pages, page_size)) return st;
  if (!slots && n > S) return FA_ERR_SHAPE;
  if (!ints_aligned({block_table, seqlens, refcount, slots, add})) return FA_ERR_ALIGN;
  if (const int st = workspace_check(workspace, workspace_bytes, fa_pages_workspace_bytes(n, S, num_pages))) return st;
  fa::PagesArgs a = pages_of(block_table, seqlens, refcount, n, S, pages_per_seq, num_pages, page_size, workspace);
  a.a = slots;
  a.b = add;
  return run(fa::launch_pages_extend, a, stream);
}

int fa_pages_free(int* block_table, int* seqlens, int* refcount, const int* slots, int n, int S, int pages_per_seq, int num_pages,
                  int page_size, fa_stream_t stream) {
  if (!block_table || !seqlens || !refcount || !slots) return FA_ERR_NULL;
  if (const int st = pages_shape(n, S, pages_per_seq, num_pages, page_size)) return st;
  if (!ints_aligned({block_table, seqlens, refcount, slots})) return FA_ERR_ALIGN;
  fa::PagesArgs a = pages_of(block_table, seqlens, refcount, n, S, pages_per_seq, num_pages, page_size, nullptr);
  a.a = slots;
  return run(fa::launch_pages_free, a, stream);
}

int fa_pages_fork(int* block_table, int* seqlens, int* refcount, const int* src, const int* dst, int n, int S, int pages_per_seq,
                  int num_pages, int page_size, void* const* pools, const size_t* page_bytes, int n_pools, void* workspace,
                  size_t workspace_bytes, fa_stream_t stream) {
  if (!block_table || !seqlens || !refcount || !src || !dst || (n_pools > 0 && (!pools || !page_bytes))) return FA_ERR_NULL;
  if (const int st = pages_shape(n, S, pages_per_seq, num_pages, page_size)) return st;
  if (n_pools < 0 || n_pools > 65536) return FA_ERR_SHAPE;
  if (const int st = pools_check(pools, page_bytes, n_pools)) return st;
  if (!ints_aligned({block_table, seqlens, refcount, src, dst})) return FA_ERR_ALIGN;
  if (const int st = workspace_check(workspace, workspace_bytes, fa_pages_workspace_bytes(n, S, num_pages))) return st;
  fa::PagesArgs a = pages_of(block_table, seqlens, refcount, n, S, pages_per_seq, num_pages, page_size, workspace);
  a.a = src;
  a.b = dst;
  a.pools = pools;
  a.page_bytes = page_bytes;
  a.n_pools = n_pools;
  return run(fa::launch_pages_fork, a, stream);
}

int fa_pages_compact(const int* block_table, const int* seqlens, const int* refcount, int* block_table_out, int* refcount_out,
                     int* remap, int* n_live, int S, int pages_per_seq, int num_pages, int page_size, void* const* pools,
                     const size_t* page_bytes, int n_pools, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (!block_table || !seqlens || !refcount || !block_table_out || !refcount_out || !remap || !n_live || (n_pools > 0 && (!pools || !page_bytes)))
    return FA_ERR_NULL;
  if (const int st = pages_shape(1, S, pages_per_seq, num_pages, page_size)) return st;
  if (n_pools < 0 || n_pools > 65536) return FA_ERR_SHAPE;
  if (const int st = pools_check(pools, page_bytes, n_pools)) return st;
  if (!ints_aligned({block_table, seqlens, refcount, block_table_out, refcount_out, remap, n_live})) return FA_ERR_ALIGN;
  if (const int st = workspace_check(workspace, workspace_bytes, fa_pages_workspace_bytes(1, S, num_pages))) return st;
  fa::PagesArgs a = pages_of(const_cast<int*>(block_table), const_cast<int*>(seqlens), const_cast<int*>(refcount), 1, S, pages_per_seq,
                             num_pages, page_size, workspace);
  a.table_out = block_table_out;
  a.refs_out = refcount_out;
  a.remap = remap;
  a.n_live = n_live;
  a.pools = pools;
  a.page_bytes = page_bytes;
  a.n_pools = n_pools;
  return run(fa::launch_pages_compact, a, stream);
}

int fa_pages_copy(const void* const* src_pools, void* const* dst_pools, const size_t* page_bytes, int n_pools, const int* src,
                  const int* dst, int n, int src_num_pages, int dst_num_pages, void* workspace, size_t workspace_bytes,
                  fa_stream_t stream) {
  if (!src_pools || !dst_pools || !page_bytes || !src || !dst) return FA_ERR_NULL;
  const int most = src_num_pages > dst_num_pages ? src_num_pages : dst_num_pages;
  if (n_pools < 1 || n_pools > 65536 || src_num_pages < 1 || dst_num_pages < 1) return FA_ERR_SHAPE;
  if (const int st = pages_shape(n, 1, 1, most, 16)) return st;
  if (const int st = pools_check(src_pools, page_bytes, n_pools)) return st;
  if (const int st = pools_check(dst_pools, page_bytes, n_pools)) return st;
  if (!ints_aligned({src, dst})) return FA_ERR_ALIGN;
  if (const int st = workspace_check(workspace, workspace_bytes, fa_pages_workspace_bytes(n, 1, most))) return st;
  fa::PagesArgs a = pages_of(nullptr, nullptr, nullptr, n, 1, 1, most, 16, workspace);
  a.num_pages = src_num_pages;
  a.dst_pages = dst_num_pages;
  a.a = src;
  a.b = dst;
  a.src_pools = src_pools;
  a.pools = dst_pools;
  a.page_bytes = page_bytes;
  a.n_pools = n_pools;
  return run(fa::launch_pages_copy, a, stream);
}

}  // extern "C"
